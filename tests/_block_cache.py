"""FP8 E4M3 caches with a scale per (block, kv head), drawn directly, and the plain definition of
their writes on the CPU, for the tests of the block-scaled operators."""
import torch

F8 = torch.float8_e4m3fn


class BlockCache:
    """Codes and scales of sequences of the given lengths. Rows and pages that no sequence
    owns hold NaN codes and NaN scales. spread: pages' scales differ by up to 2^spread."""

    def __init__(self, lens, kv_heads, D, bs, seed=0, spread=3, spare=2, extra_tokens=0,
                 base=-6):
        g = torch.Generator().manual_seed(seed)
        S = len(lens)
        self.lens, self.H, self.D, self.bs = list(lens), kv_heads, D, bs
        pages = [-(-(n + extra_tokens) // bs) for n in lens]
        self.MB = max([1] + pages)
        NB = sum(pages) + spare
        perm = torch.randperm(NB, generator=g).tolist()
        self.tables = torch.full((S, self.MB), -1, dtype=torch.int32)
        at = 0
        for s in range(S):
            for i in range(pages[s]):
                self.tables[s, i] = perm[at]
                at += 1
        owned = torch.zeros(NB, bs, dtype=torch.bool)
        for s, n in enumerate(lens):
            for t in range(n):
                owned[self.tables[s, t // bs], t % bs] = True
        codes, scales = [], []
        for _ in range(2):
            x = (torch.randn(NB, kv_heads, bs, D, generator=g) * 90).clamp(-448, 448)
            x = x.to(F8).view(torch.uint8)
            codes.append(torch.where(owned[:, None, :, None], x, torch.tensor(0x7F, dtype=torch.uint8)))
            e = torch.randint(0, spread + 1, (NB, kv_heads), generator=g).float()
            scales.append(torch.where(owned.any(1)[:, None], torch.exp2(base - e),
                                      torch.tensor(float("nan"))))
        self.k, self.v = codes
        self.ks, self.vs = scales

    def dev(self):
        """The device copies, made once."""
        if not hasattr(self, "_dev"):
            self._dev = {x: getattr(self, x).cuda() for x in ("k", "v", "ks", "vs", "tables")}
            self._dev["lens"] = torch.tensor(self.lens, dtype=torch.int32).cuda()
        return self._dev

    def rows(self, s, g, n=None):
        """K and V of sequence s, kv head g in 64 bits [n, D], V's codes, V's scales [n]."""
        n = self.lens[s] if n is None else n
        t = torch.arange(n)
        blk, off = self.tables[s].long()[t // self.bs], t % self.bs
        k, v = (x[blk, g, off].view(F8).double().numpy() for x in (self.k, self.v))
        ks, vs = (x[blk, g].double().numpy() for x in (self.ks, self.vs))
        return k * ks[:, None], v * vs[:, None], v, vs


def power_above(a: float) -> float:
    """The smallest power of two s >= 2^-126 with a <= 448 s; 0 for 0."""
    if a == 0:
        return 0.0
    s = 2.0 ** -126
    while 448.0 * s < a:
        s *= 2.0
    return s


def encode(x: torch.Tensor) -> torch.Tensor:
    """E4M3 values of float64 quotients: to binary32 first (exact here or a NaN), then the
    library's cast after saturation."""
    return torch.where(x.isnan(), x, x.clamp(-448, 448)).float().to(F8)


def append(cache_k, cache_v, ks, vs, tables, cu, lens, key, value, bs):
    """pa_append_fp8_block on CPU tensors, in place, page by page."""
    for codes, scales, x in ((cache_k, ks, key), (cache_v, vs, value)):
        vals = codes.view(F8)
        for s, n in enumerate(lens):
            new = cu[s + 1] - cu[s]
            begin = n - new
            if new == 0:
                continue
            for page in range(begin // bs, (n - 1) // bs + 1):
                a, b = max(begin, page * bs), min(n, (page + 1) * bs)
                blk, kept = int(tables[s, page]), a - page * bs
                for h in range(codes.shape[1]):
                    rows = x[cu[s] + a - begin: cu[s] + b - begin, h].double()
                    fin = rows[rows.isfinite()].abs()
                    p = power_above(float(fin.max()) if fin.numel() else 0.0)
                    old = float(scales[blk, h])
                    now = p if kept == 0 else max(p, old)
                    div = now if now else 1.0
                    if kept and now != old:
                        was = vals[blk, h, :kept].double()
                        vals[blk, h, :kept] = encode(was * (old / div))
                    vals[blk, h, kept: kept + b - a] = encode(rows / div)
                    scales[blk, h] = now
