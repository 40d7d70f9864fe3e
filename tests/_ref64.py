"""Paged caches drawn directly, and attention over them in 64 bits, for the
tests of the tree, scored-decode and eviction operators.

Error bounds (u(t) = finfo(t).eps / 2, the relative size of one rounding to t):
with p the exact weights and A = sum_j p_j |V_j|,
  * a logit's absolute error is at most d = (D + 8) 2^-23 scale sum_d |q_d K_jd| (products
    exact or rounded once, an accumulation in 32 bits that may truncate, the scale and the
    subtraction of the maximum), so a weight's relative error is at most
    e = 2 d + (L + 16) 2^-23 (its own and the sum's, L summands, the exponential's 2 ulp);
  * the weights are rounded once to the type w that the products take: u(w) A, and where w
    is f16 at most half its smallest step, 2^-25, per unit of |V| besides (weights are held
    relative to a sum of at least one);
  * the output is rounded once: u(out) |o|.
"""
import math

import numpy as np
import torch

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


class Cache:
    """Caches with NaN (or the highest code) in every row that no sequence owns."""

    def __init__(self, lens, kv_heads, D, bs, kv="auto", dtype=torch.bfloat16, seed=0, spare=2,
                 extra_tokens=0):
        g = torch.Generator().manual_seed(seed)
        S = len(lens)
        self.lens, self.H, self.D, self.bs, self.kv, self.dtype = list(lens), kv_heads, D, bs, kv, dtype
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
        shape = (NB, kv_heads, bs, D)
        self.k_scale = self.v_scale = 1.0
        self.ks = self.vs = None
        owned = torch.zeros(NB, bs, dtype=torch.bool)
        for s, n in enumerate(lens):
            for t in range(n):
                owned[self.tables[s, t // bs], t % bs] = True
        ow = owned[:, None, :, None].expand(shape)
        if kv == "int8":
            self.k = torch.randint(-127, 128, shape, generator=g, dtype=torch.int8)
            self.v = torch.randint(-127, 128, shape, generator=g, dtype=torch.int8)
            nan = torch.tensor(float("nan"))
            sc = [(0.5 + torch.rand(shape[:3], generator=g)) * (1.7 / 127) for _ in range(2)]
            self.ks, self.vs = (torch.where(ow[..., 0], x, nan) for x in sc)
        elif kv == "fp8_e4m3":
            self.k_scale, self.v_scale = 0.03125, 0.0208740234375
            for name, f in (("k", 32.0), ("v", 48.0)):
                x = (torch.randn(shape, generator=g) * f).clamp(-448, 448)
                x = x.to(torch.float8_e4m3fn).view(torch.uint8)
                setattr(self, name, torch.where(ow, x, torch.tensor(0x7F, dtype=torch.uint8)))
        else:
            for name in ("k", "v"):
                x = torch.randn(shape, generator=g).to(dtype)
                setattr(self, name, torch.where(ow, x, torch.tensor(float("nan"), dtype=dtype)))

    def dev(self):
        """The device copies, made once."""
        if not hasattr(self, "_dev"):
            names = [x for x in ("k", "v", "ks", "vs") if getattr(self, x) is not None]
            self._dev = {x: getattr(self, x).cuda() for x in names}
            self._dev["tables"] = self.tables.cuda()
            self._dev["lens"] = torch.tensor(self.lens, dtype=torch.int32).cuda()
        return self._dev

    def rows(self, s, g, n=None):
        """K and V of sequence s, kv head g in 64 bits [n, D], and V's codes."""
        n = self.lens[s] if n is None else n
        t = torch.arange(n)
        blk, off = self.tables[s].long()[t // self.bs], t % self.bs
        out = []
        for x, sc, one in ((self.k, self.ks, self.k_scale), (self.v, self.vs, self.v_scale)):
            r = x[blk, g, off]
            r = (r.view(torch.float8_e4m3fn) if self.kv == "fp8_e4m3" else r).double().numpy()
            out.append(r)
            out.append(r * (sc[blk, g, off].double().numpy()[:, None] if sc is not None else one))
        return out[1], out[3], out[2]


def attend(q, K, V, codes, seen, scale, out_dtype, w_dtype):
    """(output, its error bound, weights, their relative error) of one row q [D]; seen bool [n]."""
    D = q.shape[0]
    if not seen.any():
        return np.zeros(D), np.zeros(D), np.zeros(len(seen)), 0.0
    idx = np.nonzero(seen)[0]
    Ks, Vs = K[idx], V[idx]
    x = Ks @ q * scale
    e = np.exp(x - x.max())
    p = e / e.sum()
    o = p @ Vs
    A = p @ np.abs(Vs)
    d = (D + 8) * 2.0 ** -23 * abs(scale) * (np.abs(Ks) @ np.abs(q)).max()
    rel = 2 * d + (len(idx) + 16) * 2.0 ** -23
    bound = (U[w_dtype] * 1.01 + rel) * A + U[out_dtype] * 1.01 * np.abs(o)
    if w_dtype == torch.float16:
        # (8-bit caches: the rounded weight meets the codes)
        bound = bound + 2.0 ** -25 * np.maximum(np.abs(codes[idx]), np.abs(Vs)).sum(0)
    full = np.zeros(len(seen))
    full[idx] = p
    return o, bound + 1e-30, full, rel


def weight_type(cache, dtype):
    """What the tensor-core products round the weights to."""
    return torch.float16 if cache.kv != "auto" else dtype


def bits64(words, n):
    """bool [n] of a row of int64 words."""
    w = [int(x) & (1 << 64) - 1 for x in words]
    return np.array([(w[k // 64] >> (k % 64)) & 1 if k // 64 < len(w) else 0 for k in range(n)],
                    dtype=bool)


def default_scale(D):
    return 1.0 / math.sqrt(D)
