"""What runs between a model's projections and its attention output, as cases to measure.

Five operators over caches [num_blocks, num_kv_heads, block_size, head_dim] reached through
block tables:

  rope     the norm of every query and key head and the rotation by its token's position, in one
           pass; a position has one axis, or several (time, height, width) for images and video
  store    the same, with the keys and the values written to the paged cache
  append   new keys and values written to an FP8 E4M3 cache that holds a scale for each block and
           kv head: a block's scale grows with its rows, and the rows it has are written anew
  decode   attention of one token a sequence over that cache
  prefill  causal attention of the last tokens of each sequence over that cache: a whole prompt,
           or a chunk of one

``own`` chooses between the plain form in elementary torch operations and the calls of
``paged_kv_cache_context_gb300.pa``.
"""
import math

import torch

own = False

GOLD = 0.6180339887498949
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
F8 = torch.float8_e4m3fn


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one user's next token: what counts is the latency of the call
        dict(name="rope_one", op="rope", dtype="bf16", tokens=1, heads=32, kv_heads=8, dim=128,
             rot=128, axes=1, pairs="halves", norm=True),
        # prompts of a batch, packed
        dict(name="rope_prompt", op="rope", dtype="bf16", tokens=16384, heads=32, kv_heads=8,
             dim=128, rot=128, axes=1, pairs="halves", norm=True),
        # the patches of images between text: three axes, a part of each head rotated, neighbours
        # paired
        dict(name="rope_axes", op="rope", dtype="f16", tokens=5003, heads=16, kv_heads=4, dim=96,
             rot=64, axes=3, pairs="neighbours", norm=True),
        # the next tokens of a batch of chats, straight into a cache of the model's type
        dict(name="store_chat", op="store", kv="auto", dtype="bf16", tokens=32, heads=32,
             kv_heads=8, dim=128, bs=32, rot=128, axes=1, pairs="halves", norm=True),
        # chunks of prompts into an FP8 cache, no norms
        dict(name="store_fp8", op="store", kv="fp8", dtype="bf16", tokens=4099, heads=32,
             kv_heads=32, dim=64, bs=32, rot=64, axes=1, pairs="halves", norm=False),
        # the next tokens of a batch of chats
        dict(name="append_chat", op="append", dtype="bf16", seqs=32, kv_heads=8, dim=128, bs=32,
             lo=512, hi=4096, new_lo=1, new_hi=1),
        # the prompts of a batch, ragged, after short cached beginnings
        dict(name="append_prompt", op="append", dtype="bf16", seqs=32, kv_heads=8, dim=128, bs=32,
             lo=512, hi=4096, new_lo=500, new_hi=4096),
        # one user's next token on a short chat
        dict(name="decode_one", op="decode", dtype="bf16", seqs=1, heads=32, kv_heads=8, dim=128,
             bs=32, lo=500, hi=500),
        # the decode workload of a batch of chats
        dict(name="decode_chat", op="decode", dtype="bf16", seqs=32, heads=32, kv_heads=8,
             dim=128, bs=32, lo=512, hi=4096),
        # 64 sequences, one query head a kv head, head_dim 96
        dict(name="decode_wide", op="decode", dtype="f16", seqs=64, heads=32, kv_heads=32, dim=96,
             bs=32, lo=1024, hi=8192),
        # chunks of 512 tokens at the end of a batch of chats
        dict(name="prefill_chunk", op="prefill", dtype="bf16", seqs=32, heads=32, kv_heads=8,
             dim=128, bs=32, lo=512, hi=4096, new_lo=512, new_hi=512),
        # one whole prompt
        dict(name="prefill_prompt", op="prefill", dtype="bf16", seqs=1, heads=32, kv_heads=8,
             dim=128, bs=32, lo=8191, hi=8191, new_lo=8191, new_hi=8191),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope", "store", "append", "decode", "decode", "prefill", "prefill"])
    H = rng.choice([1, 2, 4, 8, 8, 16, 32])
    G = rng.choice([1, 2, 4, 4, 8, 3, 5])
    c = dict(op=op, kv_heads=H)
    if op in ("rope", "store"):
        c["dim"] = rng.choice([64, 96, 128, 128, 80, 256] if op == "rope" else [64, 96, 128])
        c["heads"] = min(H * G, 64 // H * H)
        c["dtype"] = rng.choice(["bf16", "bf16", "f16", "f32"])
        row = (c["heads"] + 2 * H) * c["dim"] * (4 if c["dtype"] == "f32" else 2)
        c["tokens"] = _log_int(rng, 1, min(16384, 160_000_000 // row))
        c["axes"] = rng.choice([1, 1, 3, 2])
        c["rot"] = c["dim"] if rng.random() < 0.6 else 16 * rng.randint(1, c["dim"] // 16)
        c["pairs"] = rng.choice(["halves", "halves", "neighbours"])
        c["norm"] = rng.random() < 0.7
        if op == "store":
            c["kv"] = rng.choice(["auto", "fp8"])
            c["bs"] = rng.choice([16, 32, 32, 64])
        return c
    c["bs"] = rng.choice([16, 32, 32, 64])
    c["dim"] = rng.choice([64, 96, 128, 128])
    c["dtype"] = rng.choice(["bf16", "bf16", "f16"])
    c["seqs"] = _log_int(rng, 1, 64)
    # at most about 200 MB of codes in the batch
    most = max(64, int(1e8 / (c["seqs"] * H * c["dim"])))
    c["hi"] = _log_int(rng, 2, min(16384, most))
    c["lo"] = max(1, int(c["hi"] * rng.uniform(0.2, 1.0)))
    if op == "append":
        c["dtype"] = rng.choice(["bf16", "bf16", "f16", "f32"])
        c["new_hi"] = c["hi"] if rng.random() < 0.3 else _log_int(rng, 1, c["hi"])
        c["new_lo"] = max(1, int(c["new_hi"] * rng.uniform(0.3, 1.0)))
        return c
    c["heads"] = H * G
    if op == "prefill":
        # at most about 1e9 logits in the plain form's padded batch
        top = max(1, int(1e9 / (c["seqs"] * c["heads"] * c["hi"])))
        c["new_hi"] = _log_int(rng, 1, min(top, c["hi"]))
        c["new_lo"] = max(1, int(c["new_hi"] * rng.uniform(0.3, 1.0)))
    return c


def _spread(lo, hi, n, phase=0.0):
    """n whole numbers over [lo, hi], the same for every seed."""
    return [lo + int(((i + 1) * GOLD + phase) % 1.0 * (hi - lo + 1)) for i in range(n)]


def _lens(case):
    return _spread(case["lo"], case["hi"], case["seqs"])


def _news(case):
    """New tokens a sequence, no more than it has."""
    return [min(a, n) for a, n in zip(_spread(case["new_lo"], case["new_hi"], case["seqs"], 0.37),
                                      _lens(case))]


def _size(case):
    return 4 if case["dtype"] == "f32" else 2


def work(case):
    op, H, D = case["op"], case["kv_heads"], case["dim"]
    if op in ("rope", "store"):
        T, e = case["tokens"], _size(case)
        b = T * (case["heads"] + H) * D * e + T * case["heads"] * D * e
        b += 4 * T * case["axes"] + 4 * case["axes"] * case["rot"]
        if op == "rope":
            return {"bytes": b + T * H * D * e, "flops": 0}
        b += T * H * D * e + 8 * T  # values and slots
        return {"bytes": b + 2 * T * H * D * (1 if case["kv"] == "fp8" else e), "flops": 0}
    lens, bs = _lens(case), case["bs"]
    table = 4 * sum(-(-n // bs) for n in lens) + 4 * case["seqs"]
    if op == "append":
        new = _news(case)
        pages = sum((n - 1) // bs - (n - a) // bs + 1 for n, a in zip(lens, new))
        return {"bytes": 2 * sum(new) * H * D * (_size(case) + 1) + 2 * pages * H * 4 +
                4 * pages + 8 * case["seqs"], "flops": 0}
    new = [1] * case["seqs"] if op == "decode" else _news(case)
    pages = sum(-(-n // bs) for n in lens)
    pairs = sum(a * n - a * (a - 1) // 2 for n, a in zip(lens, new))
    return {"bytes": 2 * sum(lens) * H * D + 8 * pages * H + 4 * sum(new) * case["heads"] * D + table,
            "flops": 4 * pairs * case["heads"] * D}


# ------------------------------------------------------------------ inputs
def _inv_freq(case):
    """[axes, rot / 2] radians a position, in 64 bits: a pair of dims turns with one axis."""
    R = case["rot"] // 2
    f = 10000.0 ** (-torch.arange(R, dtype=torch.float64) / R)
    axis = torch.arange(R) * case["axes"] // R
    return torch.where(axis[None, :] == torch.arange(case["axes"])[:, None], f[None, :], 0.0).cuda()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = dict(device="cuda")
    op, H, D, dt = case["op"], case["kv_heads"], case["dim"], DT[case["dtype"]]
    st = dict(case=case)

    def randn(*shape):
        return torch.randn(*shape, generator=g, dtype=torch.float32, **dev)

    if op in ("rope", "store"):
        T, Hq = case["tokens"], case["heads"]
        # the projection's output, a few outlying dims in it
        qkv = randn(T, (Hq + 2 * H) * D) * torch.exp(0.5 * randn((Hq + 2 * H) * D))
        qkv = qkv.to(dt)
        st["q"] = qkv[:, : Hq * D].view(T, Hq, D)
        st["k"] = qkv[:, Hq * D: (Hq + H) * D].view(T, H, D)
        st["qw"] = 1.0 + 0.2 * randn(D) if case["norm"] else None
        st["kw"] = 1.0 + 0.2 * randn(D) if case["norm"] else None
        st["eps"] = 1e-6
        st["freq"] = _inv_freq(case)
        # runs of tokens at places of their own, up to 131072; on the further axes small numbers
        first = torch.randint(0, 131072 - 16384, (-(-T // 512),), generator=g, **dev)
        pos = first.repeat_interleave(512)[:T] + torch.arange(T, **dev) % 512
        more = torch.randint(0, 64, (case["axes"] - 1, T), generator=g, **dev)
        st["pos"] = torch.cat([pos[None, :], more]).int().contiguous()
        st["q_out"] = torch.empty(T, Hq, D, dtype=dt, **dev)
        if op == "rope":
            st["k_out"] = torch.empty(T, H, D, dtype=dt, **dev)
            return st
        st["v"] = qkv[:, (Hq + H) * D:].view(T, H, D)
        bs = case["bs"]
        NB = -(-T // bs) + 3
        slots = torch.randperm(NB * bs, generator=g, **dev)[:T]
        # some tokens are padding
        st["slots"] = torch.where(torch.rand(T, generator=g, **dev) < 0.02, -1, slots)
        st["k_scale"], st["v_scale"] = (1.0 / 32, 1.0 / 16) if case["kv"] == "fp8" else (1.0, 1.0)
        k, v = randn(NB, H, bs, D), randn(NB, H, bs, D)
        if case["kv"] == "fp8":
            st["kc"], st["vc"] = k.to(F8).view(torch.uint8), v.to(F8).view(torch.uint8)
        else:
            st["kc"], st["vc"] = k.to(dt), v.to(dt)
        return st

    S, bs, lens = case["seqs"], case["bs"], _lens(case)
    own_pages = [-(-n // bs) for n in lens]
    NB, MB = sum(own_pages) + 3, max(own_pages)
    perm = torch.randperm(NB, generator=g, **dev).int()
    first = torch.tensor([sum(own_pages[:s]) for s in range(S)], **dev)[:, None]
    page = torch.arange(MB, **dev)[None, :]
    has = page < torch.tensor(own_pages, **dev)[:, None]
    st["tables"] = torch.where(has, perm[(first + page).clamp(max=NB - 1)], -1).int().contiguous()
    st["lens"] = torch.tensor(lens, dtype=torch.int32, **dev)
    # codes that fill a page's range, and scales as the pages' largest values give them
    st["kc"] = (randn(NB, H, bs, D) * 90).clamp_(-448, 448).to(F8).view(torch.uint8)
    st["vc"] = (randn(NB, H, bs, D) * 90).clamp_(-448, 448).to(F8).view(torch.uint8)
    st["ks"] = torch.exp2(torch.randint(-7, -5, (NB, H), generator=g, **dev).float())
    st["vs"] = torch.exp2(torch.randint(-8, -5, (NB, H), generator=g, **dev).float())
    st["scale"] = 1.0 / math.sqrt(D)
    if op == "decode":
        st["q"] = randn(S, case["heads"], D).to(dt)
        st["out"] = torch.empty_like(st["q"])
        return st
    new = _news(case)
    st["new"], st["cu"] = new, torch.tensor([0] + new, **dev).cumsum(0).int()
    if op == "append":
        both = randn(sum(new), 2, H, D) * torch.exp(0.5 * randn(2, H, D)) * torch.exp(
            0.3 * randn(sum(new), 2, 1, 1))
        both = both.to(dt)
        st["key"], st["value"] = both[:, 0], both[:, 1]
        return st
    live = torch.arange(max(new))[None, :] < torch.tensor(new)[:, None]
    st["live"], st["max_new"] = live.cuda(), max(new)
    st["q"] = randn(sum(new), case["heads"], D).to(dt)
    st["out"] = torch.empty_like(st["q"])
    return st


# ------------------------------------------------------------------ plain forms
def _turned(st, x, w):
    """The norm and the rotation in 32 bits; the angles in 64 (positions up to 131072)."""
    case = st["case"]
    R = case["rot"]
    y = x.float()
    if w is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + st["eps"]) * w
    angle = (st["pos"].double()[:, :, None] * st["freq"][:, None, :]).sum(0)
    c, s = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]
    if case["pairs"] == "halves":
        u, v = y[..., : R // 2], y[..., R // 2: R]
        turned = torch.cat([u * c - v * s, v * c + u * s], dim=-1)
    else:
        u, v = y[..., 0:R:2], y[..., 1:R:2]
        turned = torch.stack([u * c - v * s, v * c + u * s], dim=-1).flatten(-2)
    return torch.cat([turned, y[..., R:]], dim=-1)


def _plain_rope(st):
    dt = st["q"].dtype
    return _turned(st, st["q"], st["qw"]).to(dt), _turned(st, st["k"], st["kw"]).to(dt)


def _plain_store(st):
    q, k = _plain_rope(st)
    kc, vc, slots = st["kc"], st["vc"], st["slots"]
    NB, H, bs, D = kc.shape
    used = slots >= 0
    at, head = slots[used], torch.arange(H, device="cuda")[None, :]
    row = ((at[:, None] // bs * H + head) * bs + at[:, None] % bs).reshape(-1)
    for cache, x, scale in ((kc, k, st["k_scale"]), (vc, st["v"], st["v_scale"])):
        x = x[used]
        if cache.dtype == torch.uint8:
            x = (x.float() / scale).clamp(-448, 448).to(F8).view(torch.uint8)
        cache.view(NB * H * bs, D).index_copy_(0, row, x.reshape(-1, D))
    return q, _codes(kc), _codes(vc)


def _codes(cache):
    return cache.view(F8) if cache.dtype == torch.uint8 else cache


def _power(amax):
    """The smallest power of two s with amax <= 448 s, at least 2^-126; 0 for 0."""
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    k = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-126)
    return torch.where(amax == 0, 0.0, torch.ldexp(torch.ones_like(amax), k))


def _plain_append(st):
    tables, lens, cu = st["tables"].long(), st["lens"].long(), st["cu"].long()
    S = lens.numel()
    T, H, D = st["key"].shape
    NB, _, bs, _ = st["kc"].shape
    new = cu[1:] - cu[:-1]
    seq = torch.repeat_interleave(torch.arange(S, device="cuda"), new, output_size=T)
    pos = torch.arange(T, device="cuda") - cu[seq] + (lens - new)[seq]
    block, off = tables[seq, pos // bs], pos % bs
    begin = lens - new                  # where a sequence's new tokens begin
    head_block = tables.gather(1, (begin // bs)[:, None])[:, 0]
    old_rows = begin % bs               # rows its first block has already
    fresh = torch.ones(NB, dtype=torch.bool, device="cuda")
    fresh[head_block] = old_rows == 0
    touched = torch.zeros(NB, dtype=torch.bool, device="cuda")
    touched[block] = True
    keep = torch.arange(bs, device="cuda")[None, :] < old_rows[:, None]
    for x, cache, scales in ((st["key"], st["kc"], st["ks"]), (st["value"], st["vc"], st["vs"])):
        x = x.float()
        amax = torch.zeros(NB, H, device="cuda").scatter_reduce_(
            0, block[:, None].expand(T, H), x.abs().amax(-1), "amax")
        want = _power(amax)
        was = scales.clone()
        now = torch.where(fresh[:, None], want, torch.maximum(want, was))
        scales.copy_(torch.where(touched[:, None], now, was))
        # the rows that the first blocks have, in the new scale
        ratio = (was / torch.where(scales == 0, 1.0, scales))[head_block][:, :, None, None]
        rows = cache[head_block]
        again = (rows.view(F8).float() * ratio).to(F8).view(torch.uint8)
        cache[head_block] = torch.where(keep[:, None, :, None], again, rows)
        s = scales[block][:, :, None]
        code = (x / torch.where(s == 0, 1.0, s)).clamp(-448, 448).to(F8).view(torch.uint8)
        cache[block[:, None], torch.arange(H, device="cuda")[None, :], off[:, None]] = code
    return st["kc"].view(F8), st["vc"].view(F8), st["ks"], st["vs"]


def _rows_of(st, cache, scales):
    """[S, H, MB * bs, D] in 32 bits: every table's blocks in order."""
    at = st["tables"].long().clamp(min=0)
    S, MB = at.shape
    _, H, bs, D = cache.shape
    x = cache[at].view(F8).float() * scales[at][..., None, None]
    return x.permute(0, 2, 1, 3, 4).reshape(S, H, MB * bs, D)


def _attend(q, k, v, see, scale):
    """Softmax attention of q [S, H, R, D]; see [S, 1, R, L] or [S, 1, 1, L]."""
    x = ((q.float() @ k.transpose(-1, -2)) * scale).masked_fill(~see, -math.inf)
    top = x.amax(-1, keepdim=True)
    e = (x - torch.where(top == -math.inf, 0.0, top)).exp()
    total = e.sum(-1, keepdim=True)
    return (e @ v) / torch.where(total == 0, 1.0, total)


def _plain_decode(st):
    case = st["case"]
    S, H, G, D = case["seqs"], case["kv_heads"], case["heads"] // case["kv_heads"], case["dim"]
    k, v = _rows_of(st, st["kc"], st["ks"]), _rows_of(st, st["vc"], st["vs"])
    see = torch.arange(k.shape[2], device="cuda")[None, :] < st["lens"][:, None]
    o = _attend(st["q"].view(S, H, G, D), k, v, see[:, None, None, :], st["scale"])
    return o.reshape(S, H * G, D).to(st["q"].dtype)


def _plain_prefill(st):
    case = st["case"]
    S, N = st["live"].shape
    H, G, D = case["kv_heads"], case["heads"] // case["kv_heads"], case["dim"]
    k, v = _rows_of(st, st["kc"], st["ks"]), _rows_of(st, st["vc"], st["vs"])
    cu, n = st["cu"].long(), st["lens"].long()
    spot = (cu[:-1, None] + torch.arange(N, device="cuda")).clamp(max=st["q"].shape[0] - 1)
    q = st["q"][spot].view(S, N, H, G, D).permute(0, 2, 1, 3, 4).reshape(S, H, N * G, D)
    at = torch.arange(k.shape[2], device="cuda")
    last = (n - (cu[1:] - cu[:-1]))[:, None] + torch.arange(N, device="cuda")  # a row's position
    see = at[None, None, :] <= torch.minimum(last, n[:, None] - 1)[:, :, None]
    see = see[:, None, :, None, :].expand(S, 1, N, G, -1).reshape(S, 1, N * G, -1)
    o = _attend(q, k, v, see, st["scale"])
    o = o.view(S, H, N, G, D).permute(0, 2, 1, 3, 4).reshape(S, N, H * G, D)
    return o[st["live"]].to(st["q"].dtype)


# ------------------------------------------------------------------ one pass
def run(st):
    case = st["case"]
    op = case["op"]
    if not own:
        return {"rope": _plain_rope, "store": _plain_store, "append": _plain_append,
                "decode": _plain_decode, "prefill": _plain_prefill}[op](st)
    from paged_kv_cache_context_gb300 import pa
    if op in ("rope", "store"):
        turns = st.get("turns")
        if turns is None:  # made once, as weights are
            turns = st["turns"] = pa.rope_turns(st["freq"])
        rest = dict(q_weight=st["qw"], k_weight=st["kw"], eps=st["eps"],
                    interleaved=case["pairs"] == "neighbours")
        if op == "rope":
            pa.norm_rope(st["q_out"], st["k_out"], st["q"], st["k"], turns, st["pos"], **rest)
            return st["q_out"], st["k_out"]
        pa.norm_rope_and_cache(st["q_out"], st["q"], st["k"], st["v"], st["kc"], st["vc"],
                               st["slots"], turns, st["pos"],
                               kv_dtype="fp8_e4m3" if case["kv"] == "fp8" else "auto",
                               k_scale=st["k_scale"], v_scale=st["v_scale"], **rest)
        return st["q_out"], _codes(st["kc"]), _codes(st["vc"])
    cache = (st["kc"], st["vc"], st["ks"], st["vs"], st["tables"])
    if op == "append":
        pa.append_fp8_block(st["key"], st["value"], *cache, st["cu"], st["lens"])
        return st["kc"].view(F8), st["vc"].view(F8), st["ks"], st["vs"]
    ws = st.get("ws")
    if ws is None:
        if op == "decode":
            size = pa.decode_workspace_size(case["seqs"], case["heads"], case["kv_heads"],
                                            case["dim"], case["bs"], st["tables"].shape[1])
        else:
            size = pa.prefill_fp8_block_workspace_size(case["heads"], case["kv_heads"],
                                                       case["dim"])
        ws = st["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    if op == "decode":
        pa.decode_fp8_block(st["out"], st["q"], *cache, st["lens"], case["kv_heads"],
                            st["scale"], ws)
    else:
        pa.prefill_fp8_block(st["out"], st["q"], *cache, st["cu"], st["lens"], case["kv_heads"],
                             st["max_new"], st["scale"], ws)
    return st["out"]


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_turn(st, x, w):
    """Row by row of the definition, as complex numbers."""
    case = st["case"]
    R = case["rot"]
    y = x.double()
    if w is not None:
        y = y / (y.pow(2).sum(-1, keepdim=True) / case["dim"] + st["eps"]).sqrt() * w.double()
    angle = torch.einsum("at,ai->ti", st["pos"].double(), st["freq"])
    turn = torch.polar(torch.ones_like(angle), angle)[:, None, :]
    r = y[..., :R]
    z = torch.complex(r[..., : R // 2], r[..., R // 2:]) if case["pairs"] == "halves" else \
        torch.view_as_complex(r.reshape(*r.shape[:-1], R // 2, 2).contiguous())
    z = z * turn
    out = y.clone()
    out[..., :R] = torch.cat([z.real, z.imag], -1) if case["pairs"] == "halves" else \
        torch.view_as_real(z).flatten(-2)
    return out


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("rope", "store"):
        q, k = _exact_turn(st, st["q"], st["qw"]), _exact_turn(st, st["k"], st["kw"])
        if op == "rope":
            return q, k
        got = [q]
        for cache, x, scale in ((st["kc"], k, st["k_scale"]), (st["vc"], st["v"], st["v_scale"])):
            full = _codes(cache).double()
            slots = st["slots"]
            at = slots[slots >= 0]
            x = x.double()[slots >= 0]
            if cache.dtype == torch.uint8:
                x = (x / scale).clamp(-448.0, 448.0)
            full.transpose(1, 2)[at // case["bs"], at % case["bs"]] = x
            got.append(full)
        return got
    lens, bs = _lens(case), case["bs"]
    if op == "append":
        if sum(_news(case)) > 40000:
            return None
        got = []
        cu = st["cu"].tolist()
        for x, cache, scales in ((st["key"], st["kc"], st["ks"]), (st["value"], st["vc"], st["vs"])):
            codes, sc = cache.view(F8).double(), scales.double()
            for s in range(case["seqs"]):
                begin = lens[s] - (cu[s + 1] - cu[s])
                for p in range(begin // bs, (lens[s] - 1) // bs + 1):
                    a, b = max(begin, p * bs), min(lens[s], (p + 1) * bs)
                    rows = x[cu[s] + a - begin: cu[s] + b - begin].double().transpose(0, 1)
                    blk, kept = int(st["tables"][s, p]), a - p * bs
                    top = rows.abs().amax((1, 2))
                    m, e = torch.frexp(top / 448.0)  # a quotient that is a power of two has m 0.5
                    e = torch.where(m == 0.5, e - 1, e).clamp(min=-126)
                    s2 = torch.where(top == 0, 0.0, torch.ldexp(torch.ones_like(top), e))
                    old = sc[blk].clone()
                    sc[blk] = s2 if kept == 0 else torch.maximum(s2, old)
                    div = torch.where(sc[blk] == 0, 1.0, sc[blk])[:, None, None]
                    codes[blk, :, :kept] = codes[blk, :, :kept] * (old[:, None, None] / div)
                    codes[blk, :, kept: kept + b - a] = rows / div
            got.append((codes, sc))
        return got[0][0], got[1][0], got[0][1], got[1][1]
    out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    cu = list(range(case["seqs"] + 1)) if op == "decode" else st["cu"].tolist()
    G = case["heads"] // case["kv_heads"]
    for s in range(case["seqs"]):
        pages = st["tables"][s, : -(-lens[s] // bs)].long()
        K, V = (torch.cat(list(c[pages].view(F8).double() * sc[pages].double()[:, :, None, None]),
                          dim=1)[:, : lens[s]] for c, sc in ((st["kc"], st["ks"]),
                                                             (st["vc"], st["vs"])))
        t = cu[s + 1] - cu[s]
        hidden = torch.ones(t, lens[s], dtype=torch.bool, device="cuda").triu(lens[s] - t + 1)
        for h in range(case["heads"]):
            x = st["q"][cu[s]: cu[s + 1], h].double() @ K[h // G].T * st["scale"]
            out[cu[s]: cu[s + 1], h] = torch.softmax(x.masked_fill(hidden, -math.inf), -1) @ V[h // G]
    return out
