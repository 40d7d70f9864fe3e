"""The block-scaled FP8 cache on the GPU: the write bit for bit against its plain definition, the
decode against attention in 64 bits over the same codes and scales.

The decode's bounds: tests/_ref64.py, with f16 weights. The product of weight and V scale is what is
rounded, relative to the largest product of weight and scale in a page or two of the row (at
least 2^6 units): half of f16's smallest step, 2^-25, is 2^-31 of it for each unit of |code|."""
import numpy as np
import pytest
import torch

import _block_cache as bc
from _block_cache import BlockCache
from _ref64 import attend, default_scale
from paged_kv_cache_context_gb300 import pa

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def draw_rows(T, H, D, dtype, seed, grow=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, 2, H, D, generator=g) * torch.exp(torch.randn(T, 1, 1, 1, generator=g))
    x = (x * grow).to(dtype)
    return x[:, 0], x[:, 1]


def same(a, b):
    """Equal codes, any NaN code for any other."""
    a, b = a.cpu(), b.cpu()
    nan = ((a & 0x7F) == 0x7F) & ((b & 0x7F) == 0x7F)
    return bool(((a == b) | nan).all())


class Pool:
    """The same cache on both sides, of sequences that grow up to `cap` tokens."""

    def __init__(self, S, cap, H, D, bs, seed):
        self.c = BlockCache([0] * S, H, D, bs, seed=seed, extra_tokens=cap)
        g = torch.Generator().manual_seed(seed)
        for x in ("k", "v"):  # pages hold anything before they are used
            t = getattr(self.c, x)
            t.copy_(torch.randint(0, 256, t.shape, generator=g, dtype=torch.uint8))
        self.d = {x: v.clone() for x, v in self.c.dev().items()}
        self.bs, self.lens = bs, [0] * S

    def step(self, news, key, value, strided=True):
        self.lens = [a + b for a, b in zip(self.lens, news)]
        cu = [0]
        for a in news:
            cu.append(cu[-1] + a)
        c, d = self.c, self.d
        bc.append(c.k, c.v, c.ks, c.vs, c.tables, cu, self.lens, key, value, self.bs)
        if strided:  # views of one buffer
            both = torch.stack([key, value], 1).cuda()
            k, v = both[:, 0], both[:, 1]
        else:
            k, v = key.contiguous().cuda(), value.contiguous().cuda()
        pa.append_fp8_block(k, v, d["k"], d["v"], d["ks"], d["vs"], d["tables"], i32(cu),
                            i32(self.lens))
        assert pa.get_device_error() == 0
        self.same()

    def same(self):
        c, d = self.c, self.d
        for x in ("ks", "vs"):
            assert torch.equal(d[x].cpu().view(torch.int32), getattr(c, x).view(torch.int32)), x
        assert same(d["k"], c.k) and same(d["v"], c.v)


APPENDS = [
    # D, H, bs, dtype, steps of new tokens a sequence
    (128, 2, 32, torch.bfloat16, [[5, 0, 33], [1, 1, 1], [1, 64, 1], [0, 0, 1], [31, 2, 100]]),
    (64, 3, 16, torch.float16, [[16, 1], [1, 15], [1, 1], [40, 3]]),
    (96, 1, 64, torch.float32, [[1], [62], [1], [1], [130]]),
    (128, 1, 64, torch.float32, [[64, 63], [1, 1], [200, 70]]),
    (128, 8, 32, torch.bfloat16, [[1] * 40, [1] * 40, [(7 * s) % 40 for s in range(40)], [1] * 40]),
    (96, 2, 32, torch.bfloat16, [[0] * 33 + [70] + [0] * 40 + [3], [1] * 75]),
    (64, 1, 16, torch.bfloat16, [[1000], [1]]),
]


@pytest.mark.parametrize("D,H,bs,dtype,steps", APPENDS)
def test_append_is_its_definition_bit_for_bit(D, H, bs, dtype, steps):
    pa.get_device_error()
    S = len(steps[0])
    cap = max(sum(st[s] for st in steps) for s in range(S))
    pool = Pool(S, cap, H, D, bs, D + H)
    for i, news in enumerate(steps):
        pool.step(news, *draw_rows(sum(news), H, D, dtype, 10 * D + i, 1.5 ** i), strided=i % 2 == 0)


def test_scales_grow_far_and_stay():
    """Tokens that are larger each time, then smaller; zeros first."""
    pool = Pool(1, 32, 2, 64, 32, 3)
    key, value = draw_rows(12, 2, 64, torch.float32, 4)
    for i, f in enumerate((0.0, 0.0, 1e-38, 1e-30, 1e-6, 1.0, 1.0, 300.0, 1e4, 1.0, 1e30, 1e-3)):
        pool.step([1], key[i:i + 1] * f, value[i:i + 1] * f)
    assert float(pool.d["ks"][pool.c.tables[0, 0].item()].max()) > 1e26


def test_values_that_are_not_finite():
    pool = Pool(2, 40, 1, 64, 16, 5)
    key, value = draw_rows(20, 1, 64, torch.bfloat16, 6)
    key[3, 0, 1], key[4, 0, 2], value[5, 0, 3] = float("inf"), float("-inf"), float("nan")
    value[6:8] = float("nan")
    pool.step([10, 10], key, value)
    only = torch.full((2, 1, 64), float("inf"), dtype=torch.bfloat16)
    pool.step([1, 1], only, only)
    pool.step([7, 7], *draw_rows(14, 1, 64, torch.bfloat16, 7, 50.0))


def test_append_leaves_what_it_does_not_own():
    """Bad offsets, lengths and blocks are flagged, and other sequences are written all the same."""
    pa.get_device_error()
    H, D, bs = 2, 128, 32
    for what, bit in (("cu", 16), ("len", 4), ("long", 4), ("block", 2)):
        pool = Pool(3, 70, H, D, bs, 11)
        key, value = draw_rows(60, H, D, torch.bfloat16, 12)
        cu, lens = [0, 20, 40, 60], [20, 20, 20]
        tables = pool.d["tables"].clone()
        if what == "cu":
            cu[2] = 15  # the second has a negative length, the third more tokens than positions
            lens = [20, 20, 45]
        elif what == "len":
            lens[1] = 19
        elif what == "long":
            lens[1] = tables.shape[1] * bs + 1
        else:
            tables[1, 0] = 10 ** 6
        k, v = key.cuda(), value.cuda()
        before = {x: y.clone() for x, y in pool.d.items()}
        pa.append_fp8_block(k, v, pool.d["k"], pool.d["v"], pool.d["ks"], pool.d["vs"], tables,
                            i32(cu), i32(lens))
        assert pa.get_device_error() == bit, what
        c = pool.c
        good = [(0, 20), (0, 0), (15, 60)] if what == "cu" else [(0, 20), (0, 0), (40, 60)]
        for s, (a, b) in enumerate(good):
            if b > a:
                bc.append(c.k, c.v, c.ks, c.vs, c.tables[s:s + 1], [0, b - a], [lens[s]], key[a:b],
                          value[a:b], bs)
        pool.same()
        own = c.tables[1][c.tables[1] >= 0].long()
        assert torch.equal(before["k"][own], pool.d["k"][own])


def test_append_captured_and_replayed_on_another_stream():
    a, b = Pool(4, 100, 2, 128, 32, 20), Pool(4, 100, 2, 128, 32, 20)
    first = draw_rows(160, 2, 128, torch.bfloat16, 21)
    a.step([40] * 4, *first)
    b.step([40] * 4, *first)
    key, value = (x.contiguous().cuda() for x in draw_rows(4, 2, 128, torch.bfloat16, 22, 9.0))
    cu, lens = i32([0, 1, 2, 3, 4]), i32([41] * 4)
    st = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    args = [b.d[x] for x in ("k", "v", "ks", "vs", "tables")]
    with torch.cuda.graph(graph, stream=st):
        pa.append_fp8_block(key, value, *args, cu, lens)
    for i in range(3):
        new = draw_rows(4, 2, 128, torch.bfloat16, 30 + i, 3.0 ** i)
        a.step([1] * 4, *new)
        key.copy_(new[0])
        value.copy_(new[1])
        lens.fill_(41 + i)
        graph.replay()
    torch.cuda.synchronize()
    for x in ("k", "v", "ks", "vs"):
        assert torch.equal(a.d[x].view(torch.uint8), b.d[x].view(torch.uint8)), x


# ------------------------------------------------------------------ decode
def workspace(S, Hq, c):
    n = pa.decode_workspace_size(S, Hq, c.H, c.D, c.bs, c.MB)
    return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")


def decode(c, q, scale, ws=None, out=None, stream=None):
    d = c.dev()
    ws = workspace(q.shape[0], q.shape[1], c) if ws is None else ws
    out = torch.full_like(q, float("nan")) if out is None else out
    pa.decode_fp8_block(out, q, d["k"], d["v"], d["ks"], d["vs"], d["tables"], d["lens"], c.H, scale,
                        ws, stream=stream)
    return out


def row_bound(q, K, V, codes, vs, seen, scale, dtype):
    o, bound, p, _ = attend(q, K, V, np.zeros_like(codes), seen, scale, dtype, torch.float16)
    if seen.any():
        bound = bound + 2.0 ** -31 * p.max() * vs[seen].max() * np.abs(codes[seen]).sum(0)
    return o, bound


def check_decode(c, G, q, out, scale):
    got, qd = out.double().cpu().numpy(), q.double().cpu().numpy()
    for s, n in enumerate(c.lens):
        for g in range(c.H):
            K, V, codes, vs = c.rows(s, g)
            for h in range(g * G, (g + 1) * G):
                o, bound = row_bound(qd[s, h], K, V, codes, vs, np.ones(n, bool), scale, q.dtype)
                assert (np.abs(got[s, h] - o) <= bound).all(), (s, h)


DECODES = [
    # dtype, D, Hkv, G, bs, lens, spread
    (torch.bfloat16, 128, 2, 4, 32, [1, 31, 32, 33, 0, 500], 3),
    (torch.float16, 128, 1, 8, 16, [1, 15, 16, 17, 1000], 8),
    (torch.bfloat16, 96, 4, 1, 32, [1, 100, 333], 0),
    (torch.float16, 96, 2, 3, 64, [128, 1, 63, 65], 5),
    (torch.bfloat16, 64, 1, 5, 16, [(13 * s) % 70 for s in range(40)], 3),
    (torch.bfloat16, 64, 8, 2, 64, [700, 64], 12),
    (torch.bfloat16, 128, 1, 4, 32, [9000], 3),
    (torch.float16, 64, 1, 1, 16, [3], 3),
]


@pytest.mark.parametrize("dtype,D,Hkv,G,bs,lens,spread", DECODES)
def test_decode_matches_the_definition(dtype, D, Hkv, G, bs, lens, spread):
    pa.get_device_error()
    c = BlockCache(lens, Hkv, D, bs, seed=D + G, spread=spread)
    g = torch.Generator().manual_seed(3)
    q = (torch.randn(len(lens), Hkv * G, D, generator=g) * 1.5).to(dtype)
    out = decode(c, q.cuda(), default_scale(D))
    assert pa.get_device_error() == 0
    check_decode(c, G, q, out, default_scale(D))
    assert torch.equal(out, decode(c, q.cuda(), default_scale(D)))  # the same bits again


@pytest.mark.parametrize("base", [-58, -30, 20, 50])
def test_decode_over_small_and_large_scales(base):
    c = BlockCache([300, 40], 2, 128, 32, seed=base % 97, spread=2, base=base)
    c.ks = torch.where(c.ks.isnan(), c.ks, torch.exp2(c.ks.log2() - base - 6))  # K as usual
    g = torch.Generator().manual_seed(4)
    q = torch.randn(2, 8, 128, generator=g).to(torch.bfloat16)
    out = decode(c, q.cuda(), default_scale(128))
    check_decode(c, 4, q, out, default_scale(128))


def test_decode_with_pages_of_zeros_beside_others():
    """A scale of zero: the page's logits and values are zero, its weights count."""
    c = BlockCache([200], 1, 64, 16, seed=8, spread=2)
    for p in (0, 3, 7):
        blk = int(c.tables[0, p])
        c.ks[blk], c.vs[blk] = 0.0, 0.0
    q = torch.randn(1, 4, 64, generator=torch.Generator().manual_seed(1)).to(torch.float16)
    out = decode(c, q.cuda(), 0.3)
    check_decode(c, 4, q, out, 0.3)


def test_decode_flags_bad_blocks_and_lengths():
    pa.get_device_error()
    c = BlockCache([100, 64, 20], 2, 128, 32, seed=5)
    q = torch.randn(3, 4, 128, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    good = decode(c, q, 0.1)
    d = c.dev()
    d["tables"][1, 0] = -7
    d["lens"][2] = -1
    out = decode(c, q, 0.1)
    assert pa.get_device_error() == 2 | 4
    assert torch.equal(out[0], good[0]) and bool((out[2] == 0).all()) and bool(out.isfinite().all())


def test_decode_of_an_empty_batch_and_on_another_stream():
    c = BlockCache([70, 3], 1, 128, 32, seed=6)
    q = torch.randn(2, 4, 128, generator=torch.Generator().manual_seed(3)).to(torch.float16).cuda()
    a = decode(c, q, 0.1)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    ws, out = workspace(2, 4, c), torch.zeros_like(q)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        decode(c, q, 0.1, ws=ws, out=out, stream=st)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, out)


# ------------------------------------------------------------------ prefill
def prefill(c, q, news, scale, ws=None, out=None, stream=None, max_new=None):
    d = c.dev()
    if ws is None:
        n = pa.prefill_fp8_block_workspace_size(q.shape[1], c.H, c.D)
        ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.full_like(q, float("nan")) if out is None else out
    cu = i32([0] + list(np.cumsum(news)))
    pa.prefill_fp8_block(out, q, d["k"], d["v"], d["ks"], d["vs"], d["tables"], cu, d["lens"], c.H,
                         max_new or max(news), scale, ws, stream=stream)
    return out


def check_prefill(c, G, q, news, out, scale, every=1):
    got, qd = out.double().cpu().numpy(), q.double().cpu().numpy()
    at = 0
    for s, (n, t) in enumerate(zip(c.lens, news)):
        for g in range(c.H if t else 0):
            K, V, codes, vs = c.rows(s, g)
            for i in sorted(set(list(range(0, t, every)) + [t - 1])):
                for h in range(g * G, (g + 1) * G):
                    seen = np.arange(n) <= n - t + i
                    o, bound = row_bound(qd[at + i, h], K, V, codes, vs, seen, scale, q.dtype)
                    assert (np.abs(got[at + i, h] - o) <= bound).all(), (s, i, h)
        at += t
    assert np.isfinite(got[:at]).all()


def queries(news, heads, D, dtype, seed=3):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(sum(news), heads, D, generator=g) * 1.5).to(dtype)


PREFILLS = [
    # dtype, D, Hkv, G, bs, lens, news, spread, check every
    (torch.bfloat16, 128, 1, 4, 32, [1], [1], 3, 1),
    (torch.bfloat16, 128, 2, 4, 32, [5, 64, 33, 100], [5, 1, 3, 31], 3, 1),
    (torch.float16, 64, 1, 8, 16, [16, 17, 0, 130], [16, 16, 0, 7], 6, 1),
    (torch.bfloat16, 96, 2, 1, 64, [100, 127], [100, 128 - 1], 3, 5),
    (torch.bfloat16, 128, 1, 4, 32, [300, 129, 700], [300, 64, 33], 3, 7),
    (torch.float16, 128, 2, 3, 32, [257, 86], [257, 86], 8, 9),
    (torch.bfloat16, 96, 1, 5, 16, [400, 51], [333, 51], 3, 11),
    (torch.float16, 64, 2, 2, 64, [1000], [1000], 3, 41),
    (torch.bfloat16, 64, 1, 7, 16, [200, 1, 90], [150, 1, 90], 10, 13),
    (torch.bfloat16, 128, 1, 8, 32, [2500], [2], 3, 1),
    (torch.bfloat16, 128, 1, 1, 32, [6000], [1], 3, 1),
    (torch.bfloat16, 128, 8, 4, 32, [(37 * s) % 90 for s in range(40)],
     [min((37 * s) % 90, 1 + s % 5) for s in range(40)], 3, 1),
    (torch.float16, 64, 1, 4, 32, [128 + s for s in range(70)], [s for s in range(70)], 3, 17),
]


@pytest.mark.parametrize("dtype,D,Hkv,G,bs,lens,news,spread,every", PREFILLS)
def test_prefill_matches_the_definition(dtype, D, Hkv, G, bs, lens, news, spread, every):
    pa.get_device_error()
    c = BlockCache(lens, Hkv, D, bs, seed=D + G, spread=spread)
    q = queries(news, Hkv * G, D, dtype)
    out = prefill(c, q.cuda(), news, default_scale(D))
    assert pa.get_device_error() == 0
    check_prefill(c, G, q, news, out, default_scale(D), every)
    assert torch.equal(out, prefill(c, q.cuda(), news, default_scale(D)))  # the same bits again


def test_prefill_of_one_token_is_the_decode():
    c = BlockCache([400, 31, 64], 2, 128, 32, seed=2)
    q = queries([1, 1, 1], 8, 128, torch.float16)
    a, b = prefill(c, q.cuda(), [1, 1, 1], 0.1), decode(c, q.cuda(), 0.1)
    check_prefill(c, 4, q, [1, 1, 1], a, 0.1)
    check_decode(c, 4, q, b, 0.1)


@pytest.mark.parametrize("D,Hkv,G,bs", [(128, 2, 4, 32), (64, 1, 8, 16), (96, 3, 1, 64)])
def test_a_lone_token_answers_its_value_exactly(D, Hkv, G, bs):
    """With one weight the mean is V whatever the weight is: f16 holds a code times a power
    of two (2^-6 to 2^-9 here) as it is, so its rounding may not show."""
    c = BlockCache([1, 1], Hkv, D, bs, seed=4, spread=3)
    q = queries([1, 1], Hkv * G, D, torch.float16)
    for out in (decode(c, q.cuda(), 0.3), prefill(c, q.cuda(), [1, 1], 0.3)):
        for s in range(2):
            for g in range(Hkv):
                v = torch.from_numpy(c.rows(s, g)[1][0])
                assert (out[s, g * G:(g + 1) * G].double().cpu() == v).all(), (s, g)


@pytest.mark.parametrize("scale", [-0.2, 0.0, 3.0])
@pytest.mark.parametrize("news", [[20], [150]])
def test_prefill_with_other_scales(scale, news):
    c = BlockCache([150], 1, 64, 32, seed=12)
    q = queries(news, 4, 64, torch.bfloat16)
    check_prefill(c, 4, q, news, prefill(c, q.cuda(), news, scale), scale, 7)


@pytest.mark.parametrize("base", [-58, -30, 20, 50])
@pytest.mark.parametrize("news", [[20, 40], [180, 3]])
def test_prefill_over_small_and_large_scales(base, news):
    c = BlockCache([300, 40], 2, 128, 32, seed=base % 97, spread=2, base=base)
    c.ks = torch.where(c.ks.isnan(), c.ks, torch.exp2(c.ks.log2() - base - 6))  # K as usual
    q = queries(news, 8, 128, torch.bfloat16)
    check_prefill(c, 4, q, news, prefill(c, q.cuda(), news, default_scale(128)),
                  default_scale(128), 17)


def test_prefill_with_pages_of_zeros_and_scales_that_are_no_powers():
    c = BlockCache([200], 1, 64, 16, seed=8, spread=2)
    c.ks *= 1.3
    c.vs *= 0.77
    for p in (0, 3, 7):
        blk = int(c.tables[0, p])
        c.ks[blk], c.vs[blk] = 0.0, 0.0
    for news in ([30], [200]):
        q = queries(news, 4, 64, torch.float16)
        check_prefill(c, 4, q, news, prefill(c, q.cuda(), news, 0.3), 0.3, 3)


def test_prefill_flags_what_does_not_fit():
    """Bad blocks read as zeros, bad lengths give zero rows, bad offsets leave theirs."""
    pa.get_device_error()
    c = BlockCache([100, 64, 200, 50], 2, 128, 32, seed=5)
    news = [40, 64, 50, 50]
    q = queries(news, 4, 128, torch.bfloat16).cuda()
    good = prefill(c, q, news, 0.1)
    assert pa.get_device_error() == 0
    d = c.dev()
    bad = int(c.tables[0, 1])
    d["tables"][0, 1] = 10 ** 7
    d["lens"][1] = 63  # fewer than its new tokens
    out = prefill(c, q, news, 0.1)
    assert pa.get_device_error() == 2 | 4
    assert torch.equal(out[104:], good[104:]) and bool((out[40:104] == 0).all())
    c.k[bad], c.v[bad] = 0, 0
    c.ks[bad], c.vs[bad] = 1.0, 1.0
    check_prefill(c, 2, q.cpu()[:40], [40], out[:40], 0.1, 3)
    c2 = BlockCache([100, 64, 200, 50], 2, 128, 32, seed=5)
    out = prefill(c2, q, news, 0.1, max_new=63)
    assert pa.get_device_error() == 16
    assert bool(out[40:104].isnan().all()) and torch.equal(out[:40], good[:40])
    assert torch.equal(out[104:], good[104:])


def test_prefill_captured_and_replayed_on_another_stream():
    c = BlockCache([170, 33], 2, 128, 32, seed=6)
    news = [170, 20]
    q = queries(news, 8, 128, torch.float16).cuda()
    a = prefill(c, q, news, 0.1)
    st = torch.cuda.Stream()
    ws = torch.zeros(pa.prefill_fp8_block_workspace_size(8, 2, 128), dtype=torch.uint8, device="cuda")
    out, cu, d = torch.zeros_like(q), i32([0, 170, 190]), c.dev()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        pa.prefill_fp8_block(out, q, d["k"], d["v"], d["ks"], d["vs"], d["tables"], cu, d["lens"], 2,
                             170, 0.1, ws, stream=st)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, out)


# ------------------------------------------------------------------ together
def test_projection_to_attention_step_by_step():
    """norm_rope, append, prefill and decode as a model's layer calls them, against the definition
    over the codes that are in the cache; and those codes against the rows that were written."""
    pa.get_device_error()
    H, G, D, bs, S = 2, 4, 128, 32, 3
    pool = Pool(S, 90, H, D, bs, 40)
    inv = 10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))
    turns = pa.rope_turns(inv, "cuda")
    g = torch.Generator().manual_seed(41)
    w = (1 + 0.2 * torch.randn(D, generator=g)).cuda()
    rows = [[] for _ in range(S)]
    for news in ([30, 1, 64], [1, 1, 1], [1, 1, 1], [5, 0, 1], [1, 1, 1]):
        T = sum(news)
        qkv = torch.randn(T, (H * G + 2 * H) * D, generator=g).to(torch.bfloat16).cuda()
        q = qkv[:, : H * G * D].view(T, H * G, D)
        k = qkv[:, H * G * D: (H * G + H) * D].view(T, H, D)
        v = qkv[:, (H * G + H) * D:].view(T, H, D)
        pos = torch.cat([torch.arange(n, n + a) for n, a in zip(pool.lens, news)]).int().cuda()
        pa.norm_rope(q, k, q, k, turns, pos, w, w)
        pool.step(news, k.cpu(), v.cpu())
        at = 0
        for s, a in enumerate(news):
            rows[s].append(k[at: at + a].cpu())
            at += a
        c = pool.c
        c.lens, c._dev = pool.lens, dict(pool.d, lens=i32(pool.lens))
        if min(news) == max(news) == 1:
            out = decode(c, q.contiguous(), default_scale(D))
            check_decode(c, G, q, out, default_scale(D))
        else:
            out = prefill(c, q.contiguous(), news, default_scale(D))
            check_prefill(c, G, q, news, out, default_scale(D), 9)
    assert pa.get_device_error() == 0
    for s in range(S):
        want = torch.cat(rows[s]).double()
        for h in range(H):
            K, _, _, _ = pool.c.rows(s, h)
            blk = pool.c.tables[s].long()[torch.arange(len(want)) // bs]
            step = pool.c.ks[blk, h].double().numpy()[:, None]
            # a code is off by half a step: 2^-4 of itself, or 2^-10 of the scale near zero (and
            # 2^-9 for what growing has lost)
            tol = np.abs(want[:, h].numpy()) * 2.0 ** -4 * 1.001 + step * 2.0 ** -9
            assert (np.abs(K - want[:, h].numpy()) <= tol).all()


def test_blocks_past_32_bit_offsets():
    """Codes beyond 4 GB of cache: append, decode and prefill as in a small one, bit for bit."""
    H, D, bs, S = 8, 128, 32, 3
    lens, news = [70, 33, 200], [70, 1, 64]
    c = BlockCache(lens, H, D, bs, seed=9)
    key, value = (x.cuda() for x in draw_rows(sum(news), H, D, torch.bfloat16, 10))
    q = queries(news, 16, D, torch.bfloat16).cuda()
    cu = i32([0, 70, 71, 135])
    small = {x: c.dev()[x].clone() for x in ("k", "v", "ks", "vs")}
    n = small["k"].shape[0]
    first = 2 ** 32 // (H * bs * D) + 5
    big = {x: torch.empty((first + n,) + t.shape[1:], dtype=t.dtype, device="cuda")
           for x, t in small.items()}
    for x, t in small.items():
        big[x][first:] = t
    results = []
    for d, off in ((small, 0), (big, first)):
        tables = torch.where(c.dev()["tables"] < 0, -1, c.dev()["tables"] + off)
        pa.append_fp8_block(key, value, d["k"], d["v"], d["ks"], d["vs"], tables, cu, i32(lens))
        assert pa.get_device_error() == 0
        c._dev = dict(d, tables=tables, lens=i32(lens))
        one = queries([1] * S, 16, D, torch.bfloat16, 4).cuda()
        results.append((decode(c, one, 0.1), prefill(c, q, news, 0.1)))
    for a, b in zip(*results):
        assert torch.equal(a, b) and bool(a.isfinite().all())
    for x, t in small.items():
        assert torch.equal(big[x][first:].view(torch.uint8), t.view(torch.uint8)), x


def test_two_streams_at_once():
    """Calls that overlap, each with its own workspace, answer as alone."""
    c = BlockCache([900, 40, 333, 2000], 2, 128, 32, seed=14)
    news = [200, 3, 64, 1]
    q = queries(news, 8, 128, torch.bfloat16).cuda()
    one = queries([1] * 4, 8, 128, torch.bfloat16, 5).cuda()
    want = prefill(c, q, news, 0.1), decode(c, one, 0.1)
    d, cu = c.dev(), i32([0, 200, 203, 267, 268])
    streams = [torch.cuda.Stream() for _ in range(4)]
    pre = [torch.full((pa.prefill_fp8_block_workspace_size(8, 2, 128),), 0xFF, dtype=torch.uint8,
                      device="cuda") for _ in range(2)]
    dec = [workspace(4, 8, c) for _ in range(2)]
    outs = [[torch.empty_like(q if i < 2 else one) for _ in range(10)] for i in range(4)]
    args = [d[x] for x in ("k", "v", "ks", "vs", "tables")]
    torch.cuda.synchronize()
    for k in range(10):
        for i, st in enumerate(streams):
            if i < 2:
                pa.prefill_fp8_block(outs[i][k], q, *args, cu, d["lens"], 2, 200, 0.1, pre[i],
                                     stream=st)
            else:
                pa.decode_fp8_block(outs[i][k], one, *args, d["lens"], 2, 0.1, dec[i - 2],
                                    stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i // 2]) for i in range(4) for o in outs[i])
