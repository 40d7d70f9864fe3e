"""NaN in a block-scaled FP8 cache reaches the elements of the rows that see it and nothing else:
against a call over the same cache without it, what may not change is the same bits."""
import numpy as np
import pytest
import torch

from _block_cache import BlockCache
from _ref64 import default_scale
from paged_kv_cache_context_gb300 import pa
from test_gpu_fp8_block import decode, prefill, queries

pytestmark = pytest.mark.gpu

NAN = 0x7F

SHAPES = [
    # dtype, D, Hkv, G, bs, lens, news
    (torch.bfloat16, 128, 2, 4, 32, [300, 129, 700], [300, 64, 33]),
    (torch.bfloat16, 128, 1, 1, 32, [900, 50], [700, 20]),   # 256 tokens a row tile
    (torch.float16, 64, 2, 2, 16, [433], [300]),
    (torch.bfloat16, 96, 1, 8, 64, [200, 77], [200, 30]),
    (torch.bfloat16, 96, 2, 1, 16, [300, 100], [127, 100]),  # one query tile
    (torch.float16, 128, 1, 4, 32, [5000], [20]),
    (torch.bfloat16, 64, 1, 5, 32, [2000], [1700]),
    (torch.bfloat16, 64, 8, 4, 16, [(11 * s) % 60 + 1 for s in range(200)],
     [min((11 * s) % 60 + 1, 1 + s % 31) for s in range(200)]),
    (torch.bfloat16, 128, 8, 8, 32, [(17 * s) % 150 + 1 for s in range(90)],
     [min((17 * s) % 150 + 1, 1 + (29 * s) % 90) for s in range(90)]),
]


def spots(lens, news, D, seed):
    """(sequence, position, dim) of NaN codes: anywhere, and around the chunk's ends."""
    rng = np.random.default_rng(seed)
    at = []
    for s, (n, t) in enumerate(zip(lens, news)):
        if len(lens) > 8 and s % 3:
            continue
        some = {n - 1, n - t, max(n - t - 1, 0), int(rng.integers(n)), n - t + int(rng.integers(t))}
        at += [(s, j, int(rng.integers(D))) for j in some]
    return at


def expected(lens, news, heads, D, at):
    """Where NaN has to be in kv head 0's rows, bool [T, D]."""
    bad = np.zeros((sum(news), D), bool)
    cu = np.concatenate([[0], np.cumsum(news)])
    for s, j, dim in at:
        first = max(j - (lens[s] - news[s]), 0)  # the first new token that sees position j
        bad[cu[s] + first: cu[s + 1], dim] = True
    return bad


@pytest.mark.parametrize("dtype,D,Hkv,G,bs,lens,news", SHAPES)
def test_a_nan_code_in_v_reaches_the_rows_that_see_it(dtype, D, Hkv, G, bs, lens, news):
    pa.get_device_error()
    c = BlockCache(lens, Hkv, D, bs, seed=D)
    q = queries(news, Hkv * G, D, dtype).cuda()
    clean = prefill(c, q, news, default_scale(D))
    at = spots(lens, news, D, D + G)
    for s, j, dim in at:
        c.dev()["v"][c.tables[s, j // bs].item(), 0, j % bs, dim] = NAN + (128 if j % 2 else 0)
    out = prefill(c, q, news, default_scale(D))
    assert pa.get_device_error() == 0
    bad = torch.from_numpy(expected(lens, news, Hkv * G, D, at))[:, None, :].expand(-1, G, -1).cuda()
    got = out[:, :G]
    assert bool(got[bad].isnan().all())
    assert torch.equal(got[~bad], clean[:, :G][~bad])
    assert torch.equal(out[:, G:], clean[:, G:])


@pytest.mark.parametrize("dtype,D,Hkv,G,bs,lens,news", SHAPES)
def test_a_nan_code_in_the_decode(dtype, D, Hkv, G, bs, lens, news):
    c = BlockCache(lens, Hkv, D, bs, seed=D)
    q = queries([1] * len(lens), Hkv * G, D, dtype).cuda()
    clean = decode(c, q, default_scale(D))
    at = spots(lens, news, D, D + G)
    bad = torch.zeros(len(lens), D, dtype=torch.bool)
    for s, j, dim in at:
        c.dev()["v"][c.tables[s, j // bs].item(), 0, j % bs, dim] = NAN
        bad[s, dim] = True
    out = decode(c, q, default_scale(D))
    bad = bad[:, None, :].expand(-1, G, -1).cuda()
    assert bool(out[:, :G][bad].isnan().all())
    assert torch.equal(out[:, :G][~bad], clean[:, :G][~bad])
    assert torch.equal(out[:, G:], clean[:, G:])


@pytest.mark.parametrize("dtype,D,Hkv,G,bs,lens,news", SHAPES)
def test_a_nan_scale_of_v_is_nan_for_the_rows_that_see_it(dtype, D, Hkv, G, bs, lens, news):
    pa.get_device_error()
    c = BlockCache(lens, Hkv, D, bs, seed=D + 1)
    q = queries(news, Hkv * G, D, dtype).cuda()
    clean = prefill(c, q, news, default_scale(D))
    rng = np.random.default_rng(G)
    pages = [(s, int(rng.integers(-(-n // bs)))) for s, n in enumerate(lens) if s % 3 == 0]
    at = [(s, page * bs, dim) for s, page in pages for dim in range(D)]
    for s, page in pages:
        c.dev()["vs"][c.tables[s, page].item(), 0] = float("nan")
    out = prefill(c, q, news, default_scale(D))
    assert pa.get_device_error() == 0
    bad = torch.from_numpy(expected(lens, news, Hkv * G, D, at))[:, None, :].expand(-1, G, -1).cuda()
    assert bool(out[:, :G][bad].isnan().all())
    # (a row's reference depends on its pages' V scales, NaN among them: rounding may differ)
    assert bool(out[:, :G][~bad].isfinite().all()) and torch.equal(out[:, G:], clean[:, G:])
    ones = queries([1] * len(lens), Hkv * G, D, dtype, 5).cuda()
    one = decode(c, ones, default_scale(D))
    for s in range(len(lens)):
        hit = any(s == t for t, _ in pages)
        assert bool(one[s, :G].isnan().all()) == hit and bool(one[s, G:].isfinite().all())


def test_a_nan_that_comes_and_goes_between_replays():
    """What a launch keeps of NaN is its own: one captured call, replayed over a clean cache, one
    with NaN and the clean one again, with one workspace throughout."""
    lens, news, Hkv, G, D, bs = [300, 129], [300, 64], 2, 4, 128, 32
    c = BlockCache(lens, Hkv, D, bs, seed=31)
    q = queries(news, Hkv * G, D, torch.float16).cuda()
    clean = prefill(c, q, news, 0.1)
    d = c.dev()
    ws = torch.full((pa.prefill_fp8_block_workspace_size(Hkv * G, Hkv, D),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    out = torch.zeros_like(q)
    cu = torch.tensor([0, 300, 364], dtype=torch.int32, device="cuda")
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        pa.prefill_fp8_block(out, q, d["k"], d["v"], d["ks"], d["vs"], d["tables"], cu, d["lens"],
                             Hkv, 300, 0.1, ws, stream=st)
    spot = (c.tables[0, 5].item(), 1, 17, 100)  # position 177, kv head 1
    was = d["v"][spot].item()
    for i in range(30):
        bad = i % 3 == 1
        d["v"][spot] = NAN if bad else was
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        hit = torch.zeros_like(out, dtype=torch.bool)
        if bad:
            hit[177:300, G:, 100] = True
        assert bool(out[hit].isnan().all()) and torch.equal(out[~hit], clean[~hit]), i
    assert pa.get_device_error() == 0
