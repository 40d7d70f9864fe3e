"""pa_decode_scored on the GPU against attention in 64 bits over the same cache bytes.

The output's bounds: tests/_ref64.py (a 32-bit cache: no weight is rounded, u(f32)). A score is
old + sum_h p_h: the weights' relative error and one rounding of the sum per head and of the
addition, u(f32) (G + 1) (old + sum_h p_h)."""
import numpy as np
import pytest
import torch

from _ref64 import U, Cache, attend, default_scale, weight_type
from paged_kv_cache_context_gb300 import pa

pytestmark = pytest.mark.gpu


def workspace(S, Hq, cache):
    n = pa.decode_scored_workspace_size(S, Hq, cache.H, cache.D, cache.bs, cache.MB)
    return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")


def run(cache, q, scores, scale, ws=None, out=None, stream=None):
    d = cache.dev()
    ws = workspace(q.shape[0], q.shape[1], cache) if ws is None else ws
    out = torch.full_like(q, float("nan")) if out is None else out
    if cache.kv == "int8":
        pa.decode_scored_int8(out, scores, q, d["k"], d["v"], d["ks"], d["vs"], d["tables"],
                              d["lens"], cache.H, scale, ws, stream=stream)
    else:
        pa.decode_scored(out, scores, q, d["k"], d["v"], d["tables"], d["lens"], cache.H, scale,
                         ws, cache.kv, cache.k_scale, cache.v_scale, stream=stream)
    return out


def inputs(cache, G, dtype, seed, qmul=1.5):
    g = torch.Generator().manual_seed(seed)
    S, N = len(cache.lens), cache.MB * cache.bs
    q = (torch.randn(S, cache.H * G, cache.D, generator=g) * qmul).to(dtype)
    scores = torch.rand(S, cache.H, N, generator=g)  # past the length too: has to stay
    return q, scores


def check(cache, G, q, before, out, scores, scale):
    got, sc = out.double().cpu().numpy(), scores.double().cpu().numpy()
    old, qd = before.double().numpy(), q.double().cpu().numpy()
    for s, n in enumerate(cache.lens):
        for g in range(cache.H):
            K, V, codes = cache.rows(s, g)
            want = old[s, g].copy()
            rel = 0.0
            for h in range(g * G, (g + 1) * G):
                o, bound, p, r = attend(qd[s, h], K, V, codes, np.ones(n, bool), scale, q.dtype,
                                        weight_type(cache, q.dtype))
                assert (np.abs(got[s, h] - o) <= bound).all(), (s, h)
                want[:n] += p
                rel = max(rel, r)
            err = np.abs(sc[s, g] - want)
            bound = rel * (want - old[s, g]) + U[torch.float32] * (G + 1) * np.abs(want)
            assert (err[:n] <= bound[:n] + 1e-30).all(), (s, g, float((err / (bound + 1e-30))[:n].max()))
            assert (err[n:] == 0).all()


CASES = [
    # kv, dtype, D, Hkv, G, bs, lens
    ("auto", torch.float32, 64, 4, 1, 32, [17, 45]),
    ("auto", torch.float32, 96, 2, 3, 16, [1, 0, 16, 33, 200]),
    ("auto", torch.float32, 128, 1, 8, 64, [65, 700]),
    ("auto", torch.bfloat16, 128, 2, 4, 32, [1, 31, 32, 33, 0, 500]),
    ("auto", torch.bfloat16, 96, 2, 4, 16, [100, 7]),
    ("auto", torch.float16, 64, 1, 8, 64, [1000, 3]),
    ("auto", torch.bfloat16, 128, 8, 1, 32, [64, 90]),
    ("auto", torch.bfloat16, 64, 1, 5, 16, [(13 * s) % 70 for s in range(40)]),
    ("auto", torch.bfloat16, 128, 1, 4, 32, [9000]),
    ("fp8_e4m3", torch.bfloat16, 96, 4, 1, 32, [1, 100, 333]),
    ("fp8_e4m3", torch.float16, 128, 1, 7, 16, [17, 400]),
    ("fp8_e4m3", torch.float32, 64, 2, 2, 32, [50, 129]),
    ("int8", torch.bfloat16, 128, 2, 4, 32, [33, 300, 5]),
    ("int8", torch.float16, 96, 2, 3, 64, [128, 1]),
    ("int8", torch.bfloat16, 64, 1, 8, 16, [2000]),
]


@pytest.mark.parametrize("kv,dtype,D,Hkv,G,bs,lens", CASES)
def test_matches_the_definition(kv, dtype, D, Hkv, G, bs, lens):
    pa.get_device_error()
    cache = Cache(lens, Hkv, D, bs, kv, dtype, seed=D + G)
    q, before = inputs(cache, G, dtype, 3)
    scores = before.cuda()
    out = run(cache, q.cuda(), scores, default_scale(D))
    assert pa.get_device_error() == 0
    check(cache, G, q, before, out, scores, default_scale(D))


@pytest.mark.parametrize("kv,dtype,D,G,bs", [
    ("auto", torch.bfloat16, 128, 4, 32), ("auto", torch.float32, 64, 1, 16),
    ("fp8_e4m3", torch.float16, 96, 1, 32), ("int8", torch.bfloat16, 128, 2, 16)])
def test_shares_of_many_pages(kv, dtype, D, G, bs):
    """More sequences than a warp has lanes and more pages than CTAs: shares that hold whole
    segments, begin and end inside one, and skip empty sequences."""
    pa.get_device_error()
    lens = [(379 * s) % 1021 if s % 5 else 0 for s in range(70)] + [2500]
    cache = Cache(lens, 3, D, bs, kv, dtype, seed=D + G)
    q, before = inputs(cache, G, dtype, 5)
    scores = before.cuda()
    out = run(cache, q.cuda(), scores, default_scale(D))
    assert pa.get_device_error() == 0
    check(cache, G, q, before, out, scores, default_scale(D))
    for _ in range(20):
        again = before.cuda()
        assert torch.equal(run(cache, q.cuda(), again, default_scale(D)), out)
        assert torch.equal(again, scores)


@pytest.mark.parametrize("scale,qmul", [(-0.2, 1.0), (0.0, 1.0), (1.0, 10.0)])
def test_other_scales_and_large_logits(scale, qmul):
    cache = Cache([200, 77], 2, 128, 32, seed=9)
    q, before = inputs(cache, 4, torch.bfloat16, 4, qmul)
    scores = before.cuda()
    out = run(cache, q.cuda(), scores, scale)
    check(cache, 4, q, before, out, scores, scale)


def test_bad_blocks_and_lengths_are_flagged():
    cache = Cache([100, 90, 64], 2, 128, 32, seed=4)
    q, before = inputs(cache, 4, torch.bfloat16, 2)
    d = cache.dev()
    pa.get_device_error()
    keep = d["tables"].clone()
    d["tables"][0, 1] = 10 ** 6
    scores = before.cuda()
    out = run(cache, q.cuda(), scores, 0.1)
    assert pa.get_device_error() == 2 and out.isfinite().all() and scores.isfinite().all()
    assert torch.equal(scores[0, :, 32:64].cpu(), before[0, :, 32:64])  # its tokens add nothing
    # every other token's weight is counted: each head's sum to one
    added = (scores.cpu().double() - before.double())[0].sum(-1)
    assert (added - 4).abs().max() <= 4 * 100 * 2.0 ** -23 + 100 * 2.0 ** -24
    d["tables"].copy_(keep)
    lens = d["lens"].clone()
    d["lens"][1] = -3
    scores = before.cuda()
    out = run(cache, q.cuda(), scores, 0.1)
    assert pa.get_device_error() == 4
    assert (out[1] == 0).all() and torch.equal(scores[1].cpu(), before[1])
    d["lens"].copy_(lens)


def test_shared_blocks_keep_scores_apart():
    cache = Cache([64, 64], 1, 64, 32, seed=3)
    cache.tables[1] = cache.tables[0]
    q, before = inputs(cache, 2, torch.bfloat16, 6)
    scores = before.cuda()
    out = run(cache, q.cuda(), scores, 0.125)
    check(cache, 2, q, before, out, scores, 0.125)


def test_same_bits_again_in_a_graph_and_on_two_streams():
    cache = Cache([700, 1500, 90], 2, 128, 32, seed=6)
    q, before = inputs(cache, 4, torch.bfloat16, 8)
    q = q.cuda()
    want_s = before.cuda()
    want = run(cache, q, want_s, 0.1)
    st = [torch.cuda.Stream() for _ in range(2)]
    ws = [workspace(3, 8, cache) for _ in range(2)]
    sc = [before.cuda() for _ in range(2)]
    outs = [torch.empty_like(q) for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(2):
        run(cache, q, sc[i], 0.1, ws[i], outs[i], st[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(outs[i], want) and torch.equal(sc[i], want_s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(cache, q, sc[0], 0.1, ws[0], outs[0])
    sc[0].copy_(before)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(sc[0], want_s)
