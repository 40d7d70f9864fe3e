"""Scored decodes over INT8 rows of any size and beside a dominant token: bounds and inputs of
test_gpu_small_weights.py, and scores within their weights' relative error."""
import numpy as np
import pytest
import torch

from _ref64 import U, Cache, default_scale
from paged_kv_cache_context_gb300 import pa
from test_gpu_scored import run as run_scored
from test_gpu_small_weights import add_sink, attend_sharp, scale_rows, signs

pytestmark = pytest.mark.gpu


def check_scored(cache, G, q, before, out, scores):
    got, sc, qd = out.double().cpu().numpy(), scores.double().cpu().numpy(), q.double().cpu().numpy()
    for s, n in enumerate(cache.lens):
        for g in range(cache.H):
            want, r = before[s, g].double().numpy().copy(), 0.0
            for h in range(g * G, (g + 1) * G):
                o, bound, p, rel = attend_sharp(cache, s, g, qd[s, h], np.ones(n, bool), q.dtype)
                err = np.abs(got[s, h] - o)
                assert (err <= bound).all(), (s, h, float((err / bound).max()))
                want[:n] += p
                r = max(r, rel)
            err = np.abs(sc[s, g] - want)[:n]
            lim = r * (want - before[s, g].double().numpy()) + U[torch.float32] * (G + 1) * want
            assert (err <= lim[:n] + 1e-30).all(), (s, g)


SCORED = [  # dtype, D, Hkv, G, bs, lens
    (torch.bfloat16, 128, 2, 4, 32, [1500, 33, 1]),
    (torch.float16, 64, 1, 8, 16, [2100, 70]),
    (torch.bfloat16, 96, 2, 1, 64, [1000, 40]),
]


@pytest.mark.parametrize("how", [1e7, 0.06, 1e-4, "mixed", "growing", "falling"])
@pytest.mark.parametrize("dtype,D,H,G,bs,lens", SCORED)
def test_scored_over_int8_rows_of_any_size(dtype, D, H, G, bs, lens, how):
    if how == 1e7:
        dtype = torch.bfloat16
    pa.get_device_error()
    cache = Cache(lens, H, D, bs, "int8", dtype, seed=D)
    scale_rows(cache, how)
    g = torch.Generator().manual_seed(3)
    q = (1.5 * torch.randn(len(lens), H * G, D, generator=g)).to(dtype)
    before = torch.rand(len(lens), H, cache.MB * bs, generator=g)
    scores = before.cuda()
    out = run_scored(cache, q.cuda(), scores, default_scale(D))
    assert pa.get_device_error() == 0
    check_scored(cache, G, q, before, out, scores)


@pytest.mark.parametrize("kv", ["auto", "fp8_e4m3", "int8"])
@pytest.mark.parametrize("dtype,D,H,G,bs,lens", SCORED)
def test_scored_keeps_small_weights_beside_a_dominant_one(dtype, D, H, G, bs, lens, kv):
    pa.get_device_error()
    cache = Cache([2 * lens[0]] + lens[1:], H, D, bs, kv, dtype, seed=D)
    add_sink(cache, signs(D), 15.0)
    g = torch.Generator().manual_seed(3)
    q = (1.5 * signs(D) + 0.1 * torch.randn(len(lens), H * G, D, generator=g)).to(dtype)
    before = torch.rand(len(lens), H, cache.MB * bs, generator=g)
    scores = before.cuda()
    out = run_scored(cache, q.cuda(), scores, default_scale(D))
    assert pa.get_device_error() == 0
    check_scored(cache, G, q, before, out, scores)


@pytest.mark.parametrize("how", ["growing", "falling"])
@pytest.mark.parametrize("dtype,D,G,bs", [(torch.bfloat16, 128, 2, 16), (torch.float16, 64, 1, 32)])
def test_scored_shares_of_many_pages_whose_scales_differ(dtype, D, G, bs, how):
    """A share is several pages long: its reference moves with the scales inside it."""
    pa.get_device_error()
    lens = [(379 * s) % 1021 if s % 5 else 0 for s in range(70)] + [2500]
    cache = Cache(lens, 3, D, bs, "int8", dtype, seed=D + G)
    scale_rows(cache, how)
    g = torch.Generator().manual_seed(3)
    q = (1.5 * torch.randn(len(lens), 3 * G, D, generator=g)).to(dtype)
    before = torch.rand(len(lens), 3, cache.MB * bs, generator=g)
    scores = before.cuda()
    out = run_scored(cache, q.cuda(), scores, default_scale(D))
    assert pa.get_device_error() == 0
    check_scored(cache, G, q, before, out, scores)
