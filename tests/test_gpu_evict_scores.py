"""pa_compact's scores beside bad blocks, and the scores of a serving loop token by token."""
import numpy as np
import pytest
import torch

from _gpu import bits
from _ref64 import U, Cache, attend, default_scale, weight_type
from paged_kv_cache_context_gb300 import pa
from test_gpu_evict import ascending, compact, moved
from test_gpu_scored import run as run_scored

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv,dtype,bs", [("auto", torch.bfloat16, 32), ("int8", torch.bfloat16, 32),
                                         ("auto", torch.float32, 24)])
@pytest.mark.parametrize("page", [0, 1])  # of destinations, and of sources alone
@pytest.mark.parametrize("bad", [999, -1])
def test_a_row_of_a_bad_block_keeps_its_score_too(kv, dtype, bs, page, bad):
    """K, V, row scales and score of an entry move together or not at all."""
    cache = Cache([70, 70, 70], 2, 64, bs, kv, dtype, seed=8)
    kept = [20, 20, 20]
    keep = ascending(cache.lens, 2, 20, kept, None, 3)
    scores = torch.rand(3, 2, cache.MB * bs)
    d = cache.dev()
    skip = set()
    # an entry is skipped in both heads: make them choose alike in sequence 1
    keep[1, 1] = keep[1, 0]
    for j in range(20):
        f = int(keep[1, 0, j])
        if f != j and page in (f // bs, j // bs):
            skip.add((1, j))
    assert skip and len(skip) < 20 or page == 0
    want, want_s = moved(cache, keep, kept, None, scores, skip=skip)
    d["tables"][1, page] = bad
    pa.get_device_error()
    got, got_s = compact(cache, keep, kept, None, scores)
    assert pa.get_device_error() == 2
    d["tables"].copy_(cache.tables)
    for x in want:
        assert torch.equal(bits(got[x]), bits(want[x])), x
    assert torch.equal(got_s.cpu(), want_s)


@pytest.mark.parametrize("kv", ["auto", "int8", "fp8_e4m3"])
def test_scores_of_several_steps_token_by_token(kv):
    """Each step adds each token's own weight: a weight's relative error (see _ref64.py) and one
    rounding of a step's sum per head and of each addition."""
    H, G, D, bs, steps = 2, 4, 128, 32, 5
    cache = Cache([100, 40, 61, 1300], H, D, bs, kv, torch.bfloat16, seed=12)
    S, N = 4, cache.MB * bs
    g = torch.Generator().manual_seed(4)
    scores = torch.zeros(S, H, N, device="cuda")
    want, lim = np.zeros((S, H, N)), np.zeros((S, H, N))
    pa.get_device_error()
    for _ in range(steps):
        q = torch.randn(S, H * G, D, generator=g).bfloat16()
        run_scored(cache, q.cuda(), scores, default_scale(D))
        for s, n in enumerate(cache.lens):
            for h in range(H * G):
                K, V, codes = cache.rows(s, h // G)
                _, _, p, rel = attend(q[s, h].double().numpy(), K, V, codes, np.ones(n, bool),
                                      default_scale(D), torch.bfloat16,
                                      weight_type(cache, torch.bfloat16))
                want[s, h // G, :n] += p
                lim[s, h // G, :n] += rel * p
        lim += U[torch.float32] * (G + 1) * want
    assert pa.get_device_error() == 0
    err = np.abs(scores.cpu().double().numpy() - want)
    assert (err <= lim + 1e-30).all(), float((err / (lim + 1e-30)).max())
    # a missing step would show at every token of every sequence
    for s, n in enumerate(cache.lens):
        assert (lim[s, :, :n] < want[s, :, :n] / steps / 4).all()
