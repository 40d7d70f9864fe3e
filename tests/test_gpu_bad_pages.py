"""A block id outside the pool: that page holds no tokens, and the pages beside it theirs. The
decodes over 8-bit caches and their scored forms, against attention in 64 bits without the page
(bounds: tests/_ref64.py; block-scaled: tests/test_gpu_fp8_block.py)."""
import numpy as np
import pytest
import torch

import test_gpu_scored as scored
from _block_cache import BlockCache
from _ref64 import U, Cache, attend, default_scale, weight_type
from paged_kv_cache_context_gb300 import pa
from test_gpu_fp8_block import row_bound

pytestmark = pytest.mark.gpu

# short sequences, and enough long ones that a CTA takes several pages of one at a time
LENS = [64, 200, 17, 500, 16] + [2000] * 16
BAD = {0: [0], 1: [4, 7], 3: [0, 1, 6, 30], 4: [0], 12: [0, 3, 24, 60],
       16: list(range(0, 62, 2))}  # sequence: pages
LOOK = [0, 1, 2, 3, 4, 5, 12, 16]  # sequences that are compared


def seen_of(lens, bs, s):
    seen = np.ones(lens[s], bool)
    for page in BAD.get(s, []):
        seen[page * bs: (page + 1) * bs] = False
    return seen


def spoil(d):
    for s, pages in BAD.items():
        for page in pages:
            d["tables"][s, page] = 10 ** 6 if page % 2 else -3


@pytest.mark.parametrize("dtype,D,G", [(torch.bfloat16, 128, 4), (torch.float16, 96, 1),
                                       (torch.bfloat16, 64, 8)])
@pytest.mark.parametrize("bs", [16, 32])
def test_block_scaled_decode(dtype, D, G, bs):
    pa.get_device_error()
    c = BlockCache(LENS, 2, D, bs, seed=D)
    q = torch.randn(len(LENS), 2 * G, D, generator=torch.Generator().manual_seed(1)).to(dtype)
    d, scale = c.dev(), default_scale(D)
    spoil(d)
    ws = torch.zeros(pa.decode_workspace_size(len(LENS), 2 * G, 2, D, bs, c.MB), dtype=torch.uint8,
                     device="cuda")
    out = torch.full_like(q, float("nan")).cuda()
    pa.decode_fp8_block(out, q.cuda(), d["k"], d["v"], d["ks"], d["vs"], d["tables"], d["lens"], 2,
                        scale, ws)
    assert pa.get_device_error() == 2
    got, qd = out.double().cpu().numpy(), q.double().numpy()
    for s in LOOK:
        seen = seen_of(LENS, bs, s)
        for h in range(2 * G):
            o, bound = row_bound(qd[s, h], *c.rows(s, h // G), seen, scale, dtype)
            assert (np.abs(got[s, h] - o) <= bound).all(), (s, h)


@pytest.mark.parametrize("kv", ["fp8_e4m3", "int8"])
@pytest.mark.parametrize("how", ["balanced", "whole", "scored"])
@pytest.mark.parametrize("dtype,D,G,bs", [(torch.bfloat16, 128, 4, 16), (torch.float16, 96, 1, 16),
                                          (torch.bfloat16, 64, 8, 16), (torch.bfloat16, 128, 2, 32)])
def test_other_8_bit_decodes(kv, how, dtype, D, G, bs):
    pa.get_device_error()
    c = Cache(LENS, 2, D, bs, kv, dtype, seed=D)
    q, before = scored.inputs(c, G, dtype, 3)
    d, scale, S = c.dev(), default_scale(D), len(LENS)
    spoil(d)
    out, ws = torch.full_like(q, float("nan")).cuda(), None
    sc = before.cuda()
    if how == "balanced":
        ws = torch.zeros(pa.decode_workspace_size(S, 2 * G, 2, D, bs, c.MB), dtype=torch.uint8,
                         device="cuda")
    if how == "scored":
        scored.run(c, q.cuda(), sc, scale, out=out)
    elif kv == "int8":
        pa.decode_int8(out, q.cuda(), d["k"], d["v"], d["ks"], d["vs"], d["tables"], d["lens"], 2,
                       scale, workspace=ws)
    else:
        pa.decode(out, q.cuda(), d["k"], d["v"], d["tables"], d["lens"], 2, scale, 0, kv, c.k_scale,
                  c.v_scale, ws)
    assert pa.get_device_error() == 2
    got, qd = out.double().cpu().numpy(), q.double().numpy()
    new, old = sc.double().cpu().numpy(), before.double().numpy()
    for s in LOOK:
        seen, n = seen_of(LENS, bs, s), LENS[s]
        for g in range(2):
            K, V, codes = c.rows(s, g)
            want, rel = old[s, g].copy(), 0.0
            for h in range(g * G, (g + 1) * G):
                o, bound, p, r = attend(qd[s, h], K, V, codes, seen, scale, dtype,
                                        weight_type(c, dtype))
                assert (np.abs(got[s, h] - o) <= bound).all(), (s, h)
                want[:n] += p
                rel = max(rel, r)
            if how == "scored":
                tol = rel * (want - old[s, g]) + U[torch.float32] * (G + 1) * np.abs(want) + 1e-30
                assert (np.abs(new[s, g] - want) <= tol).all(), (s, g)
                assert (new[s, g][:n][~seen] == old[s, g][:n][~seen]).all()
