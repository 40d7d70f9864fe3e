"""Precision of the block-scaled decode beside pages of far larger or smaller V scales.

The decode rounds products of weight and V scale to f16, in units in which the row's largest
product is 2^6 at least, so that one is off by 2^-11 of itself or by half of f16's smallest step,
2^-25, which is 2^-31 of the row's largest product, for each unit of |code|. With p the exact weights
and A = sum_j p_j |V_j| the output is then off by
  (2^-11 + rel) A + 2^-31 max_j (p_j vs_j) sum_j |code_j| + u(out) |o|
(rel: a weight's relative error, tests/_ref64.py); for f16 outputs the sum takes the rounded
weights, whose own 2^-11 moves the mean by 2^-11 |o| more."""
import math

import numpy as np
import pytest
import torch

from _block_cache import F8, BlockCache
from _ref64 import U, attend
from paged_kv_cache_context_gb300 import pa

pytestmark = pytest.mark.gpu


def bound_of(q, K, V, codes, vs, scale, dtype):
    seen = np.ones(len(K), bool)
    o, bound, p, _ = attend(q, K, V, np.zeros_like(codes), seen, scale, dtype, torch.float32)
    bound = bound + 1.01 * 2.0 ** -11 * (p @ np.abs(V) + (np.abs(o) if dtype == torch.float16 else 0))
    return o, bound + 2.0 ** -31 * (p * vs).max() * np.abs(codes).sum(0)


@pytest.mark.parametrize("dtype,D,G,bs,lens", [
    (torch.bfloat16, 128, 4, 16, [64, 33, 500]), (torch.bfloat16, 64, 8, 16, [64, 100]),
    (torch.float16, 96, 1, 16, [96, 250]), (torch.bfloat16, 128, 1, 32, [128, 300]),
    (torch.float16, 64, 2, 64, [256])])
@pytest.mark.parametrize("gap", [24, 34, 50])
@pytest.mark.parametrize("heavy", [0, 1])
def test_the_largest_product_keeps_its_precision(dtype, D, G, bs, lens, gap, heavy):
    """Every other page has logits about 2^(gap + 6) times its neighbours' weights and V scales
    of 2^-gap beside their 1: its products are the largest."""
    pa.get_device_error()
    c = BlockCache(lens, 2, D, bs, seed=gap + D)
    g = torch.Generator().manual_seed(gap)
    c.k = (1 + 0.25 * torch.rand(c.k.shape, generator=g)).to(F8).view(torch.uint8)  # 1 to 1.25
    for s, n in enumerate(lens):
        for page in range(-(-n // bs)):
            blk = int(c.tables[s, page])
            strong = page % 2 == heavy
            c.ks[blk] = (gap + 6) * math.log(2.0) if strong else 0.01
            c.vs[blk] = 2.0 ** -gap if strong else 1.0
    q = torch.ones(len(lens), 2 * G, D).to(dtype)
    scale = 1.0 / (1.125 * D)  # a code is 1.125 on average
    d = c.dev()
    ws = torch.full((pa.decode_workspace_size(len(lens), 2 * G, 2, D, bs, c.MB),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    out = torch.full_like(q, float("nan")).cuda()
    pa.decode_fp8_block(out, q.cuda(), d["k"], d["v"], d["ks"], d["vs"], d["tables"], d["lens"], 2,
                        scale, ws)
    assert pa.get_device_error() == 0
    got, qd = out.double().cpu().numpy(), q.double().numpy()
    for s in range(len(lens)):
        for h in range(2 * G):
            K, V, codes, vs = c.rows(s, h // G)
            o, bound = bound_of(qd[s, h], K, V, codes, vs, scale, dtype)
            # (f16's own smallest step for outputs of tiny V scales)
            bound = bound + (2.0 ** -25 if dtype == torch.float16 else 0.0)
            err = np.abs(got[s, h] - o)
            assert (err <= bound).all(), (s, h, float((err / bound).max()))
