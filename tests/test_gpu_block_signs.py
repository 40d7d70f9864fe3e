"""Scales below zero in a block-scaled FP8 cache: V = code * scale with the scale's sign, in the
decode and in the prefill, and K likewise."""
import pytest
import torch

from _block_cache import F8, BlockCache
from _ref64 import default_scale
from paged_kv_cache_context_gb300 import pa
from test_gpu_fp8_block import check_decode, check_prefill, decode, prefill, queries

pytestmark = pytest.mark.gpu

SHAPES = [
    # dtype, D, Hkv, G, bs, lens, news
    (torch.bfloat16, 128, 2, 4, 32, [300, 129, 700], [300, 64, 33]),
    (torch.bfloat16, 128, 1, 1, 32, [900, 50], [700, 20]),   # 256 tokens a row tile
    (torch.float16, 64, 2, 2, 16, [433], [300]),
    (torch.bfloat16, 96, 1, 8, 64, [200, 77], [200, 30]),
    (torch.bfloat16, 96, 2, 1, 16, [300, 100], [127, 100]),  # one query tile
    (torch.float16, 128, 1, 4, 32, [5000], [20]),
    (torch.bfloat16, 64, 1, 5, 32, [2000], [1700]),
]


@pytest.mark.parametrize("dtype,D,Hkv,G,bs,lens,news", SHAPES)
def test_scales_below_zero(dtype, D, Hkv, G, bs, lens, news):
    pa.get_device_error()
    c = BlockCache(lens, Hkv, D, bs, seed=D + 2)
    g = torch.Generator().manual_seed(G)
    for x in (c.ks, c.vs):
        x.mul_(torch.where(torch.rand(x.shape, generator=g) < 0.5, -1.0, 1.0))
    signs = c.vs.sign()
    q = queries(news, Hkv * G, D, dtype)
    out = prefill(c, q.cuda(), news, default_scale(D))
    ones = queries([1] * len(lens), Hkv * G, D, dtype, 5)
    one = decode(c, ones.cuda(), default_scale(D))
    assert pa.get_device_error() == 0 and bool((signs < 0).any())
    # the definition with the signs moved from the scales to the codes (bounds want |scale|)
    c.vs = c.vs.abs()
    c.v = (c.v.view(F8).float() * signs[:, :, None, None]).to(F8).view(torch.uint8)
    check_prefill(c, G, q, news, out, default_scale(D), 13)
    check_decode(c, G, ones, one, default_scale(D))
