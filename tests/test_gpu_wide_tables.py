"""Eviction's choice and scored decodes over tables wider than their sequences, and the variants
that long rows and large batches take: a choice that reads its scores from memory in every pass
(more than 53,248 positions a row), and score updates of four rounds of tokens a CTA (608 CTAs or
more of them). Definitions and bounds as in test_gpu_evict.py and test_gpu_scored.py."""
import numpy as np
import pytest
import torch

from _gpu import bits
from _ref64 import Cache, attend, default_scale, weight_type
from paged_kv_cache_context_gb300 import pa
from test_gpu_evict import check_select, choose, compact, moved, select
from test_gpu_scored import check, inputs, run

pytestmark = pytest.mark.gpu

EDGE = 53248  # the longest row whose keys are kept on chip


@pytest.mark.parametrize("N,lens,B,sink,recent", [
    (EDGE, [EDGE, 60], 700, 4, 64),
    (EDGE + 1, [EDGE + 1, 60], 700, 4, 64),       # the first that is not; rows off 16 bytes
    (EDGE + 2, [EDGE + 2, EDGE], 30000, 0, 0),
    (65538, [65537, 1, 0], 2048, 4, 512),
    (131072, [131072, 131069], 4096, 4, 512),
    (131072, [700, 33, 4097, 32769], 64, 4, 8),   # short sequences in a wide table
    (131072, [100000], 99999, 1, 1),
])
def test_select_reads_long_rows_from_memory(N, lens, B, sink, recent):
    pa.get_device_error()
    g = torch.Generator().manual_seed(N + B)
    scores = torch.exp(2 * torch.randn(len(lens), 2, N, generator=g) - 4)
    check_select(scores, lens, B, sink, recent)
    assert pa.get_device_error() == 0


def test_select_of_long_rows_with_ties_signs_infinities_and_nan():
    """Equal scores over several rounds of a row, and a search that ends at a whole bin."""
    N = 70001
    g = torch.Generator().manual_seed(2)
    few = torch.randint(-1, 3, (1, 4, N), generator=g).float()
    few[0, 1] = 2.0
    few[0, 2, ::3] = float("nan")
    few[0, 2, 1::5] = float("inf")
    few[0, 2, 2::7] = float("-inf")
    few[0, 3] = torch.where(torch.arange(N) % 2 == 0, 1.0, 2.0 ** -30)  # 35,001 in one bin
    for B, sink, recent in ((20000, 4, 100), (69000, 0, 0), (17, 1, 0), (35001, 0, 0)):
        check_select(few, [N], B, sink, recent)


@pytest.mark.parametrize("N", [4096, 30000, 131072])
def test_select_in_a_wide_table_is_that_of_a_tight_one(N):
    g = torch.Generator().manual_seed(4)
    tight = torch.rand(3, 2, 900, generator=g)
    wide = torch.full((3, 2, N), float("nan"))
    wide[..., :900] = tight
    lens = [900, 64, 257]
    a, b = select(tight, lens, 100, 4, 16), select(wide, lens, 100, 4, 16)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


LENS = [13000, 700, 1024, 1025, 1500, 2600, 3500, 4096, 4097, 5000, 0, 1, 33, 2048, 9000, 64, 4095,
        2049, 8192, 300]  # 20 sequences and 8 kv heads, four CTAs a row: 640


@pytest.mark.parametrize("kv,dtype,D,G,bs", [
    ("auto", torch.bfloat16, 64, 1, 32), ("auto", torch.bfloat16, 64, 4, 16),
    ("auto", torch.float32, 64, 2, 64), ("fp8_e4m3", torch.float16, 96, 3, 32),
    ("int8", torch.bfloat16, 64, 8, 32)])
def test_scores_of_four_rounds_a_cta(kv, dtype, D, G, bs):
    pa.get_device_error()
    cache = Cache(LENS, 8, D, bs, kv, dtype, seed=D + G)
    assert 8 * len(LENS) * -(-cache.MB * bs // 4096) >= 608
    q, before = inputs(cache, G, dtype, 3)
    scores = before.cuda()
    out = run(cache, q.cuda(), scores, default_scale(D))
    assert pa.get_device_error() == 0
    check(cache, G, q, before, out, scores, default_scale(D))
    again = before.cuda()
    assert torch.equal(run(cache, q.cuda(), again, default_scale(D)), out)
    assert torch.equal(again, scores)


@pytest.mark.parametrize("page", [5, 40, 70, 100, 200])  # in each of a CTA's rounds, and in a later CTA
def test_bad_block_in_a_later_round_adds_nothing(page):
    cache = Cache(LENS, 8, 64, 32, "auto", torch.bfloat16, seed=1)
    q, before = inputs(cache, 2, torch.bfloat16, 3)
    d = cache.dev()
    pa.get_device_error()
    d["tables"][0, page] = -1
    scores = before.cuda()
    out = run(cache, q.cuda(), scores, 0.1)
    assert pa.get_device_error() == 2 and out.isfinite().all() and scores.isfinite().all()
    d["tables"].copy_(cache.tables)
    a, b = 32 * page, 32 * page + 32
    assert torch.equal(scores[0, :, a:b].cpu(), before[0, :, a:b])
    # every other token's weight is counted: each head's sum to one
    n = LENS[0]
    added = (scores.cpu().double() - before.double())[0].sum(-1)
    assert (added - 2).abs().max() <= 2 * (n + 16) * 2.0 ** -23 + n * 2.0 ** -24


@pytest.mark.parametrize("kv,dtype", [("auto", torch.bfloat16), ("int8", torch.bfloat16)])
def test_scored_decode_in_a_wide_table_is_that_of_a_tight_one(kv, dtype):
    """Pages past the longest sequence change nothing, and their scores stay."""
    cache = Cache([700, 33, 1500, 0], 8, 64, 32, kv, dtype, seed=8)
    q, before = inputs(cache, 2, dtype, 5)
    a = before.cuda()
    want = run(cache, q.cuda(), a, 0.125)
    d = cache.dev()
    MB, wide = cache.MB, 2560  # 81,920 positions: 20 CTAs of four rounds a row
    d["tables"] = torch.nn.functional.pad(d["tables"], (0, wide - MB), value=-1).contiguous()
    cache.MB = wide
    b = torch.full((4, 8, wide * 32), 5.0, device="cuda")
    b[..., : MB * 32] = before.cuda()
    out = run(cache, q.cuda(), b, 0.125)
    assert torch.equal(out, want) and torch.equal(b[..., : MB * 32], a)
    assert b[..., MB * 32:].eq(5.0).all()
