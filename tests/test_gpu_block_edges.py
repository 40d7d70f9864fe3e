"""Calls over the block-scaled FP8 cache that are allowed and rare: no sequences or tokens, an output
off a 32-byte boundary, row tiles of 256 tokens over an unaligned prefix, wide block tables."""
import pytest
import torch

from _block_cache import BlockCache
from _ref64 import default_scale
from paged_kv_cache_context_gb300 import pa
from test_gpu_fp8_block import check_decode, check_prefill, decode, i32, prefill, queries

pytestmark = pytest.mark.gpu


def test_no_sequences_and_no_tokens():
    pa.get_device_error()
    c = BlockCache([40], 2, 128, 32, seed=1)
    d = c.dev()
    args = [d[x] for x in ("k", "v", "ks", "vs")]
    before = [x.clone() for x in args]
    none, lens = d["tables"][:0], d["lens"][:0]
    rows, heads = (torch.zeros(0, h, 128, dtype=torch.bfloat16, device="cuda") for h in (2, 8))
    some = torch.ones(3, 8, 128, dtype=torch.bfloat16, device="cuda")
    out = some.clone()
    ws = torch.zeros(pa.decode_workspace_size(1, 8, 2, 128, 32, c.MB) +
                     pa.prefill_fp8_block_workspace_size(8, 2, 128), dtype=torch.uint8, device="cuda")
    pa.append_fp8_block(rows, rows, *args, none, i32([0]), lens)                   # no sequences
    pa.append_fp8_block(rows, rows, *args, d["tables"], i32([0, 0]), d["lens"])    # no new tokens
    pa.append_fp8_block(some[:, :2], some[:, :2], *args, none, i32([0]), lens)     # nobody's tokens
    pa.decode_fp8_block(heads, heads, *args, none, lens, 2, 0.1, ws)
    pa.prefill_fp8_block(heads, heads, *args, none, i32([0]), lens, 2, 1, 0.1, ws)
    pa.prefill_fp8_block(heads, heads, *args, d["tables"], i32([0, 0]), d["lens"], 2, 1, 0.1, ws)
    pa.prefill_fp8_block(out, some, *args, none, i32([0]), lens, 2, 1, 0.1, ws)
    pa.prefill_fp8_block(out, some, *args, d["tables"], i32([1, 1]), d["lens"], 2, 3, 0.1, ws)
    assert pa.get_device_error() == 0 and torch.equal(out, some)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(args, before))


@pytest.mark.parametrize("D,G,news", [(64, 4, [150, 20]), (96, 1, [70, 3]), (128, 8, [90, 1])])
def test_an_output_off_a_sector(D, G, news):
    c = BlockCache([150, 90], 1, D, 32, seed=2)
    q = queries(news, G, D, torch.bfloat16).cuda()
    want = prefill(c, q, news, default_scale(D))
    room = torch.full((q.numel() + 24,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = room[8: 8 + q.numel()].view(q.shape)
    assert out.data_ptr() % 32 == 16
    prefill(c, q, news, default_scale(D), out=out)
    assert torch.equal(out, want) and bool((room[:8] == 7).all()) and bool((room[-16:] == 7).all())


@pytest.mark.parametrize("dtype,D,Hkv,G,bs,lens,news", [
    (torch.bfloat16, 128, 2, 1, 32, [777, 300], [600, 300]),
    (torch.float16, 64, 1, 2, 16, [901], [500]),
    (torch.bfloat16, 96, 2, 1, 64, [513], [400])])
def test_long_row_tiles_over_an_unaligned_prefix(dtype, D, Hkv, G, bs, lens, news):
    c = BlockCache(lens, Hkv, D, bs, seed=G + D)
    q = queries(news, Hkv * G, D, dtype)
    out = prefill(c, q.cuda(), news, default_scale(D))
    assert pa.get_device_error() == 0
    check_prefill(c, G, q, news, out, default_scale(D), 23)


@pytest.mark.parametrize("lens", [[1], [500], [40, 3000, 0, 700]])
def test_tables_far_wider_than_the_contexts(lens):
    c = BlockCache(lens, 2, 128, 32, seed=3)
    q = queries([1] * len(lens), 8, 128, torch.bfloat16)
    d = c.dev()
    wide = torch.full((len(lens), 4096), -1, dtype=torch.int32, device="cuda")
    wide[:, : c.MB] = d["tables"]
    d["tables"], c.MB = wide, 4096
    out = decode(c, q.cuda(), default_scale(128))
    assert pa.get_device_error() == 0
    check_decode(c, 4, q, out, default_scale(128))
