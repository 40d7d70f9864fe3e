"""NaN through the fused norm, rotation and store: codes as pa_norm_rope and then
pa_reshape_and_cache leave them, the sign of a NaN among them."""
import pytest
import torch

from paged_kv_cache_context_gb300 import pa
from test_gpu_rope import freqs, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("scale", [1.0, 0.03125, 0.037])
def test_nan_and_infinities_are_stored_as_by_the_two_calls(dtype, norm, scale):
    pa.get_device_error()
    T, H, D, bs = 9, 2, 64, 16
    q, k, v, qw, kw, pos = inputs(T, 4, H, D, 1, dtype, norm, 8)
    word, minus = {torch.bfloat16: (torch.int16, 0xFFC0 - 2 ** 16),
                   torch.float16: (torch.int16, 0xFE00 - 2 ** 16),
                   torch.float32: (torch.int32, 0xFFC00000 - 2 ** 32)}[dtype]
    for x in (k, v):
        x[1, 0, 3], x[4, 0, 0], x[5, 1, 60] = float("nan"), float("inf"), float("-inf")
        bits = x.view(word)
        bits[2, 1, 40] = bits[6, 0, 1] = minus  # NaN with its sign bit set
    turns = pa.rope_turns(freqs(32, 1), "cuda")  # the first 32 dims turn, the others pass
    slots = torch.arange(T, device="cuda") * 3
    caches = [torch.zeros(2, H, bs, D, dtype=torch.uint8, device="cuda") for _ in range(4)]
    qo, ko = (torch.zeros_like(x, memory_format=torch.contiguous_format) for x in (q, k))
    rest = dict(kv_dtype="fp8_e4m3", k_scale=scale, v_scale=scale)
    pa.norm_rope(qo, ko, q, k, turns, pos, qw, kw)
    pa.reshape_and_cache(ko, v.contiguous(), caches[0], caches[1], slots, **rest)
    pa.norm_rope_and_cache(qo, q, k, v, caches[2], caches[3], slots, turns, pos, qw, kw, **rest)
    assert pa.get_device_error() == 0
    assert torch.equal(caches[0], caches[2]) and torch.equal(caches[1], caches[3])
    assert bool((caches[1] == 0x7F).any()) and (dtype == torch.float16 or bool((caches[1] == 0xFF).any()))
