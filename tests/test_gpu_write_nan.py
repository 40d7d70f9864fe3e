"""NaN of both signs written to an FP8 cache: 0x7F with the input's sign bit, whatever the input's
type, by pa_reshape_and_cache and by the fused norm, rotation and store (which does not touch the
values)."""
import pytest
import torch

from paged_kv_cache_context_gb300 import pa
from test_gpu_rope import freqs

pytestmark = pytest.mark.gpu

WORDS = {torch.bfloat16: (torch.int16, (0x7FC0, 0x7F81, 0xFFC0, 0xFFFF)),
         torch.float16: (torch.int16, (0x7E00, 0x7C01, 0xFE00, 0xFFFF)),
         torch.float32: (torch.int32, (0x7FC00000, 0x7F800001, 0xFFC00000, 0xFFFFFFFF))}


@pytest.mark.parametrize("dtype", list(WORDS))
@pytest.mark.parametrize("scale", [1.0, 0.037])
def test_a_nan_keeps_its_sign(dtype, scale):
    word, bits = WORDS[dtype]
    T, H, D, bs = 4, 2, 64, 16
    x = torch.ones(T, H, D, dtype=dtype)
    for t, b in enumerate(bits):
        x.view(word)[t, 1, 3 * t: 3 * t + 2] = b - (2 ** (8 * x.element_size()) if t > 1 else 0)
    x = x.cuda()
    slots = torch.arange(T, device="cuda")
    kc, vc, kc2, vc2 = (torch.zeros(1, H, bs, D, dtype=torch.uint8, device="cuda") for _ in range(4))
    rest = dict(kv_dtype="fp8_e4m3", k_scale=scale, v_scale=scale)
    pa.reshape_and_cache(x, x, kc, vc, slots, **rest)
    pos = torch.zeros(T, dtype=torch.int32, device="cuda")
    pa.norm_rope_and_cache(torch.empty_like(x), x, x, x, kc2, vc2, slots,
                           pa.rope_turns(freqs(32, 1), "cuda"), pos, **rest)
    assert torch.equal(kc, vc) and torch.equal(vc, vc2)
    codes = kc.cpu()
    for t in range(T):
        want = 0xFF if t > 1 else 0x7F
        assert (codes[0, 1, t, 3 * t: 3 * t + 2] == want).all(), t
        assert ((codes[0, :, t] & 0x7F) == 0x7F).sum() == 2
