"""pa_norm_rope and pa_norm_rope_and_cache on the GPU against the definition in 64 bits.

Bounds. With y the normed head, |y - its value| <= y (D / 2 + 8) 2^-24 (a sum of D squares
truncated at each step, halved by the root; the root's 2 ulp; three products). The angle is off by
pi 2^-25 (the fraction's conversion), its sine and cosine by 2 ulp besides: 2^-21. So a pair's
results are off by (|u| + |v|) ((D / 2 + 12) 2^-24 + 2^-21), and by one rounding to the output."""
import math

import pytest
import torch

from _ref64 import U
from paged_kv_cache_context_gb300 import pa

pytestmark = pytest.mark.gpu


def freqs(R, A, base=10000.0):
    f = base ** (-torch.arange(R // 2, dtype=torch.float64) / max(R // 2, 1))
    axis = torch.arange(R // 2) * A // max(R // 2, 1)
    return torch.where(axis[None] == torch.arange(A)[:, None], f[None], 0.0)


def turned(x, w, f, pos, eps, interleaved):
    """(values in 64 bits, their error bound without the last rounding), on the CPU."""
    y = x.double().cpu()
    D, R = y.shape[-1], 2 * f.shape[1]
    if w is not None:
        y = y / (y.pow(2).mean(-1, keepdim=True) + eps).sqrt() * w.double().cpu()
    ang = torch.einsum("at,ai->ti", pos.double().cpu(), f)[:, None, :]
    c, s = ang.cos(), ang.sin()
    if interleaved:
        u, v = y[..., 0:R:2], y[..., 1:R:2]
        rot = torch.stack([u * c - v * s, v * c + u * s], -1).flatten(-2)
        size = (u.abs() + v.abs()).repeat_interleave(2, -1)
    else:
        u, v = y[..., : R // 2], y[..., R // 2: R]
        rot = torch.cat([u * c - v * s, v * c + u * s], -1)
        size = torch.cat([u.abs() + v.abs()] * 2, -1)
    out = torch.cat([rot, y[..., R:]], -1)
    size = torch.cat([size, y[..., R:].abs()], -1)
    return out, size * ((D / 2 + 12) * 2.0 ** -24 + 2.0 ** -21)


def check(got, ref, bound):
    err = (got.double().cpu() - ref).abs()
    tol = bound * 1.01 + ref.abs() * U[got.dtype] * 1.01 + 2.0 ** -25  # (f16's smallest steps)
    assert bool((err <= tol).all()), float((err / tol).max())


def inputs(T, Hq, Hkv, D, A, dtype, norm, seed, far=131072):
    g = torch.Generator().manual_seed(seed)
    qkv = (torch.randn(T, (Hq + 2 * Hkv) * D, generator=g) * 2).to(dtype).cuda()
    q, k, v = (qkv[:, a: b].view(T, -1, D) for a, b in
               ((0, Hq * D), (Hq * D, (Hq + Hkv) * D), ((Hq + Hkv) * D, (Hq + 2 * Hkv) * D)))
    w = [(1 + 0.3 * torch.randn(D, generator=g)).cuda() if norm else None for _ in range(2)]
    pos = torch.randint(-50, far, (A, T), generator=g, dtype=torch.int32).cuda()
    return q, k, v, w[0], w[1], pos


CASES = [
    # T, Hq, Hkv, D, R, A, interleaved, norm, dtype
    (1, 32, 8, 128, 128, 1, False, True, torch.bfloat16),
    (1, 1, 1, 16, 16, 1, True, True, torch.float16),
    (2, 7, 1, 64, 64, 1, False, True, torch.float32),
    (5, 5, 5, 96, 64, 3, True, True, torch.float16),
    (33, 8, 2, 80, 32, 1, False, True, torch.bfloat16),
    (17, 4, 2, 256, 256, 2, False, True, torch.bfloat16),
    (9, 3, 1, 256, 64, 8, True, True, torch.float32),
    (64, 12, 4, 112, 112, 1, False, True, torch.float16),
    (100, 40, 8, 128, 128, 3, False, False, torch.bfloat16),
    (257, 2, 1, 48, 16, 1, False, True, torch.float32),
    (700, 16, 16, 128, 96, 1, True, True, torch.bfloat16),
    (1500, 6, 2, 32, 32, 1, False, True, torch.float16),
    (4001, 8, 8, 64, 64, 1, False, False, torch.bfloat16),
    (3, 64, 64, 240, 240, 1, False, True, torch.float32),
    (11, 4, 2, 128, 0, 1, False, True, torch.bfloat16),
]


@pytest.mark.parametrize("T,Hq,Hkv,D,R,A,inter,norm,dtype", CASES)
def test_matches_the_definition(T, Hq, Hkv, D, R, A, inter, norm, dtype):
    pa.get_device_error()
    q, k, v, qw, kw, pos = inputs(T, Hq, Hkv, D, A, dtype, norm, T + D)
    f = freqs(R, A)
    turns = pa.rope_turns(f, "cuda")
    qo, ko = (torch.full_like(x, float("nan"), memory_format=torch.contiguous_format) for x in (q, k))
    pa.norm_rope(qo, ko, q, k, turns, pos, qw, kw, 1e-5, inter)
    assert pa.get_device_error() == 0
    check(qo, *turned(q, qw, f, pos, 1e-5, inter))
    check(ko, *turned(k, kw, f, pos, 1e-5, inter))


def test_one_weight_alone_and_positions_without_an_axis():
    q, k, v, qw, kw, pos = inputs(20, 8, 2, 128, 1, torch.float16, True, 5)
    f = freqs(128, 1)
    turns = pa.rope_turns(f, "cuda")
    qo, ko = q.contiguous().clone(), k.contiguous().clone()
    pa.norm_rope(qo, ko, q, k, turns, pos[0], None, kw)
    check(qo, *turned(q, None, f, pos, 1e-6, False))
    check(ko, *turned(k, kw, f, pos, 1e-6, False))


@pytest.mark.parametrize("T,D", [(3, 128), (900, 64), (50, 256)])
def test_in_place_in_the_projections_output(T, D):
    q, k, v, qw, kw, pos = inputs(T, 12, 4, D, 1, torch.bfloat16, True, T)
    f = freqs(D, 1)
    turns = pa.rope_turns(f, "cuda")
    qo, ko = torch.empty_like(q, memory_format=torch.contiguous_format), torch.empty_like(
        k, memory_format=torch.contiguous_format)
    pa.norm_rope(qo, ko, q, k, turns, pos, qw, kw)
    before = v.clone()
    pa.norm_rope(q, k, q, k, turns, pos, qw, kw)
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(v, before)


def test_far_positions_at_the_ends_of_32_bits():
    T = 8
    q, k, v, qw, kw, _ = inputs(T, 4, 1, 64, 1, torch.float32, False, 2)
    pos = torch.tensor([[0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 24 + 1, 10 ** 9 + 7, 99]],
                       dtype=torch.int32).cuda()
    # whole fractions of a turn: the angles of the definition are exact
    den = torch.arange(3, 35, dtype=torch.float64)
    frac = pos.cpu().double()[0][:, None] % den / den  # position mod den, exactly
    turns = torch.tensor([[int(2 ** 64 // int(d)) - (2 ** 64 if 2 ** 64 // int(d) >= 2 ** 63 else 0)
                           for d in den]], dtype=torch.int64).cuda()
    qo, ko = torch.empty_like(q, memory_format=torch.contiguous_format), torch.empty_like(
        k, memory_format=torch.contiguous_format)
    pa.norm_rope(qo, ko, q, k, turns, pos)
    y = q.double().cpu()
    c, s = (2 * math.pi * frac).cos()[:, None], (2 * math.pi * frac).sin()[:, None]
    u, w = y[..., :32], y[..., 32:]
    ref = torch.cat([u * c - w * s, w * c + u * s], -1)
    size = torch.cat([u.abs() + w.abs()] * 2, -1)
    check(qo, ref, size * 2.0 ** -20)


def test_another_stream_and_a_replayed_graph():
    q, k, v, qw, kw, pos = inputs(40, 8, 2, 128, 1, torch.bfloat16, True, 9)
    turns = pa.rope_turns(freqs(128, 1), "cuda")
    a, b = [torch.zeros_like(q, memory_format=torch.contiguous_format) for _ in range(2)]
    ka, kb = [torch.zeros_like(k, memory_format=torch.contiguous_format) for _ in range(2)]
    pa.norm_rope(a, ka, q, k, turns, pos, qw, kw)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        pa.norm_rope(b, kb, q, k, turns, pos, qw, kw)
    q.mul_(-1.0)
    k.mul_(-1.0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(b, -a) and torch.equal(kb, -ka)
    pa.norm_rope(b, kb, q, k, turns, pos, qw, kw, stream=st)
    st.synchronize()
    assert torch.equal(b, -a)


def test_empty_batches_do_nothing():
    q, k = torch.zeros(0, 8, 128, device="cuda"), torch.zeros(0, 2, 128, device="cuda")
    turns = pa.rope_turns(freqs(128, 1), "cuda")
    pa.norm_rope(q, k, q, k, turns, torch.zeros(1, 0, dtype=torch.int32, device="cuda"))
    assert pa.get_device_error() == 0


@pytest.mark.parametrize("kv", ["auto", "fp8_e4m3"])
@pytest.mark.parametrize("T,Hq,Hkv,D,bs,inter,norm,dtype", [
    (1, 32, 8, 128, 32, False, True, torch.bfloat16),
    (45, 4, 4, 64, 16, False, True, torch.float32),
    (333, 6, 2, 96, 64, True, True, torch.float16),
    (70, 5, 1, 256, 32, False, False, torch.bfloat16),
    (20, 9, 3, 48, 5, True, True, torch.float32),
])
def test_store_is_the_two_calls_bit_for_bit(kv, T, Hq, Hkv, D, bs, inter, norm, dtype):
    pa.get_device_error()
    q, k, v, qw, kw, pos = inputs(T, Hq, Hkv, D, 2, dtype, norm, T)
    turns = pa.rope_turns(freqs(D, 2), "cuda")
    NB = -(-T // bs) + 2
    g = torch.Generator().manual_seed(T)
    slots = torch.randperm(NB * bs, generator=g)[:T]
    slots[::7] = -1
    if T > 2:
        slots[1] = NB * bs + 3  # beyond the pool: flagged and skipped
    slots = slots.cuda()
    shape = (NB, Hkv, bs, D)
    if kv == "auto":
        kc, vc = (torch.randn(shape, generator=g).to(dtype).cuda() for _ in range(2))
    else:
        kc, vc = (torch.randint(0, 256, shape, generator=g, dtype=torch.uint8).cuda()
                  for _ in range(2))
    kc2, vc2 = kc.clone(), vc.clone()
    # (a power of two, and scales that are none)
    rest = dict(kv_dtype=kv, k_scale=0.037 if T % 2 else 0.03125, v_scale=0.011)
    qo, qo2 = (torch.zeros_like(q, memory_format=torch.contiguous_format) for _ in range(2))
    ko = torch.zeros_like(k, memory_format=torch.contiguous_format)
    pa.norm_rope(qo, ko, q, k, turns, pos, qw, kw, 1e-6, inter)
    pa.reshape_and_cache(ko, v.contiguous(), kc, vc, slots, **rest)
    first = pa.get_device_error()
    pa.norm_rope_and_cache(qo2, q, k, v, kc2, vc2, slots, turns, pos, qw, kw, 1e-6, inter, **rest)
    assert pa.get_device_error() == first == (1 if T > 2 else 0)
    assert torch.equal(qo, qo2)
    raw = (lambda x: x) if kv != "auto" else (lambda x: x.view(torch.int16 if x.element_size() == 2
                                                               else torch.int32))
    assert torch.equal(raw(kc), raw(kc2)) and torch.equal(raw(vc), raw(vc2))


def test_values_that_are_not_finite_stay_in_their_heads():
    q, k, v, qw, kw, pos = inputs(6, 4, 2, 64, 1, torch.float32, True, 1)
    q[2, 1, 5] = float("nan")
    k[3, 0, 7] = float("inf")
    turns = pa.rope_turns(freqs(64, 1), "cuda")
    qo, ko = torch.zeros(6, 4, 64, device="cuda"), torch.zeros(6, 2, 64, device="cuda")
    pa.norm_rope(qo, ko, q, k, turns, pos, qw, kw)
    bad_q, bad_k = ~qo.isfinite().all(-1), ~ko.isfinite().all(-1)
    assert bad_q.sum() == 1 and bad_q[2, 1] and bad_k.sum() == 1 and bad_k[3, 0]


@pytest.mark.parametrize("T,D,dtype", [(2, 96, torch.float16), (900, 96, torch.bfloat16),
                                       (3000, 80, torch.float32), (900, 176, torch.float16)])
def test_a_head_of_nan_or_zeros_leaves_the_others_of_its_token(T, D, dtype):
    """Head sizes that leave lanes without elements, and lanes that take many heads; eps = 0 makes
    a head of zeros NaN."""
    q, k, v, qw, kw, pos = inputs(T, 20, 4, D, 1, dtype, True, 3)
    q[:, 1, 3] = float("nan")
    q[:, 12] = 0
    k[:, 0, 5] = float("-inf")
    f = freqs(D - D % 32, 1)
    qo, ko = (torch.zeros_like(x, memory_format=torch.contiguous_format) for x in (q, k))
    pa.norm_rope(qo, ko, q, k, pa.rope_turns(f, "cuda"), pos, qw, kw, 0.0)
    keep = [h for h in range(20) if h not in (1, 12)]
    assert bool(qo[:, [1, 12]].isnan().any(-1).all())
    check(qo[:, keep], *turned(q[:, keep], qw, f, pos, 0.0, False))
    check(ko[:, 1:], *turned(k[:, 1:], kw, f, pos, 0.0, False))
