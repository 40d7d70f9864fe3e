"""Norm with rotation, and the block-scaled FP8 cache, without a GPU: refusals of the C ABI (fake
pointers are never dereferenced), the binding's checks, the angles' fixed point, the budget."""
import math
import random

import pytest
import torch

from _block_cache import power_above
from paged_kv_cache_context_gb300 import pa

P = 4096  # a fake, 16-byte aligned, never-dereferenced pointer
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    from paged_kv_cache_context_gb300 import build
    build.build()
    return pa.lib()


def rope(L, **kw):
    a = dict(qo=P, ko=P, q=P, k=P, qw=P, kw=P, tu=P, pos=P, T=3, Hq=8, Hkv=2, D=128, R=128, A=1,
             so=1024, sk=256, si=1024, sj=256, eps=1e-6, inter=0, dt=1)
    a.update(kw)
    return L.pa_norm_rope(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), -1), (dict(ko=None), -1), (dict(pos=None), -1), (dict(tu=None), -1),
    (dict(dt=3), -2), (dict(dt=-1), -2), (dict(T=-1), -3), (dict(Hq=0), -3), (dict(Hkv=0), -3),
    (dict(R=8), -3), (dict(R=144), -3), (dict(R=-16), -3), (dict(A=0), -3), (dict(A=9), -3),
    (dict(eps=-1.0), -3), (dict(eps=float("nan")), -3), (dict(eps=float("inf")), -3),
    (dict(si=1023), -3), (dict(si=1028), -3), (dict(sj=255), -3), (dict(so=0), -3),
    (dict(sk=-256), -3), (dict(si=1 << 40), -3),
    (dict(D=120), -4), (dict(D=0), -4), (dict(D=272), -4),
    (dict(q=P + 8), -10), (dict(ko=P + 2), -10), (dict(qw=P + 4), -10), (dict(tu=P + 4), -10),
    (dict(pos=P + 2), -10),
])
def test_norm_rope_rejects_bad_arguments_on_host(L, kw, code):
    assert rope(L, **kw) == code
    assert rope(L, T=0, q=None) == 0


def store(L, **kw):
    a = dict(qo=P, q=P, k=P, v=P, kc=P, vc=P, slots=P, qw=P, kw=P, tu=P, pos=P, T=3, Hq=8, Hkv=2,
             D=128, R=128, A=1, bs=32, NB=4, so=1024, si=1024, sj=256, sv=256, eps=1e-6, inter=0,
             dt=1, kv=0, k1=1.0, v1=1.0)
    a.update(kw)
    return L.pa_norm_rope_and_cache(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(v=None), -1), (dict(slots=None), -1), (dict(kc=None), -1), (dict(kv=2), -2),
    (dict(kv=3), -2), (dict(kv=pa.PA_KV_FP8_BLOCK), -2), (dict(dt=5), -2), (dict(NB=0), -3), (dict(sv=100), -3), (dict(R=24), -3),
    (dict(D=100), -4), (dict(bs=0), -5), (dict(bs=1025), -5), (dict(vc=P + 4), -10),
    (dict(slots=P + 4), -10), (dict(kv=1, k1=0.0), -11), (dict(kv=1, v1=float("nan")), -11),
])
def test_norm_rope_and_cache_rejects_bad_arguments_on_host(L, kw, code):
    assert store(L, **kw) == code
    assert store(L, T=0, q=None) == 0


def append(L, **kw):
    a = dict(k=P, v=P, kc=P, vc=P, ks=P, vs=P, bt=P, cu=P, cl=P, T=8, S=2, H=2, D=128, bs=32,
             NB=10, MB=4, sk=256, sv=256, dt=1)
    a.update(kw)
    return L.pa_append_fp8_block(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), -1), (dict(vs=None), -1), (dict(cu=None), -1), (dict(dt=9), -2),
    (dict(T=-1), -3), (dict(S=-1), -3), (dict(S=70000), -3), (dict(H=0), -3), (dict(NB=0), -3),
    (dict(MB=0), -3), (dict(MB=1 << 27), -3), (dict(sk=255), -3), (dict(sv=257), -3),
    (dict(T=1 << 30, S=60000, H=60, sk=1 << 14, sv=1 << 14), -3),
    (dict(D=80), -4), (dict(D=256), -4), (dict(bs=8), -5), (dict(bs=128), -5),
    (dict(kc=P + 8), -10), (dict(v=P + 2), -10), (dict(ks=P + 2), -10),
])
def test_append_rejects_bad_arguments_on_host(L, kw, code):
    assert append(L, **kw) == code
    assert append(L, T=0, k=None) == 0 and append(L, S=0, k=None) == 0


def decode(L, **kw):
    a = dict(out=P, q=P, kc=P, vc=P, ks=P, vs=P, bt=P, cl=P, S=2, Hq=8, Hkv=2, D=128, bs=32,
             NB=10, MB=4, scale=0.1, qd=1, ws=P, wsb=BIG)
    a.update(kw)
    return L.pa_decode_fp8_block(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), -1), (dict(ks=None), -1), (dict(ws=None), -1), (dict(qd=0), -2),
    (dict(qd=7), -2), (dict(Hq=7), -3), (dict(Hq=18), -3), (dict(S=-1), -3), (dict(NB=0), -3),
    (dict(NB=1 << 26, Hkv=8), -3), (dict(D=80), -4), (dict(bs=8), -5), (dict(wsb=1 << 20), -7),
    (dict(ws=P + 8), -10), (dict(kc=P + 2), -10), (dict(vs=P + 2), -10),
])
def test_decode_rejects_bad_arguments_on_host(L, kw, code):
    assert decode(L, **kw) == code
    assert decode(L, S=0, q=None) == 0


def prefill(L, **kw):
    a = dict(out=P, q=P, kc=P, vc=P, ks=P, vs=P, bt=P, cu=P, cl=P, T=8, S=2, Hq=8, Hkv=2, D=128,
             bs=32, NB=10, MB=4, mq=4, scale=0.1, qd=1, ws=P, wsb=BIG)
    a.update(kw)
    return L.pa_prefill_fp8_block(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), -1), (dict(ks=None), -1), (dict(cu=None), -1), (dict(ws=None), -1),
    (dict(qd=0), -2), (dict(qd=7), -2), (dict(Hq=7), -3), (dict(Hq=18), -3), (dict(S=-1), -3),
    (dict(S=70000), -3), (dict(T=-1), -3), (dict(NB=0), -3), (dict(MB=0), -3), (dict(mq=0), -3),
    (dict(mq=9), -3), (dict(MB=1 << 26), -3), (dict(NB=1 << 30, Hkv=8), -3),
    (dict(T=1 << 29, mq=1), -3), (dict(D=80), -4), (dict(bs=8), -5), (dict(wsb=1 << 20), -7),
    (dict(ws=P + 8), -10), (dict(kc=P + 2), -10), (dict(vs=P + 2), -10),
])
def test_prefill_rejects_bad_arguments_on_host(L, kw, code):
    assert prefill(L, **kw) == code
    assert prefill(L, S=0, q=None) == 0 and prefill(L, T=0, q=None) == 0
    n = L.pa_prefill_fp8_block_workspace_size(8, 2, 128)
    assert n > L.pa_prefill_fp8_block_workspace_size(8, 2, 64) > 0 and prefill(L, wsb=n - 1) == -7
    assert L.pa_prefill_fp8_block_workspace_size(8, 3, 128) == 0
    assert L.pa_prefill_fp8_block_workspace_size(8, 2, 80) == 0


def floor_sum(n, m, a, b):
    """The kernel's sum of floor((a i + b) / m) over [0, n), restated."""
    s, N, M, A, B = 0, n, m, a, b
    while N > 0:
        s += N * (N - 1) // 2 * (A // M)
        A %= M
        s += N * (B // M)
        B %= M
        y = A * N + B
        if y < M:
            break
        N, B = y // M, y % M
        A, M = M, A
    return s


def test_the_shares_cover_every_tile_once():
    """The prefill's arithmetic restated: units before a row tile (one besides its tiles each),
    the search for a share's first one, and the shares' pieces."""
    rng = random.Random(5)
    for _ in range(300):
        tt, tokens = rng.choice([(64, 128), (128, 256)])
        tokens //= rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
        q_len, pos0 = rng.randint(1, 5000), rng.randint(0, 9000)
        rts = -(-q_len // tokens)
        tiles = [-(-(pos0 + min((r + 1) * tokens, q_len)) // tt) for r in range(rts)]
        before = [floor_sum(r, tt, tokens, pos0 + tokens + tt - 1) + r for r in range(rts)]
        assert before == [sum(tiles[:r]) + r for r in range(rts)]
        total = sum(tiles) + rts
        for rem in [0, total - 1] + [rng.randrange(total) for _ in range(5)]:
            a, e = 0, rts
            while e - a > 1:
                step = (e - a + 31) // 32
                k = sum(c < e and before[c] <= rem for c in range(a, a + 32 * step, step)) - 1
                a += k * step
                e = min(e, a + step)
            assert before[a] <= rem < before[a] + tiles[a] + 1
        # every CTA walks its share; a row tile's pieces are those that its join looks for
        ctas = rng.choice([1, 2, 7, 152, 304])
        share = -(-total // ctas)
        pieces = {}
        for c in range(ctas):
            lo = min(c * share, total)
            left = min(lo + share, total) - lo
            if left == 0:
                continue
            r = max(i for i in range(rts) if before[i] <= lo)
            skip = max(1 - (lo - before[r]), 0)
            tile, left, index = lo - before[r] + skip - 1, left - skip, 0
            while left > 0:
                n = min(left, tiles[r] - tile)
                pieces.setdefault(r, []).append((c, min(index, 1), tile, n))
                index, left, tile = index + 1, left - n, tile + n
                if left > 0 and tile == tiles[r]:
                    left, tile, r = left - 1, 0, r + 1
        for r in range(rts):
            assert [p[2] for p in pieces[r]] == [sum(p[3] for p in pieces[r][:j])
                                                 for j in range(len(pieces[r]))]
            assert sum(p[3] for p in pieces[r]) == tiles[r]
            c0 = (before[r] + 1) // share
            n = (before[r] + tiles[r]) // share - c0 + 1
            first = 1 if c0 * share < before[r] else 0
            assert [p[:2] for p in pieces[r]] == [(c0 + j, first if j == 0 else 0) for j in range(n)]


def test_the_other_decodes_refuse_the_block_scaled_kind(L):
    f = L.pa_decode
    for kv in (pa.PA_KV_FP8_BLOCK, 3):
        assert f(P, P, P, P, P, P, 2, 8, 2, 128, 32, 10, 4, 0.1, 0, 1, kv, 1.0, 1.0, None, 0, None) == -2
        assert L.pa_reshape_and_cache(P, P, P, P, P, 2, 2, 128, 32, 10, 1, kv, 1.0, 1.0, None) == -2
    assert L.pa_block_budget(0, 1.0, 0, 32, 8, 128, 32, 1, 3) == -2


def test_block_budget_counts_the_page_scales(L):
    n = pa.block_budget(4, 8, 128, 32, torch.bfloat16, "fp8_block", mb=64)
    assert n == (64 << 20) // (4 * 2 * 8 * (32 * 128 + 4))
    assert pa.block_budget(1, 1, 64, 16, torch.float16, "fp8_block", context_tokens=33) == 3


def test_turns_are_exact_modulo_one():
    f = torch.tensor([1.0, 0.1, 1e-4, -0.3, 7.0, 0.0, 2 * math.pi], dtype=torch.float64)
    turns = pa.rope_turns(f)
    assert turns.shape == (1, 7) and turns.dtype == torch.int64
    for pos in (0, 1, -5, 131071, 2 ** 31 - 1, -2 ** 31):
        for i, x in enumerate(f.tolist()):
            got = (pos * int(turns[0, i])) % 2 ** 64 / 2 ** 64
            want = math.cos(pos * x), math.sin(pos * x)
            # an angle in 64 bits is off by 2^-52 of itself, a fraction by 2^-52 of a turn a step
            tol = 2.0 ** -50 * (1 + abs(pos) * (abs(x) + 7))
            assert abs(math.cos(2 * math.pi * got) - want[0]) <= tol
            assert abs(math.sin(2 * math.pi * got) - want[1]) <= tol
    two = pa.rope_turns(torch.rand(3, 8, dtype=torch.float64))
    assert two.shape == (3, 8) and two.is_contiguous()
    with pytest.raises(ValueError):
        pa.rope_turns(torch.tensor([1.0, float("inf")]))
    with pytest.raises(ValueError):
        pa.rope_turns(torch.ones(2, 2, 2))


def test_powers():
    for a, s in ((448.0, 1.0), (448.5, 2.0), (1.0, 2.0 ** -8), (1.75, 2.0 ** -8), (1.76, 2.0 ** -7),
                 (0.0, 0.0), (1e-45, 2.0 ** -126)):
        assert power_above(a) == s


def test_binding_refuses_what_it_cannot_pass():
    q, k = torch.zeros(3, 8, 128), torch.zeros(3, 2, 128)
    tu, pos = torch.zeros(1, 64, dtype=torch.int64), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        pa.norm_rope(q, k, q, k, tu, pos)
    with pytest.raises(ValueError, match="contiguous"):
        pa.norm_rope(q, k, q.transpose(0, 1).contiguous().transpose(0, 1), k, tu, pos)
    with pytest.raises(ValueError, match="query"):
        pa.norm_rope(q, k, q[0], k, tu, pos)
    with pytest.raises(ValueError, match="contiguous"):
        pa.append_fp8_block(k[:, :, ::2], k[:, :, ::2], *[k] * 7)
    with pytest.raises(ValueError, match="key"):
        pa.norm_rope(q, k, q, k[:2], tu, pos)
    with pytest.raises(ValueError, match="positions"):
        pa.norm_rope(q, k, q, k, tu, pos.long())
    with pytest.raises(ValueError, match="q_weight"):
        pa.norm_rope(q, k, q, k, tu, pos, q_weight=torch.ones(64))
    with pytest.raises(ValueError, match="q_out"):
        pa.norm_rope(q.half(), k, q, k, tu, pos)
    kc = torch.zeros(4, 2, 32, 128)
    slots = torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError, match="kv_dtype"):
        pa.norm_rope_and_cache(q, q, k, k, kc, kc, slots, tu, pos, kv_dtype="int8")
    with pytest.raises(ValueError, match="slot_mapping"):
        pa.norm_rope_and_cache(q, q, k, k, kc, kc, slots.int(), tu, pos)
    with pytest.raises(ValueError, match="k_cache"):
        pa.norm_rope_and_cache(q, q, k, k, kc.half(), kc.half(), slots, tu, pos)
    codes, sc = kc.to(torch.uint8), torch.zeros(4, 2)
    bt, cu, n = (torch.zeros(s, dtype=torch.int32) for s in ((1, 4), (2,), (1,)))
    for bad, name in (((codes, codes.int(), sc, sc, bt, cu, n), "v_cache"),
                      ((codes, codes, sc[:3], sc, bt, cu, n), "k_scales"),
                      ((codes, codes, sc, sc.double(), bt, cu, n), "v_scales"),
                      ((codes, codes, sc, sc, bt[0], cu, n), "block_tables"),
                      ((codes, codes, sc, sc, bt, cu[:1], n), "cu_q"),
                      ((codes, codes, sc, sc, bt, cu, n.long()), "context_lens"),
                      ((codes, codes, sc, sc, bt, cu, n), "CUDA tensor")):
        with pytest.raises(ValueError, match=name):
            pa.append_fp8_block(k, k, *bad)
    with pytest.raises(ValueError, match="CUDA tensor"):
        pa.decode_fp8_block(q, q, codes, codes, sc, sc, bt, n, 2, 0.1, codes)
    with pytest.raises(ValueError, match="CUDA tensor"):
        pa.prefill_fp8_block(q, q, codes, codes, sc, sc, bt, cu, n, 2, 3, 0.1, codes)
