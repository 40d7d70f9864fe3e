"""Tree attention, scored decode, eviction choice and compaction without a GPU: refusals of the C
ABI (fake pointers are never dereferenced), the binding's checks, the mask helper, and the tree
kernel's share arithmetic restated."""
import random

import pytest
import torch

from paged_kv_cache_context_gb300 import pa

P = 4096  # a fake, 16-byte aligned, never-dereferenced pointer
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    from paged_kv_cache_context_gb300 import build
    build.build()
    return pa.lib()


def tree(L, kind="", **kw):
    a = dict(out=P, q=P, k=P, v=P, ks=P, vs=P, bt=P, cu=P, cl=P, mask=P, T=8, S=2, Hq=8, Hkv=2,
             D=128, bs=32, NB=10, MB=4, mq=4, W=1, scale=0.1, k1=1.0, v1=1.0, qd=1, ws=P, wsb=BIG)
    a.update(kw)
    args = [a["out"], a["q"], a["k"], a["v"]]
    args += [a["ks"], a["vs"]] if kind == "_int8" else []
    args += [a[x] for x in ("bt", "cu", "cl", "mask", "T", "S", "Hq", "Hkv", "D", "bs", "NB", "MB",
                            "mq", "W", "scale")]
    args += [a["k1"], a["v1"]] if kind == "_fp8" else []
    return getattr(L, "pa_tree" + kind)(*args, a["qd"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kind", ["", "_int8", "_fp8"])
@pytest.mark.parametrize("kw,code", [
    (dict(q=None), -1), (dict(mask=None), -1), (dict(cu=None), -1), (dict(ws=None), -1),
    (dict(qd=0), -2), (dict(qd=9), -2),
    (dict(Hq=7), -3), (dict(Hq=18, Hkv=2), -3), (dict(S=-1), -3), (dict(S=70000), -3),
    (dict(T=-1), -3), (dict(NB=0), -3), (dict(MB=0), -3), (dict(mq=0), -3), (dict(mq=9), -3),
    (dict(W=0), -3), (dict(T=200, mq=65), -3), (dict(MB=1 << 27), -3),
    (dict(T=1 << 20, mq=1 << 20, W=1 << 14, Hq=80, Hkv=10), -3),
    (dict(D=96), -4), (dict(D=256), -4), (dict(bs=8), -5), (dict(bs=128), -5),
    (dict(wsb=1024), -7), (dict(q=P + 8), -10), (dict(ws=P + 8), -10), (dict(mask=P + 4), -10),
])
def test_tree_rejects_bad_arguments_on_host(L, kind, kw, code):
    assert tree(L, kind, **kw) == code


def test_tree_kinds_reject_their_own(L):
    assert tree(L, NB=1 << 26, Hkv=8, Hq=8) == -3            # rows past 32-bit coordinates
    assert tree(L, "_int8", ks=None) == -1 and tree(L, "_int8", vs=P + 4) == -10
    for bad in (0.0, -1.0, float("inf"), float("nan")):
        assert tree(L, "_fp8", k1=bad) == -11 and tree(L, "_fp8", v1=bad) == -11
    for kind in ("", "_int8", "_fp8"):
        assert tree(L, kind, T=0, q=None) == 0 and tree(L, kind, S=0, q=None) == 0
    assert L.pa_tree_workspace_size(8, 2, 96) == 0 and L.pa_tree_workspace_size(7, 2, 64) == 0
    assert L.pa_tree_workspace_size(8, 2, 128) > L.pa_tree_workspace_size(8, 2, 64) > 0


def scored(L, int8=False, **kw):
    a = dict(out=P, sc=P, q=P, k=P, v=P, ks=P, vs=P, bt=P, cl=P, S=2, Hq=8, Hkv=2, D=128, bs=32,
             NB=10, MB=4, scale=0.1, qd=1, kvd=0, k1=1.0, v1=1.0, ws=P, wsb=BIG)
    a.update(kw)
    head = [a["out"], a["sc"], a["q"], a["k"], a["v"]]
    mid = [a[x] for x in ("bt", "cl", "S", "Hq", "Hkv", "D", "bs", "NB", "MB", "scale", "qd")]
    if int8:
        return L.pa_decode_scored_int8(*head, a["ks"], a["vs"], *mid, a["ws"], a["wsb"], None)
    return L.pa_decode_scored(*head, *mid, a["kvd"], a["k1"], a["v1"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(q=None), -1), (dict(sc=None), -1), (dict(ws=None), -1), (dict(qd=7), -2),
    (dict(Hq=7), -3), (dict(Hq=18, Hkv=2), -3), (dict(S=-1), -3), (dict(NB=0), -3),
    (dict(MB=1 << 26), -3), (dict(D=80), -4), (dict(bs=8), -5), (dict(wsb=1 << 20), -7),
    (dict(sc=P + 4), -10), (dict(ws=P + 8), -10), (dict(k=P + 2), -10),
])
def test_scored_rejects_bad_arguments_on_host(L, int8, kw, code):
    assert scored(L, int8, **kw) == code


def test_scored_kinds_reject_their_own(L):
    assert scored(L, kvd=2) == -2 and scored(L, kvd=1, k1=0.0) == -11
    assert scored(L, True, qd=0) == -2 and scored(L, True, vs=None) == -1
    assert scored(L, S=0, q=None) == 0 and scored(L, True, S=0, q=None) == 0
    n = L.pa_decode_scored_workspace_size(2, 8, 2, 128, 32, 4)
    assert scored(L, wsb=n - 1) == -7
    assert L.pa_decode_scored_workspace_size(4, 8, 2, 128, 32, 4) - n >= 2 * 8 * 4 * 32 * 4
    # past 32 bits
    assert L.pa_decode_scored_workspace_size(64, 32, 8, 128, 32, 1 << 16) > 1 << 32
    assert L.pa_decode_scored_workspace_size(2, 9, 2, 128, 32, 4) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(keep=None), -1), (dict(sc=None), -1), (dict(S=-1), -3), (dict(S=70000), -3),
    (dict(H=0), -3), (dict(N=0), -3), (dict(B=0), -3), (dict(sink=-1), -3), (dict(recent=-1), -3),
    (dict(sink=9, recent=8), -3), (dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1), -3),
    # 32-bit positions would run over
    (dict(N=2 ** 31 - 1), -3), (dict(B=2 ** 31 - 1), -3),
])
def test_select_rejects_bad_arguments_on_host(L, kw, code):
    a = dict(keep=P, new=P, sc=P, cl=P, S=2, H=2, N=64, B=16, sink=1, recent=4)
    a.update(kw)
    assert L.pa_evict_select(*a.values(), None) == code
    a["S"] = 0
    assert L.pa_evict_select(*a.values(), None) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), -1), (dict(keep=None), -1), (dict(kl=None), -1), (dict(ks=P), -1),
    (dict(eb=3), -2), (dict(S=-1), -3), (dict(H=0), -3), (dict(kh=3), -3), (dict(B=0), -3),
    (dict(NB=0), -3), (dict(MB=0), -3), (dict(MB=1 << 27), -3), (dict(D=0), -4), (dict(D=4), -4),
    (dict(D=1024), -4), (dict(bs=0), -5), (dict(k=P + 8), -10), (dict(sc=P + 4), -10),
    (dict(ks=P + 4, vs=P), -10),
])
def test_compact_rejects_bad_arguments_on_host(L, kw, code):
    a = dict(k=P, v=P, ks=None, vs=None, sc=None, bt=P, cl=P, keep=P, kl=P, st=None, S=2, H=2, kh=2,
             B=8, D=128, bs=32, NB=8, MB=4, eb=2)
    a.update(kw)
    assert L.pa_compact(*a.values(), None) == code
    a["S"] = 0
    assert L.pa_compact(*a.values(), None) == 0


# ---------------------------------------------------------------- binding
class Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def fn(*args):
            self.calls.append((name, args))
            return 0
        return fn


@pytest.fixture
def fake(monkeypatch):
    rec = Recorder()
    monkeypatch.setattr(pa, "lib", lambda: rec)
    monkeypatch.setattr(pa, "_stream", lambda stream=None: 0)
    monkeypatch.setattr(pa, "_is_device_tensor", lambda t: True)
    return rec


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def args(cd=torch.bfloat16):
    q = torch.zeros(5, 8, 64, dtype=torch.bfloat16)
    k = torch.zeros(10, 2, 16, 64, dtype=cd)
    return dict(out=torch.zeros_like(q), query=q, k_cache=k, v_cache=k.clone(),
                block_tables=i32(3, 4), context_lens=i32(3), num_kv_heads=2, scale=0.125,
                workspace=torch.zeros(64, dtype=torch.uint8))


def test_binding_passes_sizes(fake):
    a = args()
    pa.tree_attention(**a, cu_q=i32(4), tree_mask=torch.zeros(5, 2, dtype=torch.int64), max_q_len=3)
    name, c = fake.calls[-1]
    assert name == "pa_tree" and c[8:20] == (5, 3, 8, 2, 64, 16, 10, 4, 3, 2, 0.125, pa.PA_BF16)
    assert c[21] == 64
    sc = torch.zeros(10, 2, 16)
    pa.tree_attention_int8(**args(torch.int8), cu_q=i32(4), k_scales=sc, v_scales=sc.clone(),
                           tree_mask=torch.zeros(5, 2, dtype=torch.int64), max_q_len=3)
    assert fake.calls[-1][1][10:20] == (5, 3, 8, 2, 64, 16, 10, 4, 3, 2)
    pa.tree_attention_fp8(**args(torch.uint8), cu_q=i32(4), k_scale=2.0, v_scale=3.0,
                          tree_mask=torch.zeros(5, 2, dtype=torch.int64), max_q_len=3)
    assert fake.calls[-1][1][18:22] == (0.125, 2.0, 3.0, pa.PA_BF16)
    a = args()
    a["block_tables"], a["context_lens"] = i32(5, 4), i32(5)
    pa.decode_scored(scores=torch.zeros(5, 2, 64), **a)
    assert fake.calls[-1][1][7:16] == (5, 8, 2, 64, 16, 10, 4, 0.125, pa.PA_BF16)
    pa.evict_select(i32(5, 2, 7), i32(5), torch.zeros(5, 2, 64), i32(5), 1, 2)
    assert fake.calls[-1][1][4:10] == (5, 2, 64, 7, 1, 2)
    pa.compact(a["k_cache"], a["v_cache"], i32(5, 4), i32(5), i32(5, 1, 7), i32(5))
    assert fake.calls[-1][1][10:19] == (5, 2, 1, 7, 64, 16, 10, 4, 2)


@pytest.mark.parametrize("change", [
    dict(cu_q=i32(3)), dict(cu_q=torch.zeros(4, dtype=torch.int64)), dict(context_lens=i32(4)),
    dict(tree_mask=torch.zeros(4, 2, dtype=torch.int64)), dict(tree_mask=i32(5, 2)),
    dict(tree_mask=torch.zeros(5, dtype=torch.int64)),
    dict(out=torch.zeros(5, 8, 32, dtype=torch.bfloat16)), dict(num_kv_heads=4),
    dict(k_cache=torch.zeros(10, 2, 16, 64)), dict(block_tables=torch.zeros(3, 4)),
    dict(query=torch.zeros(5, 64, 8, dtype=torch.bfloat16).transpose(1, 2)),
])
def test_tree_mismatches_raise(fake, change):
    a = dict(args(), cu_q=i32(4), tree_mask=torch.zeros(5, 2, dtype=torch.int64), max_q_len=3)
    a.update(change)
    with pytest.raises(ValueError):
        pa.tree_attention(**a)
    assert fake.calls == []


@pytest.mark.parametrize("change", [
    dict(scores=torch.zeros(5, 2, 63)), dict(scores=torch.zeros(5, 2, 64, dtype=torch.float64)),
    dict(scores=torch.zeros(5, 8, 64)), dict(context_lens=i32(4)),
    dict(scores=torch.zeros(5, 64, 2).transpose(1, 2)),
])
def test_scored_mismatches_raise(fake, change):
    a = dict(args(), scores=torch.zeros(5, 2, 64), block_tables=i32(5, 4), context_lens=i32(5))
    a.update(change)
    with pytest.raises(ValueError):
        pa.decode_scored(**a)
    assert fake.calls == []


def test_evict_mismatches_raise(fake):
    sc = torch.zeros(5, 2, 64)
    for keep, new, s, n in ((i32(5, 3, 7), i32(5), sc, i32(5)), (i32(5, 2, 7), i32(4), sc, i32(5)),
                            (i32(5, 2, 7), i32(5), sc.double(), i32(5)),
                            (i32(5, 2, 7).long(), i32(5), sc, i32(5)),
                            (i32(5, 2), i32(5), sc, i32(5)), (i32(5, 2, 7), i32(5), sc, i32(6))):
        with pytest.raises(ValueError):
            pa.evict_select(keep, new, s, n)
    k = torch.zeros(10, 2, 16, 64, dtype=torch.int8)
    ks = torch.zeros(10, 2, 16)
    good = dict(k_cache=k, v_cache=k.clone(), block_tables=i32(5, 4), context_lens=i32(5),
                keep=i32(5, 2, 7), keep_lens=i32(5))
    for change in (dict(keep=i32(5, 3, 7)), dict(keep=i32(4, 2, 7)), dict(starts=i32(4)),
                   dict(k_scales=ks), dict(k_scales=ks, v_scales=ks[:9]), dict(keep_lens=i32(4)),
                   dict(scores=torch.zeros(5, 2, 65)), dict(v_cache=k.float()),
                   dict(v_cache=k.transpose(0, 1).contiguous().transpose(0, 1))):
        with pytest.raises(ValueError):
            pa.compact(**{**good, **change})
    assert fake.calls == []
    with pytest.raises(ValueError, match="CUDA"):
        pa._is_device_tensor = lambda t: t.is_cuda
        pa.compact(**good)


# ---------------------------------------------------------------- mask helper
def test_mask_helper_names_self_and_ancestors():
    r = random.Random(3)
    for sizes in ([1], [3, 0, 130], [64, 65], []):
        cu, par = [0], []
        for t in sizes:
            par += [r.randint(-1, i - 1) for i in range(t)]
            cu.append(cu[-1] + t)
        m = pa.tree_mask_from_parents(torch.tensor(par, dtype=torch.int64), torch.tensor(cu))
        assert m.dtype == torch.int64 and m.shape == (cu[-1], max([1] + [-(-t // 64) for t in sizes]))
        for a, b in zip(cu, cu[1:]):
            for i in range(b - a):
                want, k = set(), i
                while k >= 0:
                    want.add(k)
                    k = par[a + k]
                got = {64 * w + j for w in range(m.shape[1]) for j in range(64)
                       if int(m[a + i, w]) >> j & 1}
                assert got == want


def test_mask_helper_refuses_what_is_no_tree():
    for par, cu in (([0], [0, 1]), ([-1, 1], [0, 2]), ([-1, -2], [0, 2]), ([-1, 0], [0, 1, 2]),
                    ([-1], [0, 2]), ([-1], [1, 1]), ([-1, -1], [0, 2, 1, 2])):
        with pytest.raises(ValueError):
            pa.tree_mask_from_parents(par, cu)


# ---------------------------------------------------------------- shares of the tree kernel
@pytest.mark.parametrize("seed", range(30))
def test_tree_shares_cover_and_the_join_finds_every_piece(seed):
    """The join's enumeration of a cut segment's partial slots against what the walk writes."""
    r = random.Random(seed)
    Hkv, C = r.choice([1, 2, 8]), r.choice([1, 3, 8, 304])
    segs, P = [], 0  # (first unit, tiles) of each (sequence, kv head, row tile)
    for _ in range(r.randint(1, 40)):
        T, RT = r.choice([0, 1, 1, 2, r.randint(1, 60)]), r.randint(1, 3)
        for _ in range(Hkv * RT if T else 0):
            segs.append((P, T))
            P += T
    if P == 0:
        return
    U = -(-P // C)
    wrote, units = {}, 0
    for c in range(C):
        a = min(c * U, P)
        b = min(a + U, P)
        piece = 0
        for i, (x, T) in enumerate(segs):
            lo, hi = max(a, x), min(b, x + T)
            if lo >= hi:
                continue
            units += hi - lo
            if hi - lo < T:
                key = (c, 1 if piece > 0 else 0)
                assert key not in wrote, "two cut pieces in one slot"
                wrote[key] = i
            piece += 1
    assert units == P
    found = {}
    for i, (x, T) in enumerate(segs):
        c0 = x // U
        n = (x + T - 1) // U - c0 + 1
        if n == 1:
            continue
        for j in range(n):
            found[(c0 + j, 1 if j == 0 and x != c0 * U else 0)] = i
    assert found == wrote
