"""pa_tree on the GPU against attention in 64 bits over the same cache bytes.

Bounds: tests/_ref64.py, element by element."""
import numpy as np
import pytest
import torch

from _ref64 import Cache, attend, bits64, default_scale, weight_type
from paged_kv_cache_context_gb300 import pa

pytestmark = pytest.mark.gpu


def random_mask(nodes, words, seed, p_empty=0.1):
    """Random visible sets (self mostly among them), some rows empty; junk in bits past the draft."""
    r = np.random.RandomState(seed)
    T = sum(nodes)
    m = r.randint(0, 2, size=(T, words * 64)).astype(bool)
    at = 0
    for q in nodes:
        for i in range(q):
            m[at + i, i] = True
            if r.rand() < p_empty:
                m[at + i, :q] = False
        at += q
    return pack(m)


def pack(m):
    T, n = m.shape
    w = np.zeros((T, n // 64), dtype=np.uint64)
    for b in range(n):
        w[:, b // 64] |= m[:, b].astype(np.uint64) << np.uint64(b % 64)
    return torch.from_numpy(w.view(np.int64).copy())


def run(cache, q, cu, mask, max_q, scale, ws=None, out=None, stream=None):
    d = cache.dev()
    Hq = q.shape[1]
    if ws is None:
        ws = torch.full((pa.tree_workspace_size(Hq, cache.H, cache.D),), 0xFF, dtype=torch.uint8,
                        device="cuda")
    if out is None:
        out = torch.full_like(q, float("nan"))
    rest = (d["tables"], cu, d["lens"], mask, cache.H, max_q, scale)
    if cache.kv == "int8":
        pa.tree_attention_int8(out, q, d["k"], d["v"], d["ks"], d["vs"], *rest, ws, stream=stream)
    elif cache.kv == "fp8_e4m3":
        pa.tree_attention_fp8(out, q, d["k"], d["v"], *rest, cache.k_scale, cache.v_scale, ws,
                              stream=stream)
    else:
        pa.tree_attention(out, q, d["k"], d["v"], *rest, ws, stream=stream)
    return out


def inputs(cache, nodes, G, dtype, seed, words=None, qmul=1.5):
    g = torch.Generator().manual_seed(seed + 1)
    T = sum(nodes)
    q = (torch.randn(T, cache.H * G, cache.D, generator=g) * qmul).to(dtype)
    words = words or max(1, -(-max(nodes) // 64))
    mask = random_mask(nodes, words, seed)
    cu = torch.tensor([0] + nodes).cumsum(0).int()
    return q, cu, mask


def check(cache, nodes, G, q, mask, out, scale, heads=None):
    dtype = q.dtype
    got = out.float().cpu().double().numpy()
    qd = q.double().cpu().numpy()
    at = 0
    for s, t in enumerate(nodes):
        n = cache.lens[s]
        for g in range(cache.H):
            if heads is not None and g not in heads:
                continue
            K, V, codes = cache.rows(s, g)
            for i in range(t):
                seen = np.ones(n, dtype=bool)
                seen[n - t:] = bits64(mask[at + i].tolist(), t)
                for h in range(g * G, (g + 1) * G):
                    o, bound, _, _ = attend(qd[at + i, h], K, V, codes, seen, scale, dtype,
                                            weight_type(cache, dtype))
                    err = np.abs(got[at + i, h] - o)
                    assert (err <= bound).all(), (s, i, h, float((err / bound).max()))
        at += t


CASES = [
    # kv, dtype, D, Hkv, G, bs, lens, nodes
    ("auto", torch.bfloat16, 128, 2, 4, 32, [500], [8]),
    ("auto", torch.bfloat16, 64, 1, 1, 16, [1, 2, 63, 64, 65], [1, 2, 3, 64, 1]),
    ("auto", torch.float16, 128, 2, 3, 64, [127, 128, 129, 200], [5, 0, 17, 9]),
    ("auto", torch.bfloat16, 128, 1, 8, 32, [40, 100, 300], [40, 33, 100]),   # several row tiles
    ("auto", torch.float16, 64, 2, 4, 32, [130, 193], [130, 70]),             # no context; two words
    ("auto", torch.bfloat16, 128, 2, 1, 16, [3 + (7 * s) % 90 for s in range(40)],
     [1 + s % 3 for s in range(40)]),
    ("auto", torch.bfloat16, 128, 1, 2, 32, [5003], [6]),                     # one long sequence
    ("fp8_e4m3", torch.bfloat16, 128, 2, 1, 32, [333, 64, 1], [13, 31, 1]),
    ("fp8_e4m3", torch.float16, 64, 1, 8, 16, [100, 257], [20, 9]),
    ("int8", torch.bfloat16, 128, 2, 4, 32, [333, 65, 128], [13, 31, 2]),
    ("int8", torch.float16, 64, 1, 2, 64, [70, 700, 16], [64, 65, 16]),
    ("int8", torch.bfloat16, 128, 1, 5, 16, [2100], [7]),
    # 32, 33, 64, 65, 128, 129 rows: one row tile holds them four, two times, once; two tiles
    ("auto", torch.bfloat16, 128, 2, 1, 32, [333, 1000, 70, 65, 640, 129], [32, 33, 64, 65, 128, 129]),
    ("auto", torch.float16, 64, 2, 2, 16, [900, 77, 350], [16, 17, 32]),
    ("fp8_e4m3", torch.bfloat16, 64, 1, 4, 64, [700, 99], [8, 16]),
    ("int8", torch.float16, 128, 2, 1, 32, [500, 80], [40, 33]),
]


@pytest.mark.parametrize("kv,dtype,D,Hkv,G,bs,lens,nodes", CASES)
def test_matches_the_definition(kv, dtype, D, Hkv, G, bs, lens, nodes):
    pa.get_device_error()
    cache = Cache(lens, Hkv, D, bs, kv, dtype, seed=len(lens) + D)
    q, cu, mask = inputs(cache, nodes, G, dtype, 7)
    scale = default_scale(D)
    out = run(cache, q.cuda(), cu.cuda(), mask.cuda(), max(nodes), scale)
    assert pa.get_device_error() == 0
    check(cache, nodes, G, q, mask, out, scale)


# kv, dtype, D, G: with 24 sequences of up to 1500 tokens and 8 kv heads a CTA's
# share is several tiles long and holds whole segments, so that every ring of
# buffers goes round many times and pieces follow one another
LONG_SHARES = [
    ("auto", torch.bfloat16, 128, 1), ("auto", torch.float16, 64, 2), ("auto", torch.bfloat16, 128, 8),
    ("fp8_e4m3", torch.bfloat16, 128, 1), ("fp8_e4m3", torch.float16, 128, 2),
    ("fp8_e4m3", torch.bfloat16, 64, 1), ("fp8_e4m3", torch.bfloat16, 128, 8),
    ("int8", torch.bfloat16, 128, 1), ("int8", torch.float16, 128, 3), ("int8", torch.float16, 64, 1),
    ("int8", torch.float16, 128, 8),
]


@pytest.mark.parametrize("kv,dtype,D,G", LONG_SHARES)
def test_shares_of_many_tiles(kv, dtype, D, G):
    pa.get_device_error()
    lens = [40 + (977 * s) % (1460 if s % 3 == 0 else 300) for s in range(24)]
    nodes = [1 + s % (5 if G < 8 else 20) for s in range(24)]  # 8 rows a node: two query tiles a CTA
    cache = Cache(lens, 8, D, 32, kv, dtype, seed=D + G)
    q, cu, mask = inputs(cache, nodes, G, dtype, 11)
    args = (q.cuda(), cu.cuda(), mask.cuda(), max(nodes), default_scale(D))
    out = run(cache, *args)
    assert pa.get_device_error() == 0
    check(cache, nodes, G, q, mask, out, default_scale(D), heads=None if G <= 3 else [0, 5])
    ws = torch.zeros(pa.tree_workspace_size(8 * G, 8, D), dtype=torch.uint8, device="cuda")
    for _ in range(30):
        assert torch.equal(run(cache, *args, ws=ws), out)


@pytest.mark.parametrize("kv,dtype,D", [("auto", torch.float16, 128), ("fp8_e4m3", torch.bfloat16, 128),
                                        ("fp8_e4m3", torch.float16, 64), ("int8", torch.bfloat16, 64),
                                        ("int8", torch.float16, 128)])
def test_two_row_tiles_and_a_bound_above_every_draft(kv, dtype, D):
    """320 rows a kv head (256 and 64 of them in a tile), next to sequences of one node; then
    a max_q_len that asks for wide tiles where no draft has more than a few rows."""
    pa.get_device_error()
    cache = Cache([700, 41, 300], 2, D, 32, kv, dtype, seed=D)
    for nodes, max_q in (([40, 1, 17], 40), ([3, 1, 2], 100)):
        q, cu, mask = inputs(cache, nodes, 8, dtype, 13, words=2)
        q = torch.cat([q] * -(-max_q // q.shape[0]))      # with rows past the last sequence
        mask = torch.cat([mask, torch.zeros(q.shape[0] - mask.shape[0], 2, dtype=torch.int64)])
        out = torch.full_like(q, 7.0).cuda()
        run(cache, q.cuda(), cu.cuda(), mask.cuda(), max_q, default_scale(D), out=out)
        assert pa.get_device_error() == 0
        check(cache, nodes, 8, q, mask, out, default_scale(D))
        assert out[sum(nodes):].eq(7.0).all()


def test_a_chain_is_causal_prefill():
    cache = Cache([333, 70], 2, 128, 32, seed=5)
    nodes, G = [20, 64], 4
    q, cu, _ = inputs(cache, nodes, G, torch.bfloat16, 3)
    parents = [i - 1 for t in nodes for i in range(t)]
    mask = pa.tree_mask_from_parents(parents, cu)
    out = run(cache, q.cuda(), cu.cuda(), mask.cuda(), 64, 0.1)
    d = cache.dev()
    ref = torch.empty_like(out)
    pa.prefill(ref, q.cuda(), d["k"], d["v"], d["tables"], cu.cuda(), d["lens"], 2, 64, 0.1)
    # each rounds its weights and its output once: twice the bound of one
    qd = q.double().numpy()
    a, b = (x.float().cpu().double().numpy() for x in (out, ref))
    at = 0
    for s, t in enumerate(nodes):
        for h in range(8):
            K, V, codes = cache.rows(s, h // G)
            for i in range(t):
                seen = np.arange(cache.lens[s]) <= cache.lens[s] - t + i
                _, bound, _, _ = attend(qd[at + i, h], K, V, codes, seen, 0.1, torch.bfloat16,
                                        torch.bfloat16)
                assert (np.abs(a[at + i, h] - b[at + i, h]) <= 2 * bound).all()
        at += t


@pytest.mark.parametrize("scale,qmul", [(-0.2, 1.0), (0.0, 1.0), (1.0, 30.0)])
def test_other_scales_and_large_logits(scale, qmul):
    cache = Cache([200, 77], 1, 64, 16, seed=9)
    nodes = [9, 30]
    q, cu, mask = inputs(cache, nodes, 2, torch.bfloat16, 11, qmul=qmul)
    out = run(cache, q.cuda(), cu.cuda(), mask.cuda(), 30, scale)
    check(cache, nodes, 2, q, mask, out, scale)


def test_rows_that_see_nothing_are_zero():
    cache = Cache([5, 80], 1, 128, 32, seed=1)
    nodes = [5, 80]  # no context
    q, cu, _ = inputs(cache, nodes, 2, torch.bfloat16, 2)
    mask = torch.zeros(85, 2, dtype=torch.int64)
    mask[1, 0] = 1 << 4
    out = run(cache, q.cuda(), cu.cuda(), mask.cuda(), 80, 0.1)
    assert out[0].abs().max() == 0 and out[2:].abs().max() == 0
    v = cache.rows(0, 0)[1][4]
    assert (out[1].float().cpu().double().numpy() == v[None]).all()  # a weight of one


def test_bad_data_is_flagged_and_never_faults():
    cache = Cache([100, 90, 80, 70, 60], 2, 128, 32, seed=4)
    nodes, G = [4, 5, 6, 7, 8], 2
    q, cu, mask = inputs(cache, nodes, G, torch.bfloat16, 2)
    scale = default_scale(128)
    pa.get_device_error()
    d = cache.dev()
    good = d["lens"].clone()
    # a length below the draft's and one above the table: zero rows there, the rest as before
    want = run(cache, q.cuda(), cu.cuda(), mask.cuda(), 8, scale)
    d["lens"][1], d["lens"][3] = 4, cache.MB * 32 + 1
    out = run(cache, q.cuda(), cu.cuda(), mask.cuda(), 8, scale)
    assert pa.get_device_error() == 4
    d["lens"].copy_(good)
    c = cu.tolist()
    for s in range(5):
        a, b = out[c[s]:c[s + 1]], want[c[s]:c[s + 1]]
        assert (a == 0).all() if s in (1, 3) else torch.equal(a, b)
    # a draft longer than max_q_len, offsets past the batch: those rows are not written
    out = run(cache, q.cuda(), cu.cuda(), mask.cuda(), 7, scale)
    assert pa.get_device_error() == 16
    assert torch.equal(out[:c[4]], want[:c[4]]) and out[c[4]:].isnan().all()
    for bad in ([0, 4, 9, 15, 22, 31], [0, 4, 3, 15, 22, 30], [-1, 4, 9, 15, 22, 30]):
        run(cache, q.cuda(), torch.tensor(bad, dtype=torch.int32).cuda(), mask.cuda(), 8, scale)
        assert pa.get_device_error() == 16
    # a bad block id reads as zeros
    keep = d["tables"].clone()
    d["tables"][2, 1] = 10 ** 6
    d["tables"][0, 0] = -5
    out = run(cache, q.cuda(), cu.cuda(), mask.cuda(), 8, scale)
    assert pa.get_device_error() == 2 and not out.isnan().any()
    d["tables"].copy_(keep)
    assert torch.equal(out[c[1]:c[2]], want[c[1]:c[2]]) and torch.equal(out[c[3]:], want[c[3]:])


def test_same_bits_again_in_a_graph_and_on_two_streams():
    cache = Cache([700, 1500, 90], 2, 128, 32, seed=6)
    nodes, G = [40, 17, 3], 4
    q, cu, mask = inputs(cache, nodes, G, torch.bfloat16, 8)
    q, cu, mask = q.cuda(), cu.cuda(), mask.cuda()
    want = run(cache, q, cu, mask, 40, 0.1)
    ws = [torch.empty(pa.tree_workspace_size(8, 2, 128), dtype=torch.uint8, device="cuda")
          for _ in range(2)]
    outs = [torch.full_like(q, float("nan")) for _ in range(2)]
    st = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for i in range(2):
            run(cache, q, cu, mask, 40, 0.1, ws[i], outs[i], st[i])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
    graph = torch.cuda.CUDAGraph()
    outs[0].fill_(float("nan"))
    with torch.cuda.graph(graph):
        run(cache, q, cu, mask, 40, 0.1, ws[0], outs[0])
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want)
    # the captured call follows the inputs it reads
    q2 = q.flip(0).contiguous()
    q.copy_(q2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], run(cache, q2, cu, mask, 40, 0.1))
