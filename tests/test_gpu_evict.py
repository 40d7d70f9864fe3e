"""pa_evict_select and pa_compact on the GPU: whole numbers and moved bits, compared exactly; and
the operators run together as a serving loop runs them."""
import numpy as np
import pytest
import torch

from _gpu import bits
from _ref64 import Cache, attend, default_scale, weight_type
from paged_kv_cache_context_gb300 import pa

pytestmark = pytest.mark.gpu


def choose(scores, n, B, sink, recent):
    """The kept positions, by the definition."""
    if n <= B:
        return list(range(n))
    forced = set(range(min(sink, n))) | set(range(n - recent, n))
    rest = [t for t in range(n) if t not in forced]
    val = [float("-inf") if x != x else x + 0.0 for x in scores]
    nan = [scores[t] != scores[t] for t in range(n)]
    rest.sort(key=lambda t: (nan[t], -val[t], t))
    return sorted(forced | set(rest[: B - len(forced)]))


def select(scores, lens, B, sink, recent, stream=None):
    S, H, _ = scores.shape
    keep = torch.full((S, H, B), -7, dtype=torch.int32, device="cuda")
    new = torch.full((S,), -7, dtype=torch.int32, device="cuda")
    pa.evict_select(keep, new, scores.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), sink,
                    recent, stream=stream)
    return keep, new


def check_select(scores, lens, B, sink, recent):
    keep, new = select(scores, lens, B, sink, recent)
    for s, n in enumerate(lens):
        assert int(new[s]) == min(n, B)
        for g in range(scores.shape[1]):
            want = choose(scores[s, g].tolist(), n, B, sink, recent)
            got = keep[s, g].tolist()
            assert got == want + [-1] * (B - len(want)), (s, g)


@pytest.mark.parametrize("N,lens,B,sink,recent", [
    (48, [0, 1, 31, 32, 33, 48], 32, 4, 8),
    (700, [700, 64, 65], 64, 0, 0),
    (700, [700], 1, 0, 0),
    (700, [700, 300], 64, 0, 64),      # nothing left to choose
    (700, [700, 300], 64, 30, 34),
    (4097, [4097, 4000], 1000, 4, 100),
    (33000, [33000, 257], 2047, 4, 512),   # past the registers of one block
    (20000, [19999], 19998, 1, 1),
])
def test_select_matches_the_definition(N, lens, B, sink, recent):
    pa.get_device_error()
    g = torch.Generator().manual_seed(N + B)
    scores = torch.exp(2 * torch.randn(len(lens), 2, N, generator=g) - 4)
    check_select(scores, lens, B, sink, recent)
    assert pa.get_device_error() == 0


def test_select_ties_signs_infinities_and_nan():
    N = 900
    g = torch.Generator().manual_seed(1)
    few = torch.randint(-3, 4, (1, 3, N), generator=g).float()       # many ties, both signs
    few[0, 1] = 0.5                                                  # all equal
    few[0, 2, ::3] = float("nan")
    few[0, 2, 1::5] = float("inf")
    few[0, 2, 2::7] = float("-inf")
    few[0, 0, 100:200] = -0.0
    few[0, 0, 150] = 0.0
    for B, sink, recent in ((100, 4, 10), (500, 0, 0), (850, 1, 1), (899, 0, 5)):
        check_select(few, [N], B, sink, recent)
    tiny = torch.full((1, 1, N), 1e-42)                              # subnormal
    tiny[0, 0, 700] = 1.1e-42
    check_select(tiny, [N], 5, 0, 0)


def test_select_ties_past_the_registers_of_one_block():
    """Equal scores spread over several rounds of a row: the first of them, counted across rounds."""
    N = 40003
    g = torch.Generator().manual_seed(2)
    few = torch.randint(0, 3, (1, 2, N), generator=g).float()
    few[0, 1] = 2.0
    for B, sink, recent in ((20000, 4, 100), (39000, 0, 0), (17, 1, 0)):
        check_select(few, [N], B, sink, recent)


def test_select_from_two_host_threads():
    """Rows of different lengths, which want different amounts of shared memory, at once."""
    import threading
    made, failed = {}, []
    for i, N in enumerate((9000, 50001, 30000)):
        g = torch.Generator().manual_seed(i)
        sc = torch.rand(1, 1, N, generator=g)
        made[N] = (sc.cuda(), torch.tensor([N], dtype=torch.int32).cuda(),
                   choose(sc[0, 0].tolist(), N, 500, 4, 50), torch.cuda.Stream())
    torch.cuda.synchronize()

    def work(N):
        sc, n, want, stream = made[N]
        try:
            for _ in range(100):
                keep = torch.empty(1, 1, 500, dtype=torch.int32, device="cuda")
                new = torch.empty(1, dtype=torch.int32, device="cuda")
                torch.cuda.current_stream().synchronize()
                pa.evict_select(keep, new, sc, n, 4, 50, stream=stream)
                stream.synchronize()
                if keep[0, 0].tolist() != want:
                    failed.append((N, "other tokens"))
        except Exception as e:  # reported by the main thread
            failed.append((N, repr(e)))

    threads = [threading.Thread(target=work, args=(N,)) for N in made]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed[:3]


def test_select_clamps_bad_lengths():
    pa.get_device_error()
    scores = torch.rand(2, 1, 64)
    keep, new = select(scores, [-4, 65], 16, 0, 4)
    assert pa.get_device_error() == 4
    assert new.tolist() == [0, 16] and keep[0].eq(-1).all()
    assert keep[1, 0].tolist() == choose(scores[1, 0].tolist(), 64, 16, 0, 4)


def moved(cache, keep, keep_lens, starts, scores, skip=()):
    """What compact leaves, by the definition (entries of `skip` are not moved)."""
    got = {x: getattr(cache, x).clone() for x in ("k", "v", "ks", "vs") if getattr(cache, x) is not None}
    was = {x: t.clone() for x, t in got.items()}
    sc = None if scores is None else scores.clone()
    for s, n in enumerate(cache.lens):
        a = starts[s] if starts is not None else 0
        for g in range(cache.H):
            row = keep[s, g if keep.shape[1] > 1 else 0].tolist()
            for j in range(keep_lens[s]):
                if (s, j) in skip:
                    continue
                f, t = row[j], a + j
                bf, bt = int(cache.tables[s, f // cache.bs]), int(cache.tables[s, t // cache.bs])
                for x in got:
                    got[x][bt, g, t % cache.bs] = was[x][bf, g, f % cache.bs]
                if sc is not None:
                    sc[s, g, t] = scores[s, g, f]
            if sc is not None:
                sc[s, g, a + keep_lens[s]:n] = 0
    return got, sc


def compact(cache, keep, keep_lens, starts, scores):
    d = {x: t.clone() for x, t in cache.dev().items()}
    sc = None if scores is None else scores.cuda()
    pa.compact(d["k"], d["v"], d["tables"], d["lens"], keep.cuda(),
               torch.tensor(keep_lens, dtype=torch.int32).cuda(),
               starts=None if starts is None else torch.tensor(starts, dtype=torch.int32).cuda(),
               k_scales=d.get("ks"), v_scales=d.get("vs"), scores=sc)
    return d, sc


def ascending(lens, H, B, kept, starts, seed):
    r = np.random.RandomState(seed)
    keep = np.full((len(lens), H, B), -1, dtype=np.int32)
    for s, n in enumerate(lens):
        a = starts[s] if starts is not None else 0
        for g in range(H):
            keep[s, g, :kept[s]] = a + np.sort(r.choice(n - a, kept[s], replace=False))
    return torch.from_numpy(keep)


@pytest.mark.parametrize("kv,dtype,D,H,bs,lens,B,heads,from_start,with_scores", [
    ("auto", torch.bfloat16, 128, 2, 32, [500, 64, 1, 0], 200, 2, False, True),
    ("auto", torch.float32, 64, 3, 16, [100, 33], 40, 3, False, False),
    ("auto", torch.float16, 96, 1, 64, [300], 299, 1, False, True),
    ("auto", torch.float32, 128, 2, 32, [70, 90], 9, 1, True, False),
    ("fp8_e4m3", torch.bfloat16, 96, 2, 16, [257, 40], 30, 2, False, True),
    ("int8", torch.bfloat16, 128, 2, 32, [300, 31, 200], 120, 2, False, True),
    ("int8", torch.float16, 64, 2, 64, [130, 80], 8, 1, True, True),
    ("auto", torch.bfloat16, 128, 1, 32, [5000], 3001, 1, False, True),
])
def test_compact_moves_the_kept_rows(kv, dtype, D, H, bs, lens, B, heads, from_start, with_scores):
    pa.get_device_error()
    cache = Cache(lens, H, D, bs, kv, dtype, seed=2)
    starts = [n - min(n, 20) for n in lens] if from_start else None
    room = [n - (starts[s] if starts else 0) for s, n in enumerate(lens)]
    kept = [min(B, r) if s % 2 == 0 else min(B, r) // 2 for s, r in enumerate(room)]
    keep = ascending(lens, heads, B, kept, starts, 5)
    scores = torch.rand(len(lens), H, cache.MB * bs) if with_scores else None
    want, want_s = moved(cache, keep, kept, starts, scores)
    got, got_s = compact(cache, keep, kept, starts, scores)
    assert pa.get_device_error() == 0
    for x in want:
        assert torch.equal(bits(got[x]), bits(want[x])), x
    if with_scores:
        assert torch.equal(got_s.cpu(), want_s)


@pytest.mark.parametrize("dtype,D,bs", [(torch.bfloat16, 8, 24), (torch.float32, 256, 1),
                                         (torch.float16, 40, 100)])
def test_compact_of_other_page_and_row_sizes(dtype, D, bs):
    """The moves read no page structure: any block size and whole 16-byte pieces of a row."""
    pa.get_device_error()
    cache = Cache([130, 700, 1], 3, D, bs, "auto", dtype, seed=6)
    kept = [100, 600, 1]
    keep = ascending(cache.lens, 3, 600, kept, None, 9)
    scores = torch.rand(3, 3, cache.MB * bs)
    want, want_s = moved(cache, keep, kept, None, scores)
    got, got_s = compact(cache, keep, kept, None, scores)
    assert pa.get_device_error() == 0
    assert torch.equal(bits(got["k"]), bits(want["k"])) and torch.equal(bits(got["v"]), bits(want["v"]))
    assert torch.equal(got_s.cpu(), want_s)


def test_compact_takes_any_source_at_or_after_its_place():
    """The same source twice and sources out of order: as if all were read first."""
    cache = Cache([64], 2, 128, 32, seed=8)
    keep = torch.tensor([[[9, 9, 40, 3, 63, 5, 30]] * 2], dtype=torch.int32)
    scores = torch.rand(1, 2, 64)
    want, want_s = moved(cache, keep, [7], None, scores)
    got, got_s = compact(cache, keep, [7], None, scores)
    assert torch.equal(bits(got["k"]), bits(want["k"])) and torch.equal(bits(got["v"]), bits(want["v"]))
    assert torch.equal(got_s.cpu(), want_s)


def test_compact_flags_bad_entries_lengths_and_blocks():
    cache = Cache([64, 64, 64], 1, 64, 32, seed=8)
    keep = ascending([64] * 3, 1, 10, [10] * 3, None, 3)
    keep[0, 0, 4] = 64       # past the sequence
    keep[1, 0, 6] = 5        # before its place
    pa.get_device_error()
    want, _ = moved(cache, keep, [10] * 3, None, None, skip={(0, 4), (1, 6)})
    got, _ = compact(cache, keep, [10] * 3, None, None)
    assert pa.get_device_error() == 1
    assert torch.equal(bits(got["k"]), bits(want["k"]))
    keep = ascending([64] * 3, 1, 10, [10] * 3, None, 3)
    for kept, starts in (([10, 11, 10], None), ([10, -1, 10], None), ([10] * 3, [0, 55, 0]),
                         ([10] * 3, [0, -1, 0])):
        got, _ = compact(cache, keep, kept, starts, None)
        assert pa.get_device_error() == 4
        want, _ = moved(cache, keep, [10, 0, 10], None, None)
        assert torch.equal(bits(got["k"]), bits(want["k"]))
    d = cache.dev()
    d["tables"][2, 0] = 999
    got, _ = compact(cache, keep, [10] * 3, None, None)
    assert pa.get_device_error() == 2
    d["tables"].copy_(cache.tables)


@pytest.mark.parametrize("kv", ["auto", "int8"])
def test_a_serving_loop_decodes_evicts_and_goes_on(kv):
    """Five scored steps, an eviction to 48 tokens, five more on the thinned cache."""
    lens, H, G, D, bs, B = [100, 40, 61], 2, 4, 128, 32, 48
    cache = Cache(lens, H, D, bs, kv, torch.bfloat16, seed=12, extra_tokens=16)
    d = cache.dev()
    S, N = 3, cache.MB * bs
    scores = torch.zeros(S, H, N, device="cuda")
    ws = torch.empty(pa.decode_scored_workspace_size(S, H * G, H, D, bs, cache.MB),
                     dtype=torch.uint8, device="cuda")
    g = torch.Generator().manual_seed(4)
    pa.get_device_error()

    def step():
        new = torch.randn(2, S, H, D, generator=g).bfloat16().cuda()
        q = torch.randn(S, H * G, D, generator=g).bfloat16()
        slot = torch.empty(S, dtype=torch.int64, device="cuda")
        pa.slot_mapping(slot, d["tables"], None, d["lens"], bs)
        d["lens"] += 1
        cache.lens = d["lens"].tolist()
        out = torch.empty(S, H * G, D, dtype=torch.bfloat16, device="cuda")
        if kv == "int8":
            pa.reshape_and_cache_int8(new[0], new[1], d["k"], d["v"], d["ks"], d["vs"], slot)
            pa.decode_scored_int8(out, scores, q.cuda(), d["k"], d["v"], d["ks"], d["vs"],
                                  d["tables"], d["lens"], H, default_scale(D), ws)
        else:
            pa.reshape_and_cache(new[0], new[1], d["k"], d["v"], slot)
            pa.decode_scored(out, scores, q.cuda(), d["k"], d["v"], d["tables"], d["lens"], H,
                             default_scale(D), ws)
        for x in ("k", "v", "ks", "vs"):
            if x in d:
                setattr(cache, x, d[x].cpu())
        added = np.zeros((S, H, N))
        for s in range(S):
            for h in range(H * G):
                K, V, codes = cache.rows(s, h // G)
                n = cache.lens[s]
                o, bound, p, _ = attend(q[s, h].double().numpy(), K, V, codes, np.ones(n, bool),
                                        default_scale(D), torch.bfloat16,
                                        weight_type(cache, torch.bfloat16))
                assert (np.abs(out[s, h].double().cpu().numpy() - o) <= bound).all()
                added[s, h // G, :n] += p
        return added

    want = np.zeros((S, H, N))
    for _ in range(5):
        want += step()
    # logits of at most a few tens: each weight within (2 * 136 * |x| + L + 16) 2^-23, five sums
    assert np.abs(scores.cpu().double().numpy() - want).max() <= 5 * G * 2.0 ** -23 * 20000
    keep = torch.empty(S, H, B, dtype=torch.int32, device="cuda")
    new_lens = torch.empty(S, dtype=torch.int32, device="cuda")
    pa.evict_select(keep, new_lens, scores, d["lens"], num_sink=2, num_recent=8)
    before = scores.cpu()
    for s in range(S):
        for h in range(H):
            ref = choose(before[s, h].tolist(), cache.lens[s], B, 2, 8)
            assert keep[s, h, : len(ref)].tolist() == ref
    ref_cache, ref_scores = moved(cache, keep.cpu(), new_lens.tolist(), None, before)
    pa.compact(d["k"], d["v"], d["tables"], d["lens"], keep, new_lens, k_scales=d.get("ks"),
               v_scales=d.get("vs"), scores=scores)
    for x in ref_cache:
        assert torch.equal(bits(d[x]), bits(ref_cache[x]))
    assert torch.equal(scores.cpu(), ref_scores)
    d["lens"].copy_(new_lens)
    for _ in range(5):
        step()
    assert pa.get_device_error() == 0


def test_a_draft_is_verified_and_its_path_kept():
    """Tree attention over a draft, the accepted path's rows moved, then a decode that reads them."""
    ctx, nodes, H, G, D, bs = [90, 33], [6, 4], 2, 4, 128, 32
    lens = [c + t for c, t in zip(ctx, nodes)]
    cache = Cache(lens, H, D, bs, "auto", torch.bfloat16, seed=14, extra_tokens=4)
    d = cache.dev()
    cu = torch.tensor([0, 6, 10], dtype=torch.int32)
    mask = pa.tree_mask_from_parents([-1, 0, 0, 2, 2, 4, -1, -1, 1, 2], cu)
    g = torch.Generator().manual_seed(4)
    q = torch.randn(10, H * G, D, generator=g).bfloat16()
    ws = torch.empty(pa.tree_workspace_size(H * G, H, D), dtype=torch.uint8, device="cuda")
    out = torch.empty(10, H * G, D, dtype=torch.bfloat16, device="cuda")
    pa.get_device_error()
    pa.tree_attention(out, q.cuda(), d["k"], d["v"], d["tables"], cu.cuda(), d["lens"],
                      mask.cuda(), H, 6, default_scale(D), ws)
    paths = [[0, 2, 4, 5], [1, 2]]  # accepted nodes
    # the last accepted node saw its path and the context alone: the same as a decode of
    # the sequence that ends with it, once the path's rows are moved together
    keep = torch.full((2, 1, 4), -1, dtype=torch.int32)
    for s, path in enumerate(paths):
        keep[s, 0, : len(path)] = torch.tensor([ctx[s] + i for i in path])
    kept = torch.tensor([4, 2], dtype=torch.int32).cuda()
    starts = torch.tensor(ctx, dtype=torch.int32).cuda()
    pa.compact(d["k"], d["v"], d["tables"], d["lens"], keep.cuda(), kept, starts=starts)
    lens_now = starts + kept
    last = [5, 6 + 2]
    qd = q[last].cuda().contiguous()
    one = torch.empty(2, H * G, D, dtype=torch.bfloat16, device="cuda")
    pa.decode(one, qd, d["k"], d["v"], d["tables"], lens_now, H, default_scale(D))
    assert pa.get_device_error() == 0
    cache.k, cache.v = d["k"].cpu(), d["v"].cpu()
    for s in range(2):
        for h in range(H * G):
            n = int(lens_now[s])
            K, V, codes = cache.rows(s, h // G, n)
            o, bound, _, _ = attend(qd[s, h].double().cpu().numpy(), K, V, codes,
                                    np.ones(n, bool), default_scale(D), torch.bfloat16,
                                    torch.bfloat16)
            for x in (out[last[s], h], one[s, h]):
                assert (np.abs(x.double().cpu().numpy() - o) <= bound).all()
