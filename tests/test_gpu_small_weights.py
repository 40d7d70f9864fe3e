"""Trees whose products of weight and V are small (or large) beside f16's range:
row scales of an INT8 cache far from one, and a dominant token whose V is zero, so that the
output is made of the other tokens' small weights.

Bounds: tests/_ref64.py, but with what f16's smallest step costs in the output's own terms. The
products 2^(x - mu) vs (vs: the V row's scale, 1 for other caches) are rounded to f16: u(f16) of
their size, or 2^-25 where they are subnormal. mu is at most 7 below the largest logit plus the
exponent of the scales beside it, so one over the sum of 2^(x - mu) is at most 2^-7 p_max 2^E with
2^E <= 2 max vs (1 for other caches): 2^-32 p_max 2^E sum_j |code_j|, times v_scale for FP8. An f16
output has steps of 2^-24 at least: half of one."""
import numpy as np
import pytest
import torch

from _ref64 import U, Cache, attend, bits64, default_scale, weight_type
from paged_kv_cache_context_gb300 import pa
from test_gpu_tree import random_mask, run as run_tree

pytestmark = pytest.mark.gpu


def attend_sharp(cache, s, g, q, seen, out_dtype):
    """(output, bound, weights, their relative error), the bound relative to sum_j p_j |V_j|."""
    K, V, codes = cache.rows(s, g)
    w = weight_type(cache, out_dtype)
    o, _, p, rel = attend(q, K, V, codes, seen, default_scale(cache.D), out_dtype, w)
    if not seen.any():
        return o, np.full(cache.D, 1e-30), p, rel
    bound = (U[w] * 1.01 + rel) * (p @ np.abs(V)) + U[out_dtype] * 1.01 * np.abs(o)
    if w == torch.float16:
        unit = cache.v_scale
        if cache.kv == "int8":
            t = np.nonzero(seen)[0]
            blk, off = cache.tables[s].long()[t // cache.bs], t % cache.bs
            unit = 2 * float(cache.vs[blk, g, torch.from_numpy(off)].max())
        bound = bound + 1.01 * 2.0 ** -32 * p.max() * unit * np.abs(codes[seen]).sum(0)
    if out_dtype == torch.float16:
        bound = bound + 2.0 ** -25
    return o, bound + 1e-30, p, rel


def check_tree(cache, nodes, G, q, mask, out, heads=None):
    got, qd = out.double().cpu().numpy(), q.double().cpu().numpy()
    at = 0
    for s, t in enumerate(nodes):
        n = cache.lens[s]
        for i in range(t):
            seen = np.ones(n, dtype=bool)
            seen[n - t:] = bits64(mask[at + i].tolist(), t)
            for h in range(cache.H * G):
                if heads is not None and h // G not in heads:
                    continue
                o, bound, _, _ = attend_sharp(cache, s, h // G, qd[at + i, h], seen, q.dtype)
                err = np.abs(got[at + i, h] - o)
                assert (err <= bound).all(), (s, i, h, float((err / bound).max()))
        at += t


def scale_rows(cache, how, seed=0):
    """V row scales of an INT8 cache, by token: a factor, drawn over four decades, or growing and
    falling along the sequence."""
    g = torch.Generator().manual_seed(seed)
    for s, n in enumerate(cache.lens):
        t = torch.arange(n)
        if how == "mixed":
            f = 10.0 ** (-4 * torch.rand(n, generator=g))
        elif how == "growing":
            f = 2.0 ** (-20 + 24 * t / n)
        elif how == "falling":
            f = 2.0 ** (4 - 24 * t / n)
        else:
            f = torch.full((n,), float(how))
        blk, off = cache.tables[s].long()[t // cache.bs], t % cache.bs
        cache.vs[blk, :, off] *= f[:, None]


def add_sink(cache, b, gap):
    """Token n // 3 of every sequence gets a logit about `gap` above the others' (for queries near
    1.5 b) and V zero; the other logits are near zero and their V positive."""
    c = gap / (default_scale(cache.D) * 1.5 * cache.D)
    for s, n in enumerate(cache.lens):
        t = torch.arange(n)
        blk, off = cache.tables[s].long()[t // cache.bs], t % cache.bs
        at, o = int(cache.tables[s, n // 3 // cache.bs]), n // 3 % cache.bs
        if cache.kv == "int8":
            cache.v[blk, :, off] = cache.v[blk, :, off].abs()
            cache.ks[blk, :, off] *= 0.01
            cache.k[at, :, o] = (127 * b).to(torch.int8)
            cache.ks[at, :, o] = c / 127
            cache.v[at, :, o] = 0
        elif cache.kv == "fp8_e4m3":
            def code(x):
                return x.to(torch.float8_e4m3fn).view(torch.uint8)
            k = cache.k[blk, :, off].view(torch.float8_e4m3fn).float()
            cache.k[blk, :, off] = code(0.02 * k)
            cache.v[blk, :, off] &= 0x7F
            cache.k[at, :, o] = code(c / cache.k_scale * b)
            cache.v[at, :, o] = 0
        else:
            cache.k[blk, :, off] *= 0.02
            cache.v[blk, :, off] = cache.v[blk, :, off].abs()
            cache.k[at, :, o] = (c * b).to(cache.dtype)
            cache.v[at, :, o] = 0


def signs(D):
    return torch.randint(0, 2, (D,), generator=torch.Generator().manual_seed(D)).float() * 2 - 1


def tree_inputs(cache, nodes, G, dtype, base=None):
    g = torch.Generator().manual_seed(3)
    T = sum(nodes)
    q = torch.randn(T, cache.H * G, cache.D, generator=g)
    q = (1.5 * q if base is None else 1.5 * base + 0.1 * q).to(dtype)
    mask = random_mask(nodes, max(1, -(-max(nodes) // 64)), 5)
    return q, torch.tensor([0] + nodes).cumsum(0).int(), mask


TREES = [  # dtype, D, G, lens, nodes: one row tile of 128, and wide ones
    (torch.bfloat16, 128, 2, [1500, 200, 33], [7, 20, 1]),
    (torch.bfloat16, 64, 4, [900, 65], [5, 40]),
    (torch.float16, 128, 8, [1300, 140], [5, 20]),
]


@pytest.mark.parametrize("how", [1e7, 0.06, 1e-4, "mixed", "growing", "falling"])
@pytest.mark.parametrize("dtype,D,G,lens,nodes", TREES)
def test_tree_over_int8_rows_of_any_size(dtype, D, G, lens, nodes, how):
    if how == 1e7:
        dtype = torch.bfloat16  # (an f16 output does not hold such values)
    pa.get_device_error()
    cache = Cache(lens, 1, D, 32, "int8", dtype, seed=D)
    scale_rows(cache, how)
    q, cu, mask = tree_inputs(cache, nodes, G, dtype)
    out = run_tree(cache, q.cuda(), cu.cuda(), mask.cuda(), max(nodes), default_scale(D))
    assert pa.get_device_error() == 0
    check_tree(cache, nodes, G, q, mask, out)


@pytest.mark.parametrize("kv", ["auto", "fp8_e4m3", "int8"])
@pytest.mark.parametrize("dtype,D,G,lens,nodes", TREES)
def test_tree_keeps_small_weights_beside_a_dominant_one(dtype, D, G, lens, nodes, kv):
    pa.get_device_error()
    cache = Cache([2 * lens[0]] + lens[1:], 1, D, 32, kv, dtype, seed=D)
    add_sink(cache, signs(D), 15.0)
    q, cu, mask = tree_inputs(cache, nodes, G, dtype, signs(D))
    out = run_tree(cache, q.cuda(), cu.cuda(), mask.cuda(), max(nodes), default_scale(D))
    assert pa.get_device_error() == 0
    check_tree(cache, nodes, G, q, mask, out)


@pytest.mark.parametrize("how", ["growing", "falling"])
@pytest.mark.parametrize("dtype,D,G,top", [(torch.bfloat16, 128, 1, 5), (torch.float16, 64, 2, 5),
                                           (torch.bfloat16, 128, 8, 20)])
def test_tree_shares_of_many_tiles_whose_scales_differ(dtype, D, G, top, how):
    """A share is several tiles long: its reference moves with the scales inside it."""
    pa.get_device_error()
    lens = [40 + (977 * s) % (1460 if s % 3 == 0 else 300) for s in range(24)]
    nodes = [1 + s % top for s in range(24)]
    cache = Cache(lens, 8, D, 32, "int8", dtype, seed=D + G)
    scale_rows(cache, how)
    q, cu, mask = tree_inputs(cache, nodes, G, dtype)
    out = run_tree(cache, q.cuda(), cu.cuda(), mask.cuda(), max(nodes), default_scale(D))
    assert pa.get_device_error() == 0
    check_tree(cache, nodes, G, q, mask, out, heads=None if G == 1 else [0, 5])
