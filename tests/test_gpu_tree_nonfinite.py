"""NaN in what a tree's row attends to reaches its output, whether the row's sequence lies in one
CTA's share or is cut and joined; NaN in K of unseen nodes, and in other rows' queries, does not."""
import pytest
import torch

from _ref64 import Cache, default_scale
from paged_kv_cache_context_gb300 import pa
from test_gpu_tree import run

pytestmark = pytest.mark.gpu

NAN = float("nan")
# kv, dtype, D, G: one row tile of 128 and (24 nodes, 8 heads) wide ones
KINDS = [("auto", torch.bfloat16, 128, 2), ("auto", torch.float16, 64, 8),
         ("fp8_e4m3", torch.bfloat16, 64, 2), ("fp8_e4m3", torch.bfloat16, 128, 8),
         ("int8", torch.float16, 128, 2), ("int8", torch.bfloat16, 64, 8)]
NODES = 24


def setup(kv, dtype, D, G, n):
    cache = Cache([n, 40], 1, D, 32, kv, dtype, seed=3)
    q = torch.randn(NODES + 4, G, D, generator=torch.Generator().manual_seed(1)).to(dtype)
    cu = torch.tensor([0, NODES, NODES + 4], dtype=torch.int32)
    mask = pa.tree_mask_from_parents(list(range(-1, NODES - 1)) + [-1] * 4, cu)
    return cache, q, cu, mask


def go(cache, q, cu, mask):
    return run(cache, q.cuda(), cu.cuda(), mask.cuda(), NODES, default_scale(cache.D))


def spoil(cache, name, t, d=slice(None)):
    """NaN in token t's row of sequence 0 (an INT8 row: in its scale)."""
    b, o = int(cache.tables[0, t // cache.bs]), t % cache.bs
    if cache.kv == "int8":
        getattr(cache, name + "s")[b, 0, o] = NAN
    elif cache.kv == "fp8_e4m3":
        getattr(cache, name)[b, 0, o, d] = 0x7F
    else:
        getattr(cache, name)[b, 0, o, d] = NAN


@pytest.mark.parametrize("n", [60, 9000])  # in one share; cut
@pytest.mark.parametrize("kv,dtype,D,G", KINDS)
def test_nan_of_a_seen_token_reaches_every_row_that_sees_it(kv, dtype, D, G, n):
    good = go(*setup(kv, dtype, D, G, n))
    for what in ("k", "v"):
        cache, q, cu, mask = setup(kv, dtype, D, G, n)
        spoil(cache, what, n // 2)  # of the context: every node sees it
        out = go(cache, q, cu, mask)
        assert out[:NODES].isnan().all(), what
        assert torch.equal(out[NODES:], good[NODES:])
    if kv != "int8":  # one element of V: one column of the output
        cache, q, cu, mask = setup(kv, dtype, D, G, n)
        spoil(cache, "v", n // 2, 5)
        out = go(cache, q, cu, mask)
        assert out[:NODES, :, 5].isnan().all()
        keep = [d for d in range(D) if d != 5]
        assert torch.equal(out[..., keep], good[..., keep])


@pytest.mark.parametrize("n", [60, 9000])
@pytest.mark.parametrize("kv,dtype,D,G", KINDS)
def test_nan_of_a_query_stays_in_its_row(kv, dtype, D, G, n):
    cache, q, cu, mask = setup(kv, dtype, D, G, n)
    good = go(cache, q, cu, mask)
    q[7, 1, 3] = NAN
    out = go(cache, q, cu, mask)
    assert out[7, 1].isnan().all()
    out[7, 1] = good[7, 1]
    assert torch.equal(out, good)


@pytest.mark.parametrize("n", [60, 9000])
@pytest.mark.parametrize("kv,dtype,D,G", KINDS)
def test_nan_in_k_of_unseen_nodes_changes_nothing(kv, dtype, D, G, n):
    """A chain: node i does not see the nodes after it."""
    good = go(*setup(kv, dtype, D, G, n))
    cache, q, cu, mask = setup(kv, dtype, D, G, n)
    spoil(cache, "k", n - 4)  # node NODES - 4
    out = go(cache, q, cu, mask)
    assert torch.equal(out[: NODES - 4], good[: NODES - 4])
    assert out[NODES - 4: NODES].isnan().all() and torch.equal(out[NODES:], good[NODES:])
