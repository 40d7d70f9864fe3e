"""Trees whose work just fills, just misses or just exceeds whole shares of the CTAs: every row
against attention in 64 bits on the GPU, so that a piece that the walk or the join misses, or
takes twice, shows. Bounds: tests/_ref64.py (bf16 caches)."""
import random

import pytest
import torch

from _ref64 import U, Cache, default_scale
from paged_kv_cache_context_gb300 import pa
from test_gpu_tree import pack, run

pytestmark = pytest.mark.gpu

D, BS = 64, 32


def batch(r, Hkv, G, wide, ctas):
    """(lens, nodes) with about a whole number of units a CTA, some drafts and sequences empty."""
    tokens, rows = (128, 256) if wide else (64, 128)
    want = ctas * r.choice([1, 1, 2, 3]) + r.choice([-1, 0, 1, 5])
    lens, nodes, units = [], [], 0
    while units < want and len(lens) < 90:
        if r.random() < 0.1:
            lens.append(r.choice([0, 50]))
            nodes.append(0)
            continue
        T = r.choice([1, 1, 2, 3, r.randint(1, 40)])
        t = r.randint(rows // G + 1, 2 * rows // G) if r.random() < 0.2 else r.randint(1, rows // G)
        n = max(t, tokens * (T - 1) + r.choice([1, 7, tokens - 1, tokens]))
        # (the last sequence ends where the shares do, as near as whole tiles allow)
        left = (want - units) // (Hkv * -(-t * G // rows))
        if left and -(-n // tokens) > left and tokens * left >= t:
            n = max(t, tokens * left - r.randint(0, tokens - 1))
        lens.append(n)
        nodes.append(t)
        units += -(-n // tokens) * -(-t * G // rows) * Hkv
    return lens, nodes


@pytest.mark.parametrize("seed", range(24))
def test_every_row_of_odd_shares(seed):
    r = random.Random(seed)
    wide = seed % 2 == 1
    Hkv, G = r.choice([1, 2, 8]), 8 if wide else r.choice([1, 2, 4])
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    lens, nodes = batch(r, Hkv, G, wide, sms if wide else min(2 * sms, 304))
    if not wide:  # (the batch's largest draft chooses the tiles: none above 128 rows)
        nodes = [min(t, 128 // G) for t in nodes]
    pa.get_device_error()
    cache = Cache(lens, Hkv, D, BS, "auto", torch.bfloat16, seed=seed)
    T, W = sum(nodes), -(-max(nodes) // 64)
    g = torch.Generator().manual_seed(seed)
    q = (1.5 * torch.randn(T, Hkv * G, D, generator=g)).bfloat16()
    bits = torch.rand(T, 64 * W, generator=g) < 0.5
    out = run(cache, q.cuda(), torch.tensor([0] + nodes).cumsum(0).int().cuda(),
              pack(bits.numpy()).cuda(), max(nodes), default_scale(D))
    assert pa.get_device_error() == 0
    d, scale, u = cache.dev(), default_scale(D), U[torch.bfloat16]
    at = 0
    for s, (n, t) in enumerate(zip(lens, nodes)):
        if t == 0:
            continue
        pages = d["tables"][s, : -(-n // BS)].long()
        K, V = (d[x][pages].transpose(1, 2).reshape(-1, Hkv, D)[:n].double() for x in ("k", "v"))
        seen = torch.ones(t, n, dtype=torch.bool, device="cuda")
        seen[:, n - t:] = bits[at: at + t, :t].cuda()
        x = q[at: at + t].cuda().double().view(t, Hkv, G, D)
        logits = torch.einsum("thgd,nhd->thgn", x, K) * scale
        size = torch.einsum("thgd,nhd->thgn", x.abs(), K.abs()).amax(-1, keepdim=True)
        p = logits.masked_fill(~seen[:, None, None], float("-inf")).softmax(-1).nan_to_num(0.0)
        o = torch.einsum("thgn,nhd->thgd", p, V)
        A = torch.einsum("thgn,nhd->thgd", p, V.abs())
        rel = 2 * (D + 8) * 2.0 ** -23 * scale * size + (n + 16) * 2.0 ** -23
        bound = (u * 1.01 + rel) * A + u * 1.01 * o.abs() + 1e-30
        err = (out[at: at + t].double().view(t, Hkv, G, D) - o).abs()
        assert (err <= bound).all(), (s, n, t, float((err / bound).max()))
        at += t
