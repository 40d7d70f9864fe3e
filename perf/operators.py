"""The multi-token and cache-thinning operators of the paged cache, as cases to measure.

Four operators over caches [num_blocks, num_kv_heads, block_size, head_dim] reached through
block tables:

  tree      attention of a tree of drafted tokens: node i of a sequence attends to its whole
            context and to the nodes that its mask names (its ancestors and itself)
  scored    decode attention that also adds each cached token's softmax weight, summed over the
            query heads of its kv head, to a running score
  select    the tokens an eviction keeps: the first ones, the last ones and the best scored
  compact   the kept tokens' rows moved to the front of their sequence, in place (after an
            eviction per kv head, or after a verification the accepted path of a tree)

``own`` chooses between the plain form in elementary torch operations and the calls of
``paged_kv_cache_context_gb300.pa``.
"""
import math

import torch

own = False

GOLD = 0.6180339887498949
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one user's draft of 8 nodes on a short chat: what counts is the latency of the call
        dict(name="tree_one", op="tree", kv="auto", dtype="bf16", seqs=1, heads=32, kv_heads=8,
             dim=128, bs=32, lo=500, hi=500, nodes_lo=8, nodes_hi=8),
        # a batch of chats (the decode workload's lengths) with ragged drafts of 16 to 32 nodes
        dict(name="tree_chat", op="tree", kv="auto", dtype="bf16", seqs=32, heads=32, kv_heads=8,
             dim=128, bs=32, lo=512, hi=4096, nodes_lo=16, nodes_hi=32),
        # few long documents with wide drafts: more rows than one tensor-core tile
        dict(name="tree_long", op="tree", kv="auto", dtype="f16", seqs=4, heads=32, kv_heads=8,
             dim=128, bs=32, lo=9001, hi=32768, nodes_lo=47, nodes_hi=96),
        # an FP8 cache with one query head per kv head
        dict(name="tree_fp8", op="tree", kv="fp8", dtype="bf16", seqs=16, heads=32, kv_heads=32,
             dim=128, bs=32, lo=1024, hi=8192, nodes_lo=13, nodes_hi=61),
        # the smallest decode: two short sequences in 32 bits
        dict(name="scored_tiny", op="scored", kv="auto", dtype="f32", seqs=2, heads=4, kv_heads=4,
             dim=64, bs=32, lo=17, hi=45),
        # the decode workload of a batch of chats, with scores
        dict(name="scored_chat", op="scored", kv="auto", dtype="bf16", seqs=32, heads=32,
             kv_heads=8, dim=128, bs=32, lo=512, hi=4096),
        # the largest decode: 64 sequences over an FP8 cache, head_dim 96
        dict(name="scored_fp8", op="scored", kv="fp8", dtype="bf16", seqs=64, heads=32,
             kv_heads=32, dim=96, bs=32, lo=1024, hi=8192),
        # one sequence's eviction down to 256 tokens
        dict(name="select_one", op="select", seqs=1, kv_heads=8, bs=32, lo=700, hi=700, budget=256,
             sink=4, recent=64),
        # a batch of long sequences evicted down to 2048 tokens
        dict(name="select_long", op="select", seqs=16, kv_heads=8, bs=32, lo=3001, hi=32768,
             budget=2048, sink=4, recent=512),
        # the rows of a batch of chats after an eviction to 1024 tokens
        dict(name="compact_chat", op="compact", kv="auto", dtype="bf16", seqs=32, kv_heads=8,
             dim=128, bs=32, lo=512, hi=4096, budget=1024, sink=4, recent=256, scores=True),
        # the accepted paths (1 to 8 nodes of 32) of a batch's verified drafts
        dict(name="compact_path", op="commit", kv="auto", dtype="bf16", seqs=32, kv_heads=8,
             dim=128, bs=32, lo=512, hi=4096, nodes=32, budget=8),
        # an INT8 cache of long sequences: codes, row scales and scores move together
        dict(name="compact_int8", op="compact", kv="int8", dtype="bf16", seqs=16, kv_heads=8,
             dim=128, bs=32, lo=3001, hi=32768, budget=4096, sink=4, recent=512, scores=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "scored", "scored", "select", "compact", "commit"])
    c = dict(op=op, seqs=_log_int(rng, 1, 64), kv_heads=rng.choice([1, 2, 4, 8, 8, 32]),
             bs=rng.choice([16, 32, 32, 64]))
    if op == "select":
        c["hi"] = _log_int(rng, 2, 32768)
        c["lo"] = max(1, int(c["hi"] * rng.uniform(0.1, 1.0)))
        c["budget"] = max(1, int(c["hi"] * rng.uniform(0.05, 1.1)))
        c["sink"] = min(c["budget"], rng.choice([0, 1, 4]))
        c["recent"] = int((c["budget"] - c["sink"]) * rng.uniform(0.0, 0.6))
        return c
    c["kv"] = rng.choice(["auto", "auto", "fp8", "int8"])
    dims = [64, 128] if op == "tree" else [64, 96, 128]
    c["dim"] = rng.choice(dims)
    c["dtype"] = rng.choice(["bf16", "f16"] if op == "tree" or c["kv"] == "int8" else
                            ["bf16", "f16", "f32"])
    group = rng.choice([1, 2, 4, 4, 8, 3])
    if op in ("tree", "scored"):
        c["heads"] = c["kv_heads"] * group
    # at most about 400 MB of 16-bit keys and values in the batch
    most = max(64, int(4e8 / (c["seqs"] * c["kv_heads"] * c["dim"] * 4)))
    c["hi"] = _log_int(rng, 40, min(32768, most) if most > 40 else 41)
    c["lo"] = max(33, int(c["hi"] * rng.uniform(0.2, 1.0)))
    c["hi"] = max(c["hi"], c["lo"])
    if op == "tree":
        top = min(128, max(1, c["hi"] // 2), c["lo"])
        c["nodes_hi"] = _log_int(rng, 1, top) if top > 1 else 1
        c["nodes_lo"] = max(1, int(c["nodes_hi"] * rng.uniform(0.3, 1.0)))
    elif op == "compact":
        c["budget"] = max(1, int(c["lo"] * rng.uniform(0.1, 1.0)))
        c["sink"] = min(c["budget"], rng.choice([0, 1, 4]))
        c["recent"] = int((c["budget"] - c["sink"]) * rng.uniform(0.0, 0.6))
        c["scores"] = rng.random() < 0.7
    elif op == "commit":
        c["nodes"] = rng.randint(1, 32)
        c["budget"] = rng.randint(1, c["nodes"])
    return c


def _spread(lo, hi, n, phase=0.0):
    """n whole numbers over [lo, hi], the same for every seed."""
    return [lo + int(((i + 1) * GOLD + phase) % 1.0 * (hi - lo + 1)) for i in range(n)]


def _lens(case):
    return _spread(case["lo"], case["hi"], case["seqs"])


def _nodes(case):
    return _spread(case["nodes_lo"], case["nodes_hi"], case["seqs"], 0.37)


def _keeps(case):
    return [min(n, case["budget"]) for n in _lens(case)]


def _paths(case):
    return _spread(1, case["budget"], case["seqs"], 0.71)


def _elem(case):
    return {"fp8": 1, "int8": 1}.get(case["kv"]) or (4 if case["dtype"] == "f32" else 2)


def work(case):
    op, lens = case["op"], _lens(case)
    if op == "select":
        cells = sum(lens) * case["kv_heads"]
        kept = sum(_keeps(case)) * case["kv_heads"]
        return {"bytes": 4 * (cells + kept + 2 * case["seqs"]), "flops": 0}
    H, D = case["kv_heads"], case["dim"]
    row = D * _elem(case) + (4 if case["kv"] == "int8" else 0)
    table = 4 * sum(-(-n // case["bs"]) for n in lens) + 4 * case["seqs"]
    if op in ("tree", "scored"):
        rows = _nodes(case) if op == "tree" else [1] * case["seqs"]
        q = sum(rows) * case["heads"] * D * (4 if case["dtype"] == "f32" else 2)
        pairs = sum(t * n - (t * (t - 1) // 2 if op == "tree" else 0) for t, n in zip(rows, lens))
        b = sum(lens) * H * 2 * row + 2 * q + table
        b += 8 * sum(lens) * H if op == "scored" else 8 * sum(rows)
        return {"bytes": b, "flops": 4 * pairs * case["heads"] * D}
    if op == "compact":
        moved = sum(k - case["sink"] for k, n in zip(_keeps(case), lens) if n > k) * H
        moved_s = moved * 8 + 4 * sum(n - k for k, n in zip(_keeps(case), lens)) * H
        b = moved * 4 * row + (moved_s if case["scores"] else 0) + 4 * sum(_keeps(case)) * H
        return {"bytes": b + table, "flops": 0}
    # about half of an accepted path's nodes are not in their place already
    moved = sum(_paths(case)) * H // 2
    return {"bytes": moved * 4 * row + 4 * sum(_paths(case)) + 8 * case["seqs"], "flops": 0}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = dict(device="cuda")
    op, S, bs = case["op"], case["seqs"], case["bs"]
    lens = _lens(case)
    MB = max(-(-n // bs) for n in lens)
    st = dict(case=case, lens=torch.tensor(lens, dtype=torch.int32, **dev))

    def randn(*shape):
        return torch.randn(*shape, generator=g, dtype=torch.float32, **dev)

    def kept(H, cap):
        """H ascending choices of cap[s] tokens a sequence, the first and the last among them."""
        n = st["lens"].long()[:, None, None]
        at = torch.arange(MB * bs, **dev)[None, None, :]
        pick = torch.rand(S, H, MB * bs, generator=g, **dev)
        pick = torch.where((at < case["sink"]) | (at >= n - case["recent"]), 2.0, pick)
        pick = torch.where(at < n, pick, -1.0)
        order = pick.argsort(dim=-1, descending=True)[..., : case["budget"]]
        spot = torch.arange(case["budget"], **dev)[None, None, :]
        order = torch.where(spot < cap[:, None, None], order, MB * bs)
        order = order.sort(dim=-1).values
        return torch.where(spot < cap[:, None, None], order, -1).int().contiguous()

    if op == "select":
        # what attention weights add up to over a few hundred steps: a heavy tail
        sc = torch.exp(2.0 * randn(S, case["kv_heads"], MB * bs) - 4.0)
        st["scores"] = sc
        st["keep"] = torch.empty(S, case["kv_heads"], case["budget"], dtype=torch.int32, **dev)
        st["new_lens"] = torch.empty(S, dtype=torch.int32, **dev)
        return st

    H, D, dt = case["kv_heads"], case["dim"], DT[case["dtype"]]
    own_pages = [-(-n // bs) for n in lens]
    NB = sum(own_pages) + 3
    perm = torch.randperm(NB, generator=g, **dev).int()
    first = torch.tensor([sum(own_pages[:s]) for s in range(S)], **dev)[:, None]
    page = torch.arange(MB, **dev)[None, :]
    has = page < torch.tensor(own_pages, **dev)[:, None]
    st["tables"] = torch.where(has, perm[(first + page).clamp(max=NB - 1)], -1).int().contiguous()
    st["k_scale"] = st["v_scale"] = 1.0
    if case["kv"] == "fp8":
        st["k_scale"], st["v_scale"] = 1.0 / 64, 1.0 / 96
        k = randn(NB, H, bs, D).mul_(64.0).clamp_(-448, 448)
        k = k.to(torch.float8_e4m3fn).view(torch.uint8)
        v = randn(NB, H, bs, D).mul_(96.0).clamp_(-448, 448)
        v = v.to(torch.float8_e4m3fn).view(torch.uint8)
    elif case["kv"] == "int8":
        k = torch.randint(-127, 128, (NB, H, bs, D), generator=g, dtype=torch.int8, **dev)
        v = torch.randint(-127, 128, (NB, H, bs, D), generator=g, dtype=torch.int8, **dev)
        st["k_scales"] = (0.5 + torch.rand(NB, H, bs, generator=g, **dev)) * (1.7 / 127)
        st["v_scales"] = (0.5 + torch.rand(NB, H, bs, generator=g, **dev)) * (1.7 / 127)
    else:
        k, v = randn(NB, H, bs, D).to(dt), randn(NB, H, bs, D).to(dt)
    st["k"], st["v"] = k, v
    st["scale"] = 1.0 / math.sqrt(D)

    if op == "tree":
        nodes = _nodes(case)
        N = max(nodes)
        cu = torch.tensor([0] + nodes).cumsum(0)
        # a random tree each: a node's parent is one of the few before it, or the context's end
        back = torch.randint(1, 6, (S, N), generator=g, **dev).cpu()
        par = torch.arange(N)[None, :] - back
        see = torch.zeros(S, N, N, dtype=torch.bool)
        for i in range(N):
            p = par[:, i]
            see[:, i] = see[torch.arange(S), p.clamp(min=0)] & (p >= 0)[:, None]
            see[:, i, i] = True
        W = -(-N // 64)
        word = torch.zeros(S, N, W * 64, dtype=torch.int64)
        word[:, :, :N] = see.long()
        word = (word.view(S, N, W, 64) << torch.arange(64)).sum(-1)  # wraps into the sign bit
        live = torch.arange(N)[None, :] < torch.tensor(nodes)[:, None]
        st["mask"] = word[live].contiguous().cuda()
        st["cu"] = cu.int().cuda()
        st["live"], st["max_nodes"] = live.cuda(), N
        st["q"] = (2.0 * randn(sum(nodes), case["heads"], D)).to(dt)
        st["out"] = torch.empty_like(st["q"])
    elif op == "scored":
        st["q"] = (2.0 * randn(S, case["heads"], D)).to(dt)
        st["out"] = torch.empty_like(st["q"])
        at = torch.arange(MB * bs, **dev)[None, None, :]
        old = torch.exp(randn(S, H, MB * bs) - 2.0)
        st["scores"] = torch.where(at < st["lens"][:, None, None] - 1, old, 0.0).contiguous()
    elif op == "compact":
        st["keep_lens"] = torch.tensor(_keeps(case), dtype=torch.int32, **dev)
        st["keep"] = kept(H, st["keep_lens"])
        st["starts"] = None
        if case["scores"]:
            at = torch.arange(MB * bs, **dev)[None, None, :]
            old = torch.exp(randn(S, H, MB * bs) - 2.0)
            st["scores"] = torch.where(at < st["lens"][:, None, None], old, 0.0).contiguous()
    else:  # commit: the last `nodes` tokens are a draft, of which a path is kept
        st["keep_lens"] = torch.tensor(_paths(case), dtype=torch.int32, **dev)
        st["starts"] = st["lens"] - case["nodes"]
        gap = torch.rand(S, case["nodes"], generator=g, **dev)
        order = gap.argsort(dim=-1)[:, : case["budget"]]
        spot = torch.arange(case["budget"], **dev)[None, :]
        order = torch.where(spot < st["keep_lens"][:, None], order, case["nodes"]).sort(-1).values
        keep = torch.where(spot < st["keep_lens"][:, None], order + st["starts"][:, None], -1)
        st["keep"] = keep.int()[:, None, :].contiguous()
    return st


# ------------------------------------------------------------------ plain forms
def _rows_of(st, cache, scales, scale):
    """[S, H, MB * bs, D] in 32 bits: every table's pages in order."""
    if cache.dtype == torch.uint8:
        cache = cache.view(torch.float8_e4m3fn)
    S, MB = st["tables"].shape
    _, H, bs, D = cache.shape
    at = st["tables"].long().clamp(min=0)
    x = cache[at].float() if cache.dtype != torch.float8_e4m3fn else \
        cache.view(torch.uint8)[at].view(torch.float8_e4m3fn).float()
    if scales is not None:
        x = x * scales[at][..., None]
    elif scale != 1.0:
        x = x * scale
    return x.permute(0, 2, 1, 3, 4).reshape(S, H, MB * bs, D)


def _attend(q, k, v, see, scale):
    """Softmax attention of q [S, H, R, D]; see [S, 1, R, L] or [S, 1, 1, L]: also the weights."""
    x = (q.float() @ k.transpose(-1, -2)) * scale
    x = x.masked_fill(~see, -math.inf)
    top = x.amax(-1, keepdim=True)
    e = (x - torch.where(top == -math.inf, 0.0, top)).exp()
    total = e.sum(-1, keepdim=True)
    p = e / torch.where(total == 0, 1.0, total)
    return p @ v, p


def _plain_tree(st):
    case = st["case"]
    S, N = st["live"].shape
    H, G, D = case["kv_heads"], case["heads"] // case["kv_heads"], case["dim"]
    k = _rows_of(st, st["k"], st.get("k_scales"), st["k_scale"])
    v = _rows_of(st, st["v"], st.get("v_scales"), st["v_scale"])
    spot = (st["cu"][:-1, None] + torch.arange(N, device="cuda")).clamp(max=st["q"].shape[0] - 1)
    q = st["q"][spot].view(S, N, H, G, D).permute(0, 2, 1, 3, 4).reshape(S, H, N * G, D)
    n = st["lens"].long()[:, None, None]
    nodes = (st["cu"][1:] - st["cu"][:-1]).long()[:, None, None]
    at = torch.arange(k.shape[2], device="cuda")[None, None, :]
    node = at - (n - nodes)  # the node that a column holds; below 0: context
    bit = node.clamp(0, st["mask"].shape[1] * 64 - 1).expand(S, N, -1)
    word = st["mask"][spot].gather(2, bit >> 6)
    see = (node < 0) | (((word >> (bit & 63)) & 1 == 1) & (at < n))
    see = see[:, None, :, None, :].expand(S, 1, N, G, -1).reshape(S, 1, N * G, -1)
    o, _ = _attend(q, k, v, see, st["scale"])
    o = o.view(S, H, N, G, D).permute(0, 2, 1, 3, 4).reshape(S, N, H * G, D)
    return o[st["live"]].to(st["q"].dtype)


def _plain_scored(st):
    case = st["case"]
    S, H, G, D = case["seqs"], case["kv_heads"], case["heads"] // case["kv_heads"], case["dim"]
    k = _rows_of(st, st["k"], st.get("k_scales"), st["k_scale"])
    v = _rows_of(st, st["v"], st.get("v_scales"), st["v_scale"])
    see = torch.arange(k.shape[2], device="cuda")[None, :] < st["lens"][:, None]
    o, p = _attend(st["q"].view(S, H, G, D), k, v, see[:, None, None, :], st["scale"])
    st["scores"].add_(p.sum(2))
    return o.reshape(S, H * G, D).to(st["q"].dtype), st["scores"]


def _plain_select(st):
    case, sc = st["case"], st["scores"]
    n = st["lens"].long()[:, None, None]
    at = torch.arange(sc.shape[2], device="cuda")[None, None, :]
    rank = torch.where((at < case["sink"]) | (at >= n - case["recent"]), math.inf, sc)
    rank = torch.where(at < n, rank, -math.inf)
    B = case["budget"]
    order = rank.sort(dim=-1, descending=True, stable=True).indices[..., :B]
    order = torch.nn.functional.pad(order, (0, B - order.shape[-1]), value=sc.shape[2])
    spot = torch.arange(B, device="cuda")[None, None, :]
    kept = n.clamp(max=B)
    order = torch.where(spot < kept, order, sc.shape[2]).sort(dim=-1).values
    return torch.where(spot < kept, order, -1).int(), kept.view(-1).int()


def _plain_compact(st):
    k, v, keep = st["k"], st["v"], st["keep"].long()
    NB, H, bs, D = k.shape
    S, _, B = keep.shape
    keep = keep.expand(S, H, B)
    spot = torch.arange(B, device="cuda")[None, None, :]
    start = 0 if st["starts"] is None else st["starts"].long()[:, None, None]
    used = spot < st["keep_lens"][:, None, None]
    # an unused entry moves a row of its sequence onto itself
    to = torch.minimum((start + spot).expand(S, H, B), st["lens"].long()[:, None, None] - 1)
    src = torch.where(used, keep, to)

    def row(pos):
        blk = st["tables"].long().gather(1, (pos // bs).reshape(S, -1)).view(S, H, B)
        head = torch.arange(H, device="cuda")[None, :, None]
        return ((blk * H + head) * bs + pos % bs).reshape(-1)

    a, b = row(src), row(to)
    moved = [x.view(NB * H * bs, -1) for x in (k, v)]
    moved += [st[x].view(NB * H * bs, 1) for x in ("k_scales", "v_scales") if x in st]
    [x.index_copy_(0, b, x.index_select(0, a)) for x in moved]
    got = [k, v] + [st[x] for x in ("k_scales", "v_scales") if x in st]
    if "scores" in st:
        sc = st["scores"]
        sc.scatter_(2, to, sc.gather(2, src))
        at = torch.arange(sc.shape[2], device="cuda")[None, None, :]
        new = start + st["keep_lens"].long()[:, None, None]
        sc.masked_fill_((at >= new) & (at < st["lens"][:, None, None]), 0.0)
        got.append(sc)
    return got


# ------------------------------------------------------------------ one pass
def run(st):
    case = st["case"]
    op = case["op"]
    if not own:
        form = {"tree": _plain_tree, "scored": _plain_scored, "select": _plain_select}
        return form.get(op, _plain_compact)(st)
    from paged_kv_cache_context_gb300 import pa
    if op == "tree":
        ws = st.get("ws")
        if ws is None:
            ws = st["ws"] = torch.empty(
                pa.tree_workspace_size(case["heads"], case["kv_heads"], case["dim"]),
                dtype=torch.uint8, device="cuda")
        rest = (st["tables"], st["cu"], st["lens"], st["mask"], case["kv_heads"], st["max_nodes"],
                st["scale"])
        if case["kv"] == "auto":
            pa.tree_attention(st["out"], st["q"], st["k"], st["v"], *rest, ws)
        elif case["kv"] == "fp8":
            pa.tree_attention_fp8(st["out"], st["q"], st["k"], st["v"], *rest, st["k_scale"],
                                  st["v_scale"], ws)
        else:
            pa.tree_attention_int8(st["out"], st["q"], st["k"], st["v"], st["k_scales"],
                                   st["v_scales"], *rest, ws)
        return st["out"]
    if op == "scored":
        ws = st.get("ws")
        if ws is None:
            ws = st["ws"] = torch.empty(
                pa.decode_scored_workspace_size(case["seqs"], case["heads"], case["kv_heads"],
                                                case["dim"], case["bs"], st["tables"].shape[1]),
                dtype=torch.uint8, device="cuda")
        if case["kv"] == "int8":
            pa.decode_scored_int8(st["out"], st["scores"], st["q"], st["k"], st["v"],
                                  st["k_scales"], st["v_scales"], st["tables"], st["lens"],
                                  case["kv_heads"], st["scale"], ws)
        else:
            pa.decode_scored(st["out"], st["scores"], st["q"], st["k"], st["v"], st["tables"],
                             st["lens"], case["kv_heads"], st["scale"], ws,
                             kv_dtype={"auto": "auto", "fp8": "fp8_e4m3"}[case["kv"]],
                             k_scale=st["k_scale"], v_scale=st["v_scale"])
        return st["out"], st["scores"]
    if op == "select":
        pa.evict_select(st["keep"], st["new_lens"], st["scores"], st["lens"],
                        num_sink=case["sink"], num_recent=case["recent"])
        return st["keep"], st["new_lens"]
    pa.compact(st["k"], st["v"], st["tables"], st["lens"], st["keep"], st["keep_lens"],
               starts=st["starts"], k_scales=st.get("k_scales"), v_scales=st.get("v_scales"),
               scores=st.get("scores"))
    return [st[x] for x in ("k", "v", "k_scales", "v_scales", "scores") if x in st]


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    op, lens, bs = case["op"], _lens(case), case["bs"]

    def cached(s, cache, scales, scale):
        pages = st["tables"][s, : -(-lens[s] // bs)].long()
        x = cache[pages]
        x = (x.view(torch.float8_e4m3fn).to(torch.float64) if x.dtype == torch.uint8 else
             x.to(torch.float64)) * scale
        if scales is not None:
            x = x * scales[pages].double().unsqueeze(-1)
        return torch.cat(list(x), dim=1)[:, : lens[s]]  # [H, n, D]

    if op in ("tree", "scored"):
        out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
        score = st["scores"].double() if op == "scored" else None
        cu = st["cu"].tolist() if op == "tree" else list(range(case["seqs"] + 1))
        G = case["heads"] // case["kv_heads"]
        for s in range(case["seqs"]):
            K = cached(s, st["k"], st.get("k_scales"), st["k_scale"])
            V = cached(s, st["v"], st.get("v_scales"), st["v_scale"])
            t = cu[s + 1] - cu[s]
            allowed = torch.ones(t, lens[s], dtype=torch.bool, device="cuda")
            if op == "tree":
                words = st["mask"][cu[s]: cu[s + 1]]
                shift = torch.arange(64, device="cuda")
                bits = ((words.unsqueeze(-1) >> shift) & 1).bool().flatten(1)
                allowed[:, lens[s] - t:] = bits[:, :t]
            for h in range(case["heads"]):
                x = st["q"][cu[s]: cu[s + 1], h].double() @ K[h // G].T * st["scale"]
                w = torch.softmax(x.masked_fill(~allowed, -math.inf), dim=-1).nan_to_num(0.0)
                out[cu[s]: cu[s + 1], h] = w @ V[h // G]
                if op == "scored":
                    score[s, h // G, : lens[s]] += w[0]
        return out if op == "tree" else (out, score)
    if op == "select":
        return None
    was = {x: st[x].clone() for x in ("k", "v", "k_scales", "v_scales", "scores") if x in st}
    starts = [0] * case["seqs"] if st["starts"] is None else st["starts"].tolist()
    for s in range(case["seqs"]):
        a, cap = starts[s], int(st["keep_lens"][s])
        for h in range(case["kv_heads"]):
            src = st["keep"][s, h if st["keep"].shape[1] > 1 else 0, :cap].long()
            to = torch.arange(a, a + cap, device="cuda")
            t = st["tables"][s].long()
            for x in was:
                if x == "scores":
                    st[x][s, h, a: a + cap] = was[x][s, h, src]
                    st[x][s, h, a + cap: lens[s]] = 0
                else:
                    st[x][t[to // bs], h, to % bs] = was[x][t[src // bs], h, src % bs]
    got = [st[x] for x in ("k", "v", "k_scales", "v_scales", "scores") if x in st]
    return [x.double() if x.is_floating_point() else None for x in got]
