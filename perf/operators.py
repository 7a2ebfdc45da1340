"""Workloads of the operators that decode several candidates over a head-aware paged KV cache.

``attend``  attention of a tree of drafted tokens over the cache and over the draft itself
``commit``  appending the accepted path of the draft to the cache, in place
``reorder`` giving each sequence another sequence's cache (forks, beams), in place

Where ``own`` is false, ``run`` computes an operator in elementary torch
operations in fp32; where it is true, it makes the calls of the public API.
"""
from __future__ import annotations

import math
import random

import torch

own = False

CAPACITY = 128  # tokens a sequence may still gain in the plans below


def _attend(name, batch, q_heads, kv_heads, dim, ctx_min, ctx_max, nodes, *, sink=4, window=512, global_every=4,
            dtype="bf16", pages="bf16", page=64, tree="bushy", ragged=False):
    return dict(name=name, op="attend", batch=batch, q_heads=q_heads, kv_heads=kv_heads, dim=dim, ctx_min=ctx_min,
                ctx_max=ctx_max, nodes=nodes, sink=sink, window=window, global_every=global_every, dtype=dtype,
                pages=pages, page=page, tree=tree, ragged=ragged)


def _commit(name, batch, kv_heads, dim, ctx_min, ctx_max, nodes, path, *, sink=4, window=512, global_every=4,
            dtype="bf16", page=64):
    return dict(name=name, op="commit", batch=batch, kv_heads=kv_heads, dim=dim, ctx_min=ctx_min, ctx_max=ctx_max,
                nodes=nodes, path=path, sink=sink, window=window, global_every=global_every, dtype=dtype, page=page)


def _reorder(name, batch, kv_heads, dim, ctx, moved, common, *, sink=4, window=512, global_every=4, dtype="bf16",
             page=64):
    return dict(name=name, op="reorder", batch=batch, kv_heads=kv_heads, dim=dim, ctx_min=ctx, ctx_max=ctx,
                moved=moved, common=common, sink=sink, window=window, global_every=global_every, dtype=dtype, page=page)


def listed():
    return [
        # one user, a short chain from a small drafter: latency
        _attend("attend_one_user_chain", 1, 32, 8, 128, 1000, 1000, 5, tree="chain"),
        # the 8K layer, a tree of 32 nodes, fewer on some sequences
        _attend("attend_8k_tree32_ragged", 4, 32, 8, 128, 8192, 8192, 32, ragged=True),
        # the 32K layer at batch 8, one query tile of 128 rows for each kv-head
        _attend("attend_32k_tree16", 8, 64, 8, 128, 32768, 32768, 16, window=8192, global_every=8),
        # the same layer with the widest tree: the largest amount of arithmetic
        _attend("attend_32k_tree64", 8, 64, 8, 128, 32768, 32768, 64, window=8192, global_every=8),
        # 32 users with contexts of every length
        _attend("attend_ragged_batch32", 32, 32, 8, 128, 1024, 65536, 8),
        # the 32K layer on FP8 pages
        _attend("attend_32k_e4m3_tree16", 8, 64, 8, 128, 32768, 32768, 16, window=8192, global_every=8, pages="e4m3"),
        # no shared kv-heads: 24 rows for each head's keys
        _attend("attend_mha_tree24", 2, 64, 64, 128, 16384, 16384, 24, window=128, global_every=8),
        # the fp32 layer
        _attend("attend_f32_tree13", 2, 4, 2, 64, 200, 256, 13, dtype="f32", pages="f32", page=16, window=32,
                global_every=2),
        # one user accepts a few tokens
        _commit("commit_one_user", 1, 8, 128, 1000, 1000, 8, 4),
        # 32 users of the 32K layer accept up to 8 of 64 nodes each
        _commit("commit_batch32", 32, 8, 128, 4096, 32768, 64, 8, window=8192, global_every=8),
        # four beams that share a prompt of 1000 tokens: one beam dies
        _reorder("reorder_4_beams", 4, 8, 128, 1300, 1, 1000),
        # the 32K layer: half the sequences take over another one, nothing in common
        _reorder("reorder_32k_batch8", 8, 8, 128, 32768, 4, 0, window=8192, global_every=8),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "commit", "reorder"])
    kind = rng.choice(["bf16", "bf16", "e4m3", "f32"]) if op == "attend" else rng.choice(["bf16", "bf16", "f32"])
    dim = rng.choice([64, 128])
    f32 = kind == "f32"
    page = rng.choice([16, 64]) if f32 else 64
    hkv = rng.randint(1, 8)
    batch = _log_int(rng, 1, 16)
    ctx_max = _log_int(rng, 1, 2048 if f32 else 32768)
    nodes = _log_int(rng, 1, 24 if f32 else 64)
    window, sink, every = _log_int(rng, 1, 8192), rng.choice([0, 1, 4, 4, 4, 17, 130]), rng.choice([1, 2, 4, 8])
    dtype = "f32" if f32 else "bf16"
    if op == "attend":
        g = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        while batch * hkv * g * nodes * ctx_max > 5e8:  # half of the largest listed case's (query, key) pairs
            batch, ctx_max = (batch // 2, ctx_max) if batch > 1 else (batch, ctx_max // 2)
        return dict(op=op, batch=batch, q_heads=hkv * g, kv_heads=hkv, dim=dim, ctx_min=max(1, ctx_max // 8),
                    ctx_max=ctx_max, nodes=nodes, sink=sink, window=window, global_every=every, dtype=dtype,
                    pages=kind, page=page, tree=rng.choice(["bushy", "chain"]), ragged=rng.random() < 0.5)
    if op == "commit":
        nodes = rng.randint(1, 64)
        return dict(op=op, batch=batch, kv_heads=hkv, dim=dim, ctx_min=max(1, ctx_max // 8), ctx_max=ctx_max,
                    nodes=nodes, path=rng.randint(1, nodes), sink=sink, window=window, global_every=every,
                    dtype=dtype, page=page)
    batch = max(2, batch)
    return dict(op=op, batch=batch, kv_heads=hkv, dim=dim, ctx_min=ctx_max, ctx_max=ctx_max,
                moved=rng.randint(1, batch), common=rng.choice([0, ctx_max // 2, ctx_max - 1]), sink=sink,
                window=window, global_every=every, dtype=dtype, page=page)


# --------------------------------------------------------------------------
# What a program has before the call
# --------------------------------------------------------------------------

def _lens(c):
    """Context lengths of the batch: spread over the logarithm of the range, the first the longest."""
    r = random.Random(c["batch"] * 7919 + c["ctx_max"])
    n = [int(math.exp(r.uniform(math.log(c["ctx_min"]), math.log(c["ctx_max"])))) for _ in range(c["batch"])]
    n[0] = c["ctx_max"]
    return [min(c["ctx_max"], max(c["ctx_min"], x)) for x in n]


def _node_counts(c):
    r = random.Random(c["nodes"] * 31 + c["batch"])
    return [r.randint(1, c["nodes"]) if c["ragged"] and b else c["nodes"] for b in range(c["batch"])]


def _is_global(c):
    return [h % c["global_every"] == 0 for h in range(c["kv_heads"])]


def _element(c):
    return torch.float32 if c["dtype"] == "f32" else torch.bfloat16


def _layer(c, lens, **kw):
    from head_aware_paged_build_b200 import segpaged as S
    from head_aware_paged_build_b200.runtime import SegPagedLayer

    policy = [("global", 0, 0) if g else ("local", c["sink"], c["window"]) for g in _is_global(c)] * c["batch"]
    return SegPagedLayer(batch=c["batch"], num_q_heads=c.get("q_heads", c["kv_heads"]), num_kv_heads=c["kv_heads"],
                         head_dim=c["dim"], page_size=c["page"], dtype=c["dtype"], ctx_len=lens,
                         q_start=[n - 1 for n in lens], policy=policy, flags=S.SP_FLAG_RING,
                         append_capacity=CAPACITY, **kw)


E4M3_SCALE = 2.0 ** -6  # a power of two: the dense values below are codes times it, exactly


def _parents(c, rng, counts):
    """parent[b][i] < i (-1: a root); entries behind a sequence's nodes are not read."""
    rows = []
    for n in counts:
        if c["tree"] == "chain":
            row = [i - 1 for i in range(n)]
        else:  # most nodes hang near the top; now and then a second root
            row = [-1 if i == 0 or rng.random() < 0.05 else int(i * rng.random() ** 1.5) for i in range(n)]
        rows.append(row + [0] * (c["nodes"] - n))
    return rows


def _prepare_attend(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)
    B, T, Hq, Hkv, D, el = c["batch"], c["nodes"], c["q_heads"], c["kv_heads"], c["dim"], _element(c)
    lens, counts = _lens(c), _node_counts(c)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=el)

    st = dict(case=c, q=normal(B, T, Hq, D), k_draft=normal(B, T, Hkv, D), v_draft=normal(B, T, Hkv, D),
              parents=torch.tensor(_parents(c, rng, counts), dtype=torch.int32, device="cuda"),
              counts=torch.tensor(counts, dtype=torch.int32, device="cuda"),
              out=torch.zeros(B, T, Hq, D, dtype=el, device="cuda"),
              lse=torch.zeros(B, T, Hq, dtype=torch.float32, device="cuda"))
    k, v = normal(B, Hkv, max(lens), D), normal(B, Hkv, max(lens), D)
    kw = {}
    if c["pages"] == "e4m3":
        codes = [(x.float() / E4M3_SCALE).clamp(-448, 448).to(torch.float8_e4m3fn) for x in (k, v)]
        k, v = codes
        kw = dict(kv_dtype="e4m3", k_scale=E4M3_SCALE, v_scale=E4M3_SCALE)
    if own:
        st["layer"] = _layer(c, lens, **kw)
        if c["pages"] == "e4m3":
            k, v = [(x.float() * E4M3_SCALE).bfloat16() for x in codes]
        st["layer"].build(k, v)
        torch.cuda.synchronize()
        st["layer"].prepare_tree(T)
    else:
        st["k"], st["v"] = k, v
        st["lens"] = torch.tensor(lens, device="cuda")
        st["is_global"] = torch.tensor(_is_global(c), device="cuda")
    return st


def _records(c, n):
    """Page records of one sequence's heads in a ring plan: (records, sink pages, ring pages) of each."""
    P, out = c["page"], []
    for g in _is_global(c):
        if g:
            out.append((-(-(n + CAPACITY) // P), 0, 0))
        else:
            sink, ring = -(-c["sink"] // P), -(-c["window"] // P) + 1
            out.append((sink + ring, sink, ring))
    return out


def _pools(c, lens, g):
    """K and V pools holding normal values, as the plan's pages would (one page of each pool for each record)."""
    pages = sum(r[0] for n in lens for r in _records(c, n))
    elements = c["page"] * c["dim"]
    return [torch.randn(pages, elements, generator=g, device="cuda", dtype=_element(c)) for _ in range(2)]


def _prepare_commit(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)
    B, T, Hkv, D, el, lens = c["batch"], c["nodes"], c["kv_heads"], c["dim"], _element(c), _lens(c)
    # the longest path on the first sequence, any length on the others; node indices rise along a path
    count = [c["path"] if b == 0 else rng.randint(0, c["path"]) for b in range(B)]
    path = [sorted(rng.sample(range(T), n)) + [0] * (c["path"] - n) for n in count]
    k_pool, v_pool = _pools(c, lens, g)
    st = dict(case=c, k_pool=k_pool, v_pool=v_pool,
              k_draft=torch.randn(B, T, Hkv, D, generator=g, device="cuda", dtype=el),
              v_draft=torch.randn(B, T, Hkv, D, generator=g, device="cuda", dtype=el),
              path=torch.tensor(path, dtype=torch.int32, device="cuda"),
              count=torch.tensor(count, dtype=torch.int32, device="cuda"))
    if own:
        st["layer"] = _layer(c, lens, pools=(k_pool.view(torch.uint8).view(-1), v_pool.view(torch.uint8).view(-1)))
        torch.cuda.synchronize()
        st["table"] = st["layer"].table.clone()
    else:
        recs = [_records(c, n) for n in lens]
        first, at = [], 0
        for per in recs:
            row = []
            for r in per:
                row.append(at)
                at += r[0]
            first.append(row)
        st["first"] = torch.tensor(first, device="cuda")
        st["sink_pages"] = torch.tensor([[r[1] for r in per] for per in recs], device="cuda")
        st["ring_pages"] = torch.tensor([[max(1, r[2]) for r in per] for per in recs], device="cuda")
        st["is_global"] = torch.tensor(_is_global(c), device="cuda")
        st["lens"] = torch.tensor(lens, device="cuda")
        st["lens_now"] = st["lens"].clone()
    return st


def _prepare_reorder(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)
    B, lens = c["batch"], _lens(c)
    # `moved` sequences take over another one; when all do, a rotation
    if c["moved"] >= B:
        shift = rng.randint(1, B - 1)
        parents = [(b + shift) % B for b in range(B)]
    else:
        moved = rng.sample(range(B), c["moved"])
        kept = [b for b in range(B) if b not in moved]
        rng.shuffle(kept)
        parents = list(range(B))
        for i, b in enumerate(moved):
            parents[b] = kept[i % len(kept)]
    k_pool, v_pool = _pools(c, lens, g)
    st = dict(case=c, k_pool=k_pool, v_pool=v_pool, parents=torch.tensor(parents, dtype=torch.int32, device="cuda"),
              common=torch.full((B,), c["common"], dtype=torch.int32, device="cuda"))
    if own:
        st["layer"] = _layer(c, lens, pools=(k_pool.view(torch.uint8).view(-1), v_pool.view(torch.uint8).view(-1)))
        torch.cuda.synchronize()
    else:
        st["copied"] = torch.tensor(_copied_pages(c), device="cuda")
    return st


def _copied_pages(c):
    """Page records of a sequence that hold a token and are not wholly below the common positions."""
    P, n, out = c["page"], c["ctx_max"], []
    for (records, sink, ring), is_global in zip(_records(c, n), _is_global(c)):
        base = len(out)
        out += [False] * records
        if is_global:
            for i in range(-(-n // P)):
                out[base + i] = min(n, (i + 1) * P) > c["common"]
            continue
        for i in range(sink):
            held = min(n, c["sink"], (i + 1) * P)
            out[base + i] = held > i * P and held > c["common"]
        lo = max(c["sink"], n - c["window"])
        for block in range(lo // P, -(-n // P)):
            top = min(n, (block + 1) * P)
            if top > max(lo, block * P) and top > c["common"]:
                out[base + sink + block % ring] = True
    return out


def prepare(case, seed):
    return {"attend": _prepare_attend, "commit": _prepare_commit, "reorder": _prepare_reorder}[case["op"]](case, seed)


# --------------------------------------------------------------------------
# Plain forms
# --------------------------------------------------------------------------

def _tree_of(st):
    """(valid [B, T], ancestors-or-self [B, T, T], depth [B, T])."""
    B, T = st["parents"].shape
    node = torch.arange(T, device="cuda")
    valid = node < st["counts"][:, None]
    parents = torch.where(valid, st["parents"], -1)
    step = (parents[:, :, None] == node) | torch.eye(T, dtype=torch.bool, device="cuda")
    anc = torch.linalg.matrix_power(step.double(), T) > 0.5
    return valid, anc, anc.sum(-1) - 1


def _quantised(x):
    return (x.float() * (1.0 / E4M3_SCALE)).clamp(-448, 448).to(torch.float8_e4m3fn).float() * E4M3_SCALE


def _plain_attend(st):
    c = st["case"]
    B, T, Hq, Hkv, D = c["batch"], c["nodes"], c["q_heads"], c["kv_heads"], c["dim"]
    g = Hq // Hkv
    scale = 1.0 / math.sqrt(D)
    k, v, kd, vd = (st[n].float() for n in ("k", "v", "k_draft", "v_draft"))
    if c["pages"] == "e4m3":  # the draft's rows count as the cache will hold them
        k, v = k * E4M3_SCALE, v * E4M3_SCALE
        kd, vd = _quantised(kd), _quantised(vd)
    kd, vd = kd.transpose(1, 2), vd.transpose(1, 2)
    q = st["q"].float().view(B, T, Hkv, g, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * g, D)
    valid, anc, depth = _tree_of(st)
    pos = st["lens"][:, None] + depth
    j = torch.arange(k.shape[2], device="cuda")
    far = st["is_global"][None, :, None, None]
    see = (j < st["lens"][:, None, None, None]) & (
        far | ((j < c["sink"]) | (j > (pos - c["window"])[:, :, None]))[:, None])
    see_draft = anc[:, None] & (
        far | ((pos < c["sink"])[:, None, :] | (pos[:, None, :] > (pos - c["window"])[:, :, None]))[:, None])
    s = (q @ k.transpose(-1, -2) * scale).view(B, Hkv, T, g, -1).masked_fill(~see[:, :, :, None], -math.inf)
    sd = (q @ kd.transpose(-1, -2) * scale).view(B, Hkv, T, g, T).masked_fill(~see_draft[:, :, :, None], -math.inf)
    m = torch.maximum(s.amax(-1, keepdim=True), sd.amax(-1, keepdim=True))
    p, pd = torch.exp(s - m), torch.exp(sd - m)
    total = p.sum(-1, keepdim=True) + pd.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ v + pd.flatten(2, 3) @ vd).view(B, Hkv, T, g, D) / total
    lse = (m + total.log()).squeeze(-1)
    o = o.permute(0, 2, 1, 3, 4).reshape(B, T, Hq, D)
    lse = lse.permute(0, 2, 1, 3).reshape(B, T, Hq)
    st["out"].copy_(torch.where(valid[:, :, None, None], o, 0.0))
    st["lse"].copy_(torch.where(valid[:, :, None], lse, 0.0))
    return st["out"], st["lse"]


def _places(c, slot):
    """Element offsets in a K and a V page of the row at ``slot`` (the pages' layouts), [..., D]."""
    P, D = c["page"], c["dim"]
    i = torch.arange(D, device="cuda")
    t = slot[..., None]
    if c["dtype"] == "f32":
        return t * D + i, i * P + t
    k = (i // 64) * (P * 64) + t * 64 + (((i % 64) // 8) ^ (t & 7)) * 8 + i % 8
    v = i * 64 + ((t // 8) ^ (i & 7)) * 8 + t % 8
    return k, v


def _plain_commit(st):
    c = st["case"]
    st["lens_now"].copy_(st["lens"])
    n = st["path"].shape[1]
    step = torch.arange(n, device="cuda")
    pos = (st["lens_now"][:, None] + step)[:, None]  # [B, 1, n]
    ring_tokens = st["ring_pages"][:, :, None] * c["page"]
    in_ring = ~st["is_global"][None, :, None] & (pos >= c["sink"])
    r = pos % ring_tokens
    record = torch.where(in_ring, st["sink_pages"][:, :, None] + r // c["page"], pos // c["page"])
    slot = torch.where(in_ring, r % c["page"], pos % c["page"])
    last = ~in_ring | (step + ring_tokens >= st["count"][:, None, None])  # a later token takes an earlier one's slot
    keep = (step < st["count"][:, None])[:, None] & last
    page = st["first"][:, :, None] + record
    kat, vat = _places(c, slot)
    b = torch.arange(c["batch"], device="cuda")[:, None]
    rows_k, rows_v = (st[x][b, st["path"].long()].transpose(1, 2) for x in ("k_draft", "v_draft"))
    keep = keep & torch.ones_like(page, dtype=torch.bool)
    at = page[keep][:, None] * (c["page"] * c["dim"])
    st["k_pool"].view(-1)[at + kat[keep]] = rows_k[keep]
    st["v_pool"].view(-1)[at + vat[keep]] = rows_v[keep]
    st["lens_now"].add_(st["count"])
    return st["k_pool"], st["v_pool"]


def _plain_reorder(st):
    c = st["case"]
    parents = st["parents"].long()
    moved = parents != torch.arange(c["batch"], device="cuda")
    take = (moved[:, None] & st["copied"])[:, :, None]
    for pool in (st["k_pool"], st["v_pool"]):
        per = pool.view(c["batch"], -1, pool.shape[1])
        per.copy_(torch.where(take, per[parents], per))
    return st["k_pool"], st["v_pool"]


def run(state):
    op = state["case"]["op"]
    if not own:
        return {"attend": _plain_attend, "commit": _plain_commit, "reorder": _plain_reorder}[op](state)
    layer = state["layer"]
    if op == "attend":
        return layer.tree_attention(state["q"], state["k_draft"], state["v_draft"], state["parents"],
                                    num_nodes=state["counts"], out=state["out"], lse=state["lse"])
    if op == "commit":
        layer.table.copy_(state["table"])  # each pass appends to the same context
        layer.tree_commit(state["k_draft"], state["v_draft"], state["path"], state["count"])
    else:
        layer.reorder(state["parents"], common_len=state["common"])
    return state["k_pool"], state["v_pool"]


# --------------------------------------------------------------------------
# Work and exact values
# --------------------------------------------------------------------------

def work(case):
    c = case
    el = 4 if c["dtype"] == "f32" else 2
    D, lens = c["dim"], _lens(c)
    if c["op"] == "attend":
        eb = 1 if c["pages"] == "e4m3" else el
        g, counts = c["q_heads"] // c["kv_heads"], _node_counts(c)
        # cached tokens that a root of the tree sees
        seen = [[n if far else min(n, c["sink"] + c["window"] - 1) for far in _is_global(c)] for n in lens]
        tokens = sum(sum(s) for s in seen)
        pairs = sum(sum(s) * t * g for s, t in zip(seen, counts))
        nodes = sum(counts)
        return {"bytes": tokens * 2 * D * eb + nodes * (2 * c["q_heads"] + 2 * c["kv_heads"]) * D * el +
                nodes * c["q_heads"] * 4 + nodes * 4, "flops": 4 * D * pairs}
    if c["op"] == "commit":
        tokens = c["path"] * (1 + (c["batch"] - 1) / 2)  # the first sequence's path is the longest
        return {"bytes": tokens * c["kv_heads"] * 2 * D * el * 2, "flops": 0}
    pages = sum(_copied_pages(c))
    sources = min(c["moved"], max(1, c["batch"] - c["moved"])) if c["moved"] < c["batch"] else c["batch"]
    return {"bytes": (sources + c["moved"]) * pages * c["page"] * D * el * 2, "flops": 0}


def exact(case, seed):
    """The attention from its definition in fp64: for each node, the list of what it sees."""
    c = case
    if c["op"] != "attend":
        return None  # copies: nothing is computed
    g, lens, counts = c["q_heads"] // c["kv_heads"], _lens(c), _node_counts(c)
    if sum(n * t for n, t in zip(lens, counts)) * c["q_heads"] * c["dim"] > 4e11:
        return None
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)
    el, B, T, D = _element(c), c["batch"], c["nodes"], c["dim"]
    q = torch.randn(B, T, c["q_heads"], D, generator=gen, device="cuda", dtype=el)
    kd = torch.randn(B, T, c["kv_heads"], D, generator=gen, device="cuda", dtype=el)
    vd = torch.randn(B, T, c["kv_heads"], D, generator=gen, device="cuda", dtype=el)
    k = torch.randn(B, c["kv_heads"], max(lens), D, generator=gen, device="cuda", dtype=el)
    v = torch.randn(B, c["kv_heads"], max(lens), D, generator=gen, device="cuda", dtype=el)
    if c["pages"] == "e4m3":
        def stored(x):
            return (x.float() / E4M3_SCALE).clamp(-448, 448).to(torch.float8_e4m3fn).double() * E4M3_SCALE
        k, v, kd, vd = stored(k), stored(v), stored(kd), stored(vd)
    parents = _parents(c, rng, counts)
    out = torch.zeros(B, T, c["q_heads"], D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(B, T, c["q_heads"], dtype=torch.float64, device="cuda")
    for b in range(B):
        L, lines = lens[b], []
        for i in range(counts[b]):  # the nodes from i up to its root
            line = [i]
            while parents[b][line[-1]] >= 0:
                line.append(parents[b][line[-1]])
            lines.append(line)
        for h, far in enumerate(_is_global(c)):
            keys, vals = k[b, h, :L].double(), v[b, h, :L].double()
            heads = slice(h * g, (h + 1) * g)
            for i, line in enumerate(lines):
                at = L + len(line) - 1  # the node's position
                where = {a: L + len(lines[a]) - 1 for a in line}
                nodes = [a for a in line if far or where[a] < c["sink"] or where[a] >= at - c["window"] + 1]
                lo = 0 if far else max(0, min(L, at - c["window"] + 1))
                head = 0 if far else min(c["sink"], lo)
                kk = torch.cat([keys[:head], keys[lo:], kd[b, nodes, h].double()])
                vv = torch.cat([vals[:head], vals[lo:], vd[b, nodes, h].double()])
                s = q[b, i, heads].double() @ kk.T / math.sqrt(D)
                top = s.max(-1, keepdim=True).values
                e = torch.exp(s - top)
                z = e.sum(-1, keepdim=True)
                out[b, i, heads] = (e / z) @ vv
                lse[b, i, heads] = (top + torch.log(z)).squeeze(-1)
    return out, lse
