"""Tree commit and reorder on the GPU, and a run of them with tree attention and decode attention."""
from __future__ import annotations

import random

import pytest
import torch

from head_aware_paged_build_b200 import segpaged as S
from head_aware_paged_build_b200.runtime import SegPagedLayer
from _table import BAD_PAGE, corrupt
from _tree import lines_of, random_tree

pytestmark = pytest.mark.gpu

KINDS = [("local", 4, 40), ("global", 0, 0), ("local", 0, 3), ("local", 300, 10), ("local", 4, 130)]
FORMATS = [("bf16", 64, 128), ("bf16", 64, 64), ("e4m3", 64, 128), ("e4m3", 64, 64), ("f32", 16, 64),
           ("f32", 16, 128), ("f32", 64, 64)]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    S.load()


def _layer(pages, page, d, lens, kinds=KINDS, g=2, capacity=200, **kw):
    if pages == "e4m3":
        kw.update(kv_dtype="e4m3", k_scale=0.01, v_scale=0.02)
    policy = kinds if len(kinds) == len(lens) * 5 else list(kinds) * len(lens)
    hkv = len(policy) // len(lens)
    return SegPagedLayer(batch=len(lens), num_q_heads=hkv * g, num_kv_heads=hkv, head_dim=d, page_size=page,
                         dtype="f32" if pages == "f32" else "bf16", ctx_len=lens, q_start=[n - 1 for n in lens],
                         policy=policy, flags=S.SP_FLAG_RING, append_capacity=capacity, **kw)


def _normal(layer, *shape, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=gen, device="cuda", dtype=layer.torch_dtype)


def _build(layer, seed=0):
    shape = (layer.batch, layer.num_kv_heads, max(layer.ctx_len), layer.head_dim)
    k, v = _normal(layer, *shape, seed=seed), _normal(layer, *shape, seed=seed + 1)
    layer.build(k, v)
    return k, v


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _rows(kd, vd, path, step):
    """Contiguous [B, Hkv, d] rows of the node each sequence appends at `step`."""
    b = torch.arange(kd.shape[0], device="cuda")
    return kd[b, path[:, step].long()].contiguous(), vd[b, path[:, step].long()].contiguous()


def _same(a, b):
    torch.cuda.synchronize()
    assert torch.equal(a.table, b.table)
    assert torch.equal(a.k_pool, b.k_pool) and torch.equal(a.v_pool, b.v_pool)


@pytest.mark.parametrize("pages,page,d", FORMATS)
def test_commit_equals_appends(pages, page, d):
    """Paths of one length for all sequences, until every ring has wrapped: the same bytes as the appends."""
    lens = (70, 200, 5, 131, 1)
    a, b = _layer(pages, page, d, lens), _layer(pages, page, d, lens)
    a.k_pool.zero_(), b.k_pool.zero_(), a.v_pool.zero_(), b.v_pool.zero_()
    _build(a), _build(b)
    rng = random.Random(1)
    left, i = 200, 0
    while left:
        n, T = min(left, rng.choice([1, 2, 5, 17, 64])), 64
        packed = _normal(a, len(lens), T, 2, 5, d, seed=10 + i)
        kd, vd = packed[:, :, 0], packed[:, :, 1]
        path = _i32([[rng.randrange(T) for _ in range(n)] for _ in lens])
        a.tree_commit(kd, vd, path, _i32([n] * len(lens)))
        for step in range(n):
            b.append(*_rows(kd, vd, path, step))
        _same(a, b)
        left, i = left - n, i + 1
    assert a.device_status() == 0 and b.device_status() == 0
    packed = _normal(a, len(lens), 64, 2, 5, d, seed=5)
    path = _i32([[0]] * len(lens))
    a.tree_commit(packed[:, :, 0], packed[:, :, 1], path, _i32([0] * len(lens)))  # nothing accepted
    _same(a, b)


@pytest.mark.parametrize("pages,page,d", [("bf16", 64, 128), ("f32", 16, 64)])
def test_commit_without_room_keeps_what_fits(pages, page, d):
    lens = (61, 200)
    a, b = (_layer(pages, page, d, lens, capacity=3) for _ in range(2))
    for x in (a, b):
        x.k_pool.zero_(), x.v_pool.zero_()
        _build(x)
    kd, vd = _normal(a, 2, 40, 5, d, seed=8), _normal(a, 2, 40, 5, d, seed=9)
    path = _i32([list(range(40))] * 2)
    a.tree_commit(kd, vd, path, _i32([40, 40]))
    for step in range(40):
        b.append(*_rows(kd, vd, path, step))
    _same(a, b)
    assert a.device_status() == 6 and b.device_status() == 6


def test_commit_takes_pages_from_the_spare_pool():
    """Lengths that differ by sequence; the pool runs out for the last one alone."""
    lens, kinds = (60, 62, 64), [("global", 0, 0), ("local", 4, 40)]
    layer = _layer("bf16", 64, 128, lens, kinds, spare_pages=4, capacity=300)
    k, v = _build(layer)
    counts = [64, 30, 1]
    want = [torch.zeros(3, 2, 64 + 64, 128, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    kd, vd = _normal(layer, 3, 64, 2, 128, seed=4), _normal(layer, 3, 64, 2, 128, seed=5)
    for w, cached, draft in zip(want, (k, v), (kd, vd)):
        for b, L in enumerate(lens):
            w[b, :, :L] = cached[b, :, :L]
            w[b, :, L:L + counts[b]] = draft[b, :counts[b]].transpose(0, 1)
    layer.tree_commit(kd, vd, _i32([list(range(64))] * 3), _i32(counts))
    got = [torch.zeros_like(w) for w in want]
    layer.gather(*got)
    torch.cuda.synchronize()
    assert layer.device_status() == 0  # 64 more tokens: one page; 62 + 30: one; 64 + 1: one
    for w, x in zip(want, got):
        for b, L in enumerate(lens):
            n = L + counts[b]
            assert torch.equal(x[b, 0, :n], w[b, 0, :n])
            seen = [j for j in range(n) if j < 4 or j >= n - 40]
            assert torch.equal(x[b, 1, seen], w[b, 1, seen])
    layer.tree_commit(kd, vd, _i32([list(range(64))] * 3), _i32([0, 0, 64]))  # the last spare page
    layer.tree_commit(kd, vd, _i32([list(range(64))] * 3), _i32([64, 0, 0]))
    torch.cuda.synchronize()
    assert layer.device_status() == 7


def test_commit_refuses_bad_paths_on_the_device():
    lens = (70, 200, 64)
    for lengths, node in (((3, 5, 2), 0), ((3, -1, 2), 0), ((3, 2, 2), 9), ((3, 2, 2), -1)):
        a, b = (_layer("bf16", 64, 128, lens) for _ in range(2))
        for x in (a, b):
            x.k_pool.zero_(), x.v_pool.zero_()
            _build(x)
        kd, vd = _normal(a, 3, 9, 5, 128, seed=4), _normal(a, 3, 9, 5, 128, seed=5)
        path = _i32([[0, 1, 2, 3], [2, node, 1, 1], [8, 4, 5, 6]])
        a.tree_commit(kd, vd, path, _i32(lengths))
        path[1] = 0
        b.tree_commit(kd, vd, path, _i32([3, 0, 2]))  # sequence 1 left as it is
        _same(a, b)
        assert a.device_status() == 8 and b.device_status() == 0


def test_commit_reports_a_page_outside_the_pool():
    layer = _layer("bf16", 64, 128, (70, 200))
    _build(layer)
    corrupt(layer, 0, 1, 1)
    kd, vd = _normal(layer, 2, 9, 5, 128, seed=4), _normal(layer, 2, 9, 5, 128, seed=5)
    layer.tree_commit(kd, vd, _i32([[0, 1]] * 2), _i32([2, 2]))
    torch.cuda.synchronize()
    assert layer.device_status() == BAD_PAGE


# -- reorder ------------------------------------------------------------------

def _gathered(layer, width):
    dt = torch.uint8 if layer.kv_dtype == "e4m3" else layer.torch_dtype
    out = [torch.zeros(layer.batch, layer.num_kv_heads, width, layer.head_dim, device="cuda", dtype=dt)
           for _ in range(2)]
    layer.gather(*out)
    torch.cuda.synchronize()
    return out


def _grow(layer, counts, seed):
    B, n, T = layer.batch, max(max(counts), 1), 64
    kd, vd = (_normal(layer, B, T, layer.num_kv_heads, layer.head_dim, seed=seed + i) for i in range(2))
    layer.tree_commit(kd, vd, _i32([list(range(n))] * B), _i32(counts))


@pytest.mark.parametrize("pages,page,d", [("bf16", 64, 128), ("bf16", 64, 64), ("e4m3", 64, 128), ("f32", 16, 64),
                                          ("f32", 64, 128)])
def test_reorder_moves_whole_caches(pages, page, d):
    """Rotations, swaps, forks, two cycles and random maps over sequences that have grown apart."""
    B = 7
    layer = _layer(pages, page, d, (150,) * B)
    _build(layer)
    rng = random.Random(2)
    maps = [[1, 2, 3, 4, 5, 6, 0], [1, 0, 3, 4, 2, 5, 6], [3] * 7, list(range(7)), [0, 0, 1, 2, 3, 4, 5],
            [1, 0, 0, 1, 5, 4, 4]]
    maps += [[rng.randrange(B) for _ in range(B)] for _ in range(6)]
    for i, parents in enumerate(maps):
        _grow(layer, [rng.choice([0, 1, 3, 10]) for _ in range(B)], 100 + 2 * i)
        before = _gathered(layer, 400)
        layer.reorder(_i32(parents))
        after = _gathered(layer, 400)
        for x, y in zip(before, after):
            assert torch.equal(x[parents], y), parents
    _grow(layer, [1] * B, 300)  # and the caches still grow
    assert layer.device_status() == 0


def test_reorder_of_many_sequences():
    """More sequences than threads a block, every one of them moved."""
    B = 600
    layer = _layer("f32", 16, 64, (20,) * B, kinds=[("global", 0, 0), ("local", 4, 9)], capacity=8)
    _build(layer)
    rng = random.Random(4)
    perm = list(range(B))
    rng.shuffle(perm)
    for parents in (perm, [rng.randrange(B) for _ in range(B)], [(b + 1) % B for b in range(B)]):
        before = _gathered(layer, 40)
        layer.reorder(_i32(parents))
        after = _gathered(layer, 40)
        for x, y in zip(before, after):
            assert torch.equal(x[parents], y)
    assert layer.device_status() == 0


def test_reorder_leaves_known_equal_positions():
    """A shared prompt of 150 tokens: forks differ behind it alone, with and without common_len."""
    B, L = 4, 150
    a, b = (_layer("bf16", 64, 128, (L,) * B) for _ in range(2))
    for x in (a, b):
        k, v = (_normal(x, 1, 5, L, 128, seed=s).expand(B, -1, -1, -1).contiguous() for s in (0, 1))
        x.build(k, v)
    for i, parents in enumerate(([1, 1, 3, 2], [0, 0, 0, 0], [1, 2, 3, 0])):
        for x in (a, b):
            _grow(x, [60, 1, 0, 9], 40 + 2 * i)  # sequence 0's rings leave pages of the prompt behind
        want = [x[parents] for x in _gathered(a, 400)]
        a.reorder(_i32(parents), common_len=_i32([L] * B))
        b.reorder(_i32(parents))
        for w, x, y in zip(want, _gathered(a, 400), _gathered(b, 400)):
            assert torch.equal(w, x) and torch.equal(w, y)
    assert a.device_status() == 0 and b.device_status() == 0


def test_reorder_with_a_spare_pool():
    """A short sequence takes over a longer one: its GLOBAL head needs pages of the pool; then back."""
    kinds = [("global", 0, 0), ("local", 4, 40)]
    layer = _layer("bf16", 64, 128, (60,) * 3, kinds, spare_pages=5, capacity=300)
    _build(layer)
    for i in range(2):
        _grow(layer, [64, 0, 0], 7 + 2 * i)  # sequence 0: 188 tokens, two pages of the pool
    for parents in ([0, 0, 2], [2, 1, 2], [1, 1, 2]):
        before = _gathered(layer, 400)
        layer.reorder(_i32(parents))
        after = _gathered(layer, 400)
        for x, y in zip(before, after):
            assert torch.equal(x[parents], y), parents
    assert layer.device_status() == 0  # 4 of the 5 pages taken
    layer.reorder(_i32([0, 1, 0]))  # needs two more
    torch.cuda.synchronize()
    assert layer.device_status() == 7


def test_reorder_refuses_what_is_laid_out_otherwise():
    lens = (150, 150, 150, 400)
    kinds = list(KINDS) * 4
    kinds[5 * 1 + 2] = ("local", 0, 4)  # another window on one head of sequence 1
    layer = _layer("bf16", 64, 128, lens, kinds)
    _build(layer)
    before = _gathered(layer, 600)
    layer.reorder(_i32([2, 0, 7, -1]))  # 0 <- 2 fits; 1 and 0 differ; 7 and -1 do not exist
    after = _gathered(layer, 600)
    assert layer.device_status() == 9
    for x, y in zip(before, after):
        assert torch.equal(x[[2, 1, 2, 3]], y)
    S.segpaged_clear_device_status(layer.workspace.data_ptr(), torch.cuda.current_stream().cuda_stream)
    layer.reorder(_i32([0, 1, 2, 0]))  # 400 tokens: more page records
    torch.cuda.synchronize()
    assert layer.device_status() == 9
    corrupt(layer, 2, 1, 1)
    S.segpaged_clear_device_status(layer.workspace.data_ptr(), torch.cuda.current_stream().cuda_stream)
    layer.reorder(_i32([2, 1, 2, 3]))
    torch.cuda.synchronize()
    assert layer.device_status() == BAD_PAGE


# -- together -------------------------------------------------------------------

@pytest.mark.parametrize("pages,page", [("bf16", 64), ("e4m3", 64), ("f32", 16)])
def test_speculative_decoding_over_the_cache(pages, page):
    """Draft, attend, accept, commit, fork, decode: a node's attention is that of the decode call after its path."""
    B, T, g, d = 4, 12, 4, 128
    layer = _layer(pages, page, d, (90,) * B, g=g)
    _build(layer)
    hq, rng = 5 * g, random.Random(6)
    for step in range(5):
        q = _normal(layer, B, T, hq, d, seed=20 + step)
        kd, vd = (_normal(layer, B, T, 5, d, seed=s + step) for s in (40, 60))
        parents = [random_tree(rng, T, "random") for _ in range(B)]
        out, lse = layer.tree_attention(q, kd, vd, _i32(parents))
        last = [rng.randrange(T) for _ in range(B)]
        paths = [lines_of(p)[i][::-1] for p, i in zip(parents, last)]  # from the root down
        layer.tree_commit(kd, vd, _i32([(p + [0] * T)[:T] for p in paths]), _i32([len(p) for p in paths]))
        at = torch.arange(B, device="cuda"), torch.tensor(last, device="cuda")
        o, l = layer.attention(q[at].contiguous())
        torch.cuda.synchronize()
        # two results of the same attention, each with the roundings that assert_tree_close counts
        tol = {"bf16": 2 * 3 * 2.0 ** -8, "e4m3": 2 * 2.5 * 2.0 ** -8, "f32": 3e-4}[pages]
        assert (out[at].double() - o.double()).abs().max() <= tol * 4.5  # |v| of 12800 normals stays below 4.5
        assert (lse[at] - l).abs().max() <= (6e-4 if pages != "f32" else 1.4e-4)
        layer.reorder(_i32([rng.randrange(B) for _ in range(B)]))
    assert layer.device_status() == 0


def test_captured_round_of_drafting():
    """Tree attention, commit and reorder in one graph, replayed as the cache grows, next to an eager twin."""
    B, T, d = 3, 9, 128
    a, b = (_layer("bf16", 64, d, (120,) * B) for _ in range(2))
    for x in (a, b):
        x.k_pool.zero_(), x.v_pool.zero_()
        _build(x)
        x.prepare_tree(T)
    q, kd, vd = _normal(a, B, T, 10, d), _normal(a, B, T, 5, d, seed=1), _normal(a, B, T, 5, d, seed=2)
    par, path, n, parents = _i32([[-1, 0, 0, 1, 1, 2, 3, 3, 5]] * B), _i32([[0, 1, 3, 7]] * B), _i32([0] * B), \
        _i32([0] * B)
    out, lse = torch.zeros_like(q), torch.zeros(B, T, 10, device="cuda")

    def step(x, out, lse):
        x.tree_attention(q, kd, vd, par, out=out, lse=lse)
        x.tree_commit(kd, vd, path, n)
        x.reorder(parents)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(a, out, lse)
    rng = random.Random(3)
    for i in range(8):
        for t, s in ((q, 70), (kd, 80), (vd, 90)):
            t.copy_(_normal(a, *t.shape, seed=s + i))
        n.copy_(_i32([rng.randint(0, 4) for _ in range(B)]))
        parents.copy_(_i32([rng.randrange(B) for _ in range(B)]))
        graph.replay()
        torch.cuda.synchronize()
        o, l = torch.zeros_like(out), torch.zeros_like(lse)
        step(b, o, l)
        _same(a, b)
        assert torch.equal(out, o) and torch.equal(lse, l)
    assert a.device_status() == 0 and b.device_status() == 0
