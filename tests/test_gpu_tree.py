"""Tree attention on the GPU against its plain fp64 form."""
from __future__ import annotations

import random

import pytest
import torch

from head_aware_paged_build_b200 import segpaged as S
from head_aware_paged_build_b200.runtime import SegPagedLayer
from _table import BAD_PAGE, corrupt
from _tree import assert_tree_close, random_tree, tree_reference

pytestmark = pytest.mark.gpu

MIXED = [("global", 0, 0), ("local", 4, 40), ("local", 0, 1), ("local", 130, 64), ("dense", 0, 0),
         ("local", 300, 10)]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    S.load()


class Case:
    """A layer, its dense K/V, a draft (K and V rows in one packed tensor) and a forest a sequence."""

    def __init__(self, pages, d, g, T, lens, counts=None, policy=MIXED, hkv=6, page=64, shape="random", ring=True,
                 flags=0, seed=0, scale=0.0, **kw):
        gen = torch.Generator(device="cuda").manual_seed(seed + 977 * T + g)
        rng = random.Random(seed)
        B, hq = len(lens), hkv * g
        dtype = "f32" if pages == "f32" else "bf16"
        el = torch.float32 if dtype == "f32" else torch.bfloat16
        self.pages, self.scale, self.lens = pages, scale, list(lens)
        self.counts = [T] * B if counts is None else list(counts)
        self.policy = (list(policy) * hkv)[:hkv] * B if len(policy) != B * hkv else list(policy)

        def normal(*s):
            return torch.randn(*s, generator=gen, device="cuda", dtype=el)

        self.k, self.v = normal(B, hkv, max(lens), d), normal(B, hkv, max(lens), d)
        self.q = normal(B, T, hq, d)
        packed = normal(B, T, 2, hkv, d)
        if pages == "e4m3":
            kw.update(kv_dtype="e4m3", k_scale=0.01, v_scale=0.02)
        if ring:
            kw.setdefault("append_capacity", 70)
            flags |= S.SP_FLAG_RING
        self.layer = SegPagedLayer(batch=B, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, page_size=page,
                                   dtype=dtype, ctx_len=lens, q_start=[n - 1 for n in lens], policy=self.policy,
                                   flags=flags, **kw)
        self.layer.build(self.k, self.v)
        self.parents = [random_tree(rng, n, shape) + [0] * (T - n) for n in self.counts]
        for b, n in enumerate(self.counts):  # rows behind a draft are never read
            self.q[b, n:] = float("nan")
            packed[b, n:] = float("nan")
            self.parents[b][n:] = [1000] * (T - n)
        self.kd, self.vd = packed[:, :, 0], packed[:, :, 1]
        self.par = torch.tensor(self.parents, dtype=torch.int32, device="cuda").view(B, T)
        self.num = None if counts is None else torch.tensor(self.counts, dtype=torch.int32, device="cuda")

    def call(self, **kw):
        return self.layer.tree_attention(self.q, self.kd, self.vd, self.par, num_nodes=self.num, scale=self.scale,
                                         **kw)

    def reference(self, kept=None):
        k, v, kd, vd = self.k, self.v, self.kd, self.vd
        if self.pages == "e4m3":
            def stored(x, s):
                inv = torch.tensor(1.0, device="cuda") / torch.tensor(s, dtype=torch.float32, device="cuda")
                codes = (x.float() * inv).clamp(-448, 448).to(torch.float8_e4m3fn)
                return codes.double() * torch.tensor(s, dtype=torch.float32, device="cuda").double()
            k, v, kd, vd = stored(k, 0.01), stored(v, 0.02), stored(kd, 0.01), stored(vd, 0.02)
        return tree_reference(self.q, kd, vd, k, v, self.lens, self.parents, self.counts, self.policy,
                              self.scale or None, kept)

    def check(self, kept=None):
        out, lse = torch.full_like(self.q, 7.0), torch.full(self.q.shape[:3], 7.0, device="cuda")
        self.call(out=out, lse=lse)
        torch.cuda.synchronize()
        assert self.layer.device_status() == 0
        for b, n in enumerate(self.counts):
            assert bool((out[b, n:] == 7).all()) and bool((lse[b, n:] == 7).all()), "rows behind the draft"
            out[b, n:], lse[b, n:] = 0, 0
        assert_tree_close(out, lse, self.reference(kept), self.pages)


LENS, COUNTS = (1, 63, 64, 65, 200, 700), (13, 1, 0, 7, 13, 12)


@pytest.mark.parametrize("g", [1, 2, 3, 5, 8, 16])
@pytest.mark.parametrize("pages,d", [("bf16", 128), ("bf16", 64), ("e4m3", 128), ("e4m3", 64), ("f32", 64)])
def test_ragged_forests(pages, d, g):
    Case(pages, d, g, 13, LENS, COUNTS).check()


@pytest.mark.parametrize("pages,d,page", [("f32", 128, 16), ("f32", 64, 16), ("f32", 128, 64)])
def test_fp32_page_sizes(pages, d, page):
    Case(pages, d, 3, 21, LENS, (21, 1, 0, 17, 16, 20), page=page).check()


@pytest.mark.parametrize("pages", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("T,g", [(1, 1), (1, 16), (2, 8), (3, 8), (4, 8), (5, 8), (8, 4), (9, 4), (16, 8), (17, 8),
                                 (33, 4), (64, 1), (64, 2), (64, 3), (64, 16)])
def test_row_counts(pages, T, g):
    """One row to 1024 a kv-head: every row tile, and the sizes on both sides of each."""
    Case(pages, 128, g, T, (70, 130), hkv=2, policy=[("global", 0, 0), ("local", 4, 20)]).check()


@pytest.mark.parametrize("pages", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("shape", ["chain", "roots"])
def test_windows_narrower_than_the_draft(pages, shape):
    """A chain of 64 nodes moves a window of 40, 1 and 10 tokens past the cached ones."""
    Case(pages, 128, 2, 64, (5, 100, 333), shape=shape).check()


@pytest.mark.parametrize("ring,flags", [(False, 0), (False, S.SP_FLAG_DENSE_MASKED)])
@pytest.mark.parametrize("pages", ["bf16", "e4m3", "f32"])
def test_plans_without_a_ring(pages, ring, flags):
    Case(pages, 128, 4, 9, LENS, (9, 1, 0, 7, 9, 8), ring=ring, flags=flags).check()


def test_retrieval_heads_see_their_kept_blocks():
    lens, hkv = (700, 130), 2
    policy = [("retrieval", 4, 40, 0.6), ("local", 4, 40)] * 2
    masses, kept = [], {}
    rng = random.Random(3)
    for b, L in enumerate(lens):
        m = [rng.random() for _ in range(-(-L // 64))]
        order = sorted(range(len(m)), key=lambda i: -m[i])
        sel, total = [], 0.0
        while total < 0.6 * sum(m):
            sel.append(order[len(sel)])
            total += m[sel[-1]]
        see = torch.zeros(L, dtype=torch.bool)
        for i in sel:
            see[i * 64:(i + 1) * 64] = True
        kept[(b, 0)] = see
        masses += [m, None]
    Case("bf16", 128, 4, 11, lens, policy=policy, hkv=hkv, ring=False, block_mass=masses).check(kept)


@pytest.mark.parametrize("pages,T,g", [("bf16", 16, 8), ("bf16", 5, 2), ("bf16", 40, 8), ("e4m3", 16, 8)])
def test_a_long_context_is_split_over_many_ctas(pages, T, g):
    Case(pages, 128, g, T, (70001, 1, 3000), hkv=2, policy=[("global", 0, 0), ("local", 4, 8000)]).check()


@pytest.mark.parametrize("pages,d,T,g", [("bf16", 128, 40, 8), ("bf16", 64, 40, 8), ("e4m3", 128, 40, 8),
                                         ("e4m3", 64, 40, 8), ("bf16", 128, 13, 8), ("e4m3", 128, 13, 8)])
def test_pieces_of_one_and_two_tiles_repeat_bit_for_bit(pages, d, T, g):
    """A CTA's pieces alternate between one and two query tiles and between odd and even numbers of pages: a
    barrier that a role passes a phase early shows as another call's bits."""
    lens = [40001, 1, 700, 129, 9000, 64, 20011, 333]
    counts = [T, T, 1, T, T // 2, T, T - 3, 5]
    case = Case(pages, d, g, T, lens, counts, hkv=3, policy=[("global", 0, 0), ("local", 4, 3000), ("local", 1, 70)])
    case.check()
    first = None
    for turn in range(200):
        now = torch.zeros_like(case.q), torch.zeros(case.q.shape[:3], device="cuda")
        case.call(out=now[0], lse=now[1])
        first = first or now
        assert all(torch.equal(x, y) for x, y in zip(now, first)), turn
    assert case.layer.device_status() == 0


@pytest.mark.parametrize("pages,d", [("bf16", 128), ("e4m3", 64), ("f32", 128)])
def test_short_calls_of_changing_sizes_share_a_workspace(pages, d):
    """Few heads over few pages join their pieces by counters that one call leaves ready for the next."""
    case = Case(pages, d, 2, 16, (1500, 700), hkv=4, policy=[("global", 0, 0), ("local", 4, 600)])
    case.check()
    ones = torch.full((2,), 1, dtype=torch.int32, device="cuda")
    first = {}
    for turn in range(40):
        for t in (16, 1, 5, 8, 13):
            out, lse = torch.zeros_like(case.q[:, :t]), torch.zeros(2, t, 8, device="cuda")
            case.layer.tree_attention(case.q[:, :t].contiguous(), case.kd[:, :t].contiguous(),
                                      case.vd[:, :t].contiguous(), case.par[:, :t].contiguous(),
                                      num_nodes=ones * min(t, 1 + turn % 3), out=out, lse=lse)
            o, l = first.setdefault((t, turn % 3), (out, lse))
            assert torch.equal(o, out) and torch.equal(l, lse), (turn, t)
    assert case.layer.device_status() == 0
    want = case.call()[0]
    for t in (5, 13):  # a node's result does not depend on the nodes behind it
        out = case.layer.tree_attention(case.q[:, :t].contiguous(), case.kd[:, :t].contiguous(),
                                        case.vd[:, :t].contiguous(), case.par[:, :t].contiguous())[0]
        tol = 1e-5 if pages == "f32" else 2e-2
        assert torch.allclose(out.float(), want[:, :t].float(), rtol=tol, atol=tol)


def test_more_heads_than_threads():
    lens = [random.Random(5).randint(1, 200) for _ in range(70)]
    Case("bf16", 64, 2, 6, lens, [n % 7 for n in lens], hkv=9).check()


@pytest.mark.parametrize("pages,g", [("bf16", 2), ("bf16", 5), ("e4m3", 2), ("e4m3", 5), ("f32", 5)])
def test_heads_of_a_page_or_two(pages, g):
    """Hundreds of tiny heads: the split leaves pieces of a single page, where one softmax stream has none."""
    rng = random.Random(11)
    for T in (13, 40):
        lens = [rng.choice([1, 5, 64, 65, 130]) for _ in range(50)]
        Case(pages, 128, g, T, lens, [rng.randint(0, T) for _ in lens], policy=MIXED[:3], hkv=3).check()


def test_layers_on_two_streams_at_once():
    cases = [Case(pages, 128, 4, 16, (3000, 500), hkv=2, policy=MIXED[:2], seed=i)
             for i, pages in enumerate(("bf16", "e4m3"))]
    want = [[x.clone() for x in c.call()] for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[c.call(stream=s) for c, s in zip(cases, streams)] for _ in range(20)]
    torch.cuda.synchronize()
    for turn in got:
        for (o, l), (wo, wl) in zip(turn, want):
            assert torch.equal(o, wo) and torch.equal(l, wl)


def test_sharp_scores_move_the_running_maximum():
    """Scores of a few hundred: the maximum grows from page to page, many weights underflow."""
    c = Case("bf16", 128, 4, 12, (1000, 333), hkv=2, policy=MIXED[:2], scale=2.0)
    out, lse = c.call()
    o, l, mag = c.reference()
    # score error 23 times that of the default scale; the rest of the bound as in assert_tree_close
    assert ((out.double() - o).abs() - (2.0 ** -7 * mag + 23 * 6e-4 * mag)).max() <= 0
    assert (lse.double() - l).abs().max() <= 23 * 3e-4


def test_pages_behind_the_first_4_gb_of_a_pool():
    nbytes = (300000 + 400) * 64 * 128 * 2
    pools = tuple(torch.empty(nbytes, dtype=torch.uint8, device="cuda") for _ in range(2))
    Case("bf16", 128, 4, 9, (1000, 65), hkv=2, policy=MIXED[:2], first_page=300000, pools=pools).check()


@pytest.mark.parametrize("pages", ["bf16", "e4m3", "f32"])
def test_same_bits_on_every_call_and_stream(pages):
    c = Case(pages, 128, 4, 17, (9000, 40, 1300), hkv=2, policy=MIXED[:2])
    out, lse = [x.clone() for x in c.call()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = c.call(stream=side)
    side.synchronize()
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    raw = c.call(stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(out, raw[0]) and torch.equal(lse, raw[1])


def test_fresh_outputs_are_zero_behind_a_draft():
    c = Case("bf16", 128, 2, 6, (70, 5), (2, 0), hkv=2, policy=MIXED[:2])
    out, lse = c.call()
    assert not out[0, 2:].any() and not out[1].any() and not lse[1].any() and bool(out[0, :2].any())


def test_trees_of_other_sizes_share_a_workspace():
    """Calls of 64, 3 and 64 nodes: the second uses the first one's workspace."""
    big = Case("bf16", 128, 4, 64, (5000, 300), hkv=2, policy=MIXED[:2])
    small = Case("bf16", 128, 4, 3, (5000, 300), hkv=2, policy=MIXED[:2])
    for layer in (big.layer, small.layer):
        layer.prepare_tree(64)
    big.check()
    small.layer.tree_workspaces = big.layer.tree_workspaces
    small.check()
    big.check()
    assert len(big.layer.tree_workspaces) == 1


def test_workspaces_of_growing_trees():
    layer = Case("bf16", 64, 2, 3, (100, 5), hkv=2, policy=MIXED[:2]).layer
    for bad in (0, -1, 65):
        with pytest.raises(S.SegPagedError):
            layer.prepare_tree(bad)
    for n in range(1, 65):
        layer.prepare_tree(n)
        assert layer.tree_nodes >= n
        assert layer.tree_workspaces[-1].numel() >= S.segpaged_tree_workspace(layer.plan, n)
    assert len(layer.tree_workspaces) <= 4


def test_bad_trees_are_reported():
    """A parent at or behind its node counts as a root, a node count out of range as the nearest one in range."""
    c = Case("bf16", 128, 2, 6, (70, 200, 9), (6, 6, 6), hkv=2, policy=MIXED[:2])
    c.par[1, 3] = 3
    c.num[2] = 9
    c.parents[1][3] = -1
    out, lse = c.call()
    torch.cuda.synchronize()
    assert c.layer.device_status() == 8
    assert_tree_close(out, lse, c.reference(), "bf16")


def test_invalid_page_is_reported():
    c = Case("bf16", 128, 2, 6, (70, 200), hkv=2, policy=MIXED[:2])
    corrupt(c.layer, 1, 0, 2)
    c.call()
    torch.cuda.synchronize()
    assert c.layer.device_status() == BAD_PAGE


def test_captured_calls_equal_eager_ones():
    c = Case("bf16", 128, 4, 10, (900, 77), (10, 4), hkv=2, policy=MIXED[:2])
    graph = torch.cuda.CUDAGraph()
    out, lse = torch.zeros_like(c.q), torch.zeros(c.q.shape[:3], device="cuda")
    with pytest.raises(RuntimeError):  # no workspace yet
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            c.call(out=out, lse=lse)
    torch.cuda.synchronize()
    c.layer.prepare_tree(10)
    with torch.cuda.graph(graph):
        c.call(out=out, lse=lse)
    for seed in range(3):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        c.q[0].normal_(generator=gen)
        c.q[1, :4].normal_(generator=gen)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone(), lse.clone()
        want = c.call()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert c.layer.device_status() == 0
