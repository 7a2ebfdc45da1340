"""Tree attention on RETRIEVAL heads: kept blocks stay visible where the window has moved past them."""
from __future__ import annotations

import random

import pytest
import torch

from head_aware_paged_build_b200 import segpaged as S
from head_aware_paged_build_b200 import workloads as W
from head_aware_paged_build_b200.runtime import layer_for
from _parity import assert_close, compare
from test_gpu_tree import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    S.load()


def _retrieval_case(pages, d, g, T, lens, heads, page=64, shape="random", seed=0, **kw):
    """heads: (sink, window, one set of kept blocks for each sequence) of each kv-head, or a policy of another kind."""
    policy, masses, kept = [], [], {}
    for b, L in enumerate(lens):
        for h, head in enumerate(heads):
            if isinstance(head[0], str):
                policy.append(head), masses.append(None)
                continue
            sink, window, sets = head
            blocks = {i for i in sets[b] if (i + 1) * page > sink and i * page < L}
            policy.append(("retrieval", sink, window, 0.9999))
            masses.append([1.0 if i in blocks else 0.0 for i in range(-(-L // page))])
            kept[(b, h)] = torch.tensor([j // page in blocks for j in range(L)])
    case = Case(pages, d, g, T, lens, policy=policy, hkv=len(heads), page=page, ring=False, shape=shape, seed=seed,
                block_mass=masses, **kw)
    return case, kept


# window and context on and off page boundaries, the newest block kept and not, a kept block that the sink reaches into
HEADS = [(4, 320, [set(range(10)), {1, 2}, {0, 1, 2, 3}]),
         (4, 300, [{6}, {2}, {4}]),
         (0, 128, [{8, 9}, {3}, {0, 10}]),
         (130, 64, [{2, 7, 10}, {4}, {9, 11}]),
         ("local", 4, 40),
         (4, 1, [{10, 5}, {0, 1, 2, 3, 4}, set()])]


@pytest.mark.parametrize("pages,d", [("bf16", 128), ("bf16", 64), ("e4m3", 128), ("f32", 64)])
@pytest.mark.parametrize("g,T", [(1, 13), (4, 8), (4, 32), (8, 33)])
def test_kept_blocks_next_to_the_window(pages, d, g, T):
    case, kept = _retrieval_case(pages, d, g, T, (704, 320, 768), HEADS)
    case.check(kept)
    case, kept = _retrieval_case(pages, d, g, T, (700, 259, 705), HEADS, counts=[T, T // 2, 1])
    case.check(kept)


@pytest.mark.parametrize("pages", ["bf16", "e4m3", "f32"])
def test_a_chain_moves_the_window_past_kept_blocks(pages):
    """64 nodes in a line: the last one's window starts 63 positions further on, inside or behind a kept block."""
    case, kept = _retrieval_case(pages, 128, 2, 64, (704, 320, 768), HEADS, shape="chain")
    case.check(kept)


@pytest.mark.parametrize("pages,page", [("bf16", 64), ("e4m3", 64), ("f32", 16)])
@pytest.mark.parametrize("flags", [0, S.SP_FLAG_DENSE_MASKED])
def test_random_kept_blocks(pages, page, flags):
    rng = random.Random(page + flags)
    for seed in range(4):
        lens = [rng.randint(1, 900) for _ in range(3)]
        heads = [(rng.choice([0, 4, 70, 130]), rng.randint(1, 700),
                  [{i for i in range(-(-L // page)) if rng.random() < 0.5} for L in lens]) for _ in range(4)]
        case, kept = _retrieval_case(pages, 64, 3, 17, lens, heads, page=page, seed=seed, flags=flags)
        case.check(kept)


@pytest.mark.parametrize("dtype,page", [("bf16", 64), ("f32", 16)])
def test_prefill_of_one_query_next_to_others(dtype, page):
    """A sequence with one query in a batch of longer ones: its kept blocks next to the window are seen too."""
    lens = (700, 768, 701)
    pol = [("retrieval", 4, 300, 0.5), ("retrieval", 4, 128, 0.9)] * 3
    prob = W.Problem(W.custom("one_query", 71, 3, 4, 2, 64, dtype, page, lens, pol), lens, (699, 768 - 90, 700))
    k, v = W.dense_kv(prob, device="cpu")
    q = W.queries(prob, device="cpu")
    layer = layer_for(prob)
    layer.build(k.cuda(), v.cuda())
    out, lse = layer.attention(q.cuda())
    torch.cuda.synchronize()
    assert layer.device_status() == 0
    assert_close(compare(prob, q, k, v, out, lse), dtype)
