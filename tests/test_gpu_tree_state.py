"""Workspaces of tree attention: what a layer keeps, resets and shares with others."""
from __future__ import annotations

import pytest
import torch

from head_aware_paged_build_b200 import segpaged as S
from test_gpu_tree import MIXED, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    S.load()


def _short_case(**kw):
    """A call that joins its split rows by counters in the workspace."""
    return Case("bf16", 128, 2, 8, (1500, 700), hkv=2, policy=MIXED[:2], **kw)


def test_clearing_the_status_makes_the_workspaces_fresh():
    """What a wait that ran out leaves behind: a status code, and counters that were not returned to zero."""
    c = _short_case()
    want = [x.clone() for x in c.call()]
    attended = [x.clone() for x in c.layer.attention(c.q[:, 0].contiguous())]
    torch.cuda.synchronize()
    for ws in (c.layer.workspace, *c.layer.tree_workspaces):
        ws.view(torch.int32)[:6000].fill_(1)
    assert c.layer.device_status() == 1
    c.layer.clear_device_status()
    assert c.layer.device_status() == 0
    for _ in range(3):
        got = c.call()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        got = c.layer.attention(c.q[:, 0].contiguous())
        assert all(torch.equal(x, y) for x, y in zip(got, attended))
    assert c.layer.device_status() == 0


def test_clearing_the_status_on_a_stream():
    c = _short_case()
    want = [x.clone() for x in c.call()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        c.layer.tree_workspaces[-1].view(torch.int32)[:6000].fill_(1)
        side.wait_stream(torch.cuda.current_stream())
        c.layer.clear_device_status(stream=stream)
        got = c.call(stream=side)
        side.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert c.layer.device_status() == 0


def test_trees_that_need_no_more_bytes_keep_their_workspace():
    layer = Case("bf16", 128, 8, 3, (500, 5), hkv=2, policy=MIXED[:2]).layer
    for n in (20, 33, 48, 64, 17, 64):  # 256 rows a group from 32 nodes on
        layer.prepare_tree(n)
        assert layer.tree_workspaces[-1].numel() >= S.segpaged_tree_workspace(layer.plan, n)
    assert len(layer.tree_workspaces) == 1
    with torch.cuda.graph(torch.cuda.CUDAGraph()):
        layer.prepare_tree(64)  # nothing to allocate
        torch.zeros(1, device="cuda")


@pytest.mark.parametrize("pages", ["bf16", "e4m3", "f32"])
def test_layers_of_a_model_share_a_workspace(pages):
    """Layers of other shapes, short calls and split ones, one after another on one workspace."""
    cases = [Case(pages, 128, 2, 8, (1500, 700), hkv=2, policy=MIXED[:2], seed=1),
             Case(pages, 64, 4, 16, (9000, 3), hkv=3, policy=MIXED[:3], seed=2),
             Case(pages, 128, 2, 8, (70, 2000), hkv=2, policy=MIXED[:2], seed=3)]
    want = [[x.clone() for x in c.call()] for c in cases]
    need = max(S.segpaged_tree_workspace(c.layer.plan, 16) for c in cases)
    shared = torch.zeros(need, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for c in cases:
        c.layer.prepare_tree(16, workspace=shared)
        c.layer.prepare_tree(16, workspace=shared)
        assert c.layer.tree_workspaces[-1] is shared and c.layer.tree_nodes == 16
        c.layer.prepare_tree(9)
        assert c.layer.tree_workspaces[-1] is shared
    for _ in range(5):
        for c, w in zip(cases, want):
            assert all(torch.equal(x, y) for x, y in zip(c.call(), w))
    assert all(c.layer.device_status() == 0 for c in cases)
    cases[0].layer.prepare_tree(64)  # more than it covers: one of its own
    assert cases[0].layer.tree_workspaces[-1].numel() >= S.segpaged_tree_workspace(cases[0].layer.plan, 64)
