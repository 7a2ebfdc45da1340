"""Checks of a tree workspace that the caller gives (host only: nothing is launched)."""
from __future__ import annotations

import pytest
import torch

from head_aware_paged_build_b200 import segpaged as S
from test_runtime_checks import fake_layer


@pytest.fixture
def layer():
    lay = fake_layer()
    lay.plan = S.segpaged_plan_create(S.make_problem(2, 4, 2, 128, 64, "bf16", [100, 70], [99, 69],
                                                     [("global", 0, 0), ("local", 4, 32)] * 2,
                                                     flags=S.SP_FLAG_RING, append_capacity=8))
    lay.tree_workspaces, lay.tree_nodes = [], 0
    yield lay
    S.segpaged_plan_destroy(lay.plan)
    lay.plan = None


def _aligned(n):
    x = torch.zeros(n + 512, dtype=torch.uint8)
    at = -x.data_ptr() % 256
    return x[at:at + n], x[at + 16:at + 16 + n]


def test_a_workspace_is_taken_once(layer):
    need = S.segpaged_tree_workspace(layer.plan, 20)
    ws, _ = _aligned(need)
    for _ in range(2):
        layer.prepare_tree(20, workspace=ws)
        assert layer.tree_nodes == 20 and len(layer.tree_workspaces) == 1 and layer.tree_workspaces[0] is ws
    layer.prepare_tree(3)  # covered
    assert len(layer.tree_workspaces) == 1


def test_workspaces_that_do_not_fit_are_refused(layer):
    need = S.segpaged_tree_workspace(layer.plan, 20)
    ws, off = _aligned(need)
    for bad, error in ((ws[:-1], ValueError), (off, ValueError), (ws.view(torch.int8), TypeError),
                       (need, TypeError), (_aligned(2 * need)[0][::2], ValueError)):
        with pytest.raises(error):
            layer.prepare_tree(20, workspace=bad)
    for nodes in (0, -1, 65):
        with pytest.raises(S.SegPagedError):
            layer.prepare_tree(nodes, workspace=ws)
    assert layer.tree_nodes == 0 and not layer.tree_workspaces
