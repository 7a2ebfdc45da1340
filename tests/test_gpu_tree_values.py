"""Draft, attend, accept, commit, fork, decode: every result element by element against the fp64 form over dense K/V."""
from __future__ import annotations

import random

import pytest
import torch

from head_aware_paged_build_b200 import segpaged as S
from _tree import assert_tree_close, lines_of, random_tree, tree_reference
from test_gpu_tree_cache import KINDS, _build, _i32, _layer, _normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    S.load()


def _stored(x, pages, scale):
    if pages != "e4m3":
        return x
    scale = torch.tensor(scale, dtype=torch.float32, device="cuda")
    return (x.float() * (1 / scale)).clamp(-448, 448).to(torch.float8_e4m3fn).double() * scale.double()


@pytest.mark.parametrize("pages,page", [("bf16", 64), ("e4m3", 64), ("f32", 16)])
@pytest.mark.parametrize("g,T", [(1, 12), (4, 12)])
def test_committed_rows_are_attended_as_given(pages, page, g, T):
    """A wrong row or order of the draft, of a commit or of a fork moves the result by a share of its own weight in
    the row, which the bound (relative to the weighted mean of |v|) does not allow for on windows this narrow."""
    B, d, lens = 4, 128, [90] * 4
    layer = _layer(pages, page, d, lens, g=g)
    k, v = _build(layer)
    room = torch.zeros(B, 5, 70, d, dtype=k.dtype, device="cuda")
    k, v = torch.cat([k, room], 2), torch.cat([v, room], 2)  # as given: quantised where it is read
    policy, rng = list(KINDS) * B, random.Random(6)
    for step in range(5):
        q = _normal(layer, B, T, 5 * g, d, seed=20 + step)
        kd, vd = (_normal(layer, B, T, 5, d, seed=s + step) for s in (40, 60))
        parents = [random_tree(rng, T, "random") for _ in range(B)]
        out, lse = layer.tree_attention(q, kd, vd, _i32(parents))
        dense = [_stored(x, pages, s) for x, s in ((kd, 0.01), (vd, 0.02), (k, 0.01), (v, 0.02))]
        ref = tree_reference(q, *dense, lens, parents, [T] * B, policy)
        assert_tree_close(out, lse, ref, pages)
        last = [rng.randrange(T) for _ in range(B)]
        paths = [lines_of(p)[i][::-1] for p, i in zip(parents, last)]  # from the root down
        layer.tree_commit(kd, vd, _i32([(p + [0] * T)[:T] for p in paths]), _i32([len(p) for p in paths]))
        for b, path in enumerate(paths):
            for x, rows in ((k, kd), (v, vd)):
                x[b, :, lens[b]:lens[b] + len(path)] = rows[b, path].transpose(0, 1)
            lens[b] += len(path)
        at = torch.arange(B, device="cuda"), torch.tensor(last, device="cuda")
        o, l = layer.attention(q[at].contiguous())  # the accepted node's result, over the cache alone
        torch.cuda.synchronize()
        assert_tree_close(o, l, tuple(x[at] for x in ref), pages)
        forks = [rng.randrange(B) for _ in range(B)]
        layer.reorder(_i32(forks))
        k, v, lens = k[forks], v[forks], [lens[b] for b in forks]
    assert layer.device_status() == 0
