"""Argument checks of tree attention, tree commit and reorder (host only: nothing is launched)."""
from __future__ import annotations

import ctypes

import pytest
import torch

from head_aware_paged_build_b200 import segpaged as S
from test_runtime_checks import fake_layer

P = 4096  # a non-NULL, aligned address that no check reads


def _plan(dtype="bf16", ring=True, q_start=None, batch=2, hq=8, hkv=2, d=128, ctx=(100, 70), flags=0, **kw):
    pol = [("global", 0, 0), ("local", 4, 32)] * (batch * hkv // 2)
    q0 = [n - 1 for n in ctx] if q_start is None else q_start
    if ring:
        kw.setdefault("append_capacity", 8)
    return S.segpaged_plan_create(S.make_problem(batch, hq, hkv, d, 64 if dtype == "bf16" else 16, dtype, ctx, q0,
                                                 pol, flags=flags | (S.SP_FLAG_RING if ring else 0), **kw))


def _raises(code, fn, *args):
    with pytest.raises(S.SegPagedError) as e:
        fn(*args)
    assert e.value.status == code, e.value


@pytest.mark.parametrize("dtype,hq", [("bf16", 8), ("bf16", 2), ("bf16", 32), ("f32", 4)])
def test_workspace_covers_every_smaller_tree(dtype, hq):
    plan = _plan(dtype, hq=hq)
    need = [S.segpaged_tree_workspace(plan, n) for n in range(1, 65)]
    assert need == sorted(need) and all(n % 256 == 0 and n > 256 for n in need)
    S.segpaged_plan_destroy(plan)


def test_tree_attention_refusals():
    plan = _plan()
    ws = S.segpaged_tree_workspace(plan, 8)

    def args(**change):
        a = dict(plan=plan, table=P, k=P, v=P, q=P, kd=P, vd=P, ss=2048, st=256, sh=128, par=P, num=None, nodes=8,
                 out=P, lse=P, scale=0.0, ws=P, wb=ws, stream=0)
        a.update(change)
        return list(a.values())

    for change in (dict(table=None), dict(table=P + 4), dict(k=None), dict(v=P + 8), dict(q=None), dict(q=P + 2),
                   dict(kd=None), dict(vd=P + 8), dict(ss=-128), dict(st=4), dict(sh=7), dict(par=None),
                   dict(par=P + 2), dict(num=P + 1), dict(nodes=0), dict(nodes=-3), dict(out=None), dict(lse=P + 2),
                   dict(scale=float("nan")), dict(scale=float("inf")), dict(ws=None), dict(ws=P + 128),
                   dict(plan=None)):
        _raises(S.SP_ERR_INVALID_ARG, S.segpaged_tree_attention, *args(**change))
    _raises(S.SP_ERR_UNSUPPORTED, S.segpaged_tree_attention, *args(nodes=65))
    _raises(S.SP_ERR_WORKSPACE, S.segpaged_tree_attention, *args(wb=1024))
    _raises(S.SP_ERR_UNSUPPORTED, S.segpaged_tree_workspace, plan, 65)
    _raises(S.SP_ERR_INVALID_ARG, S.segpaged_tree_workspace, plan, 0)
    assert S.load().segpaged_tree_workspace(plan, 8, None) == S.SP_ERR_INVALID_ARG
    S.segpaged_plan_destroy(plan)
    prefill = _plan(ring=False, q_start=[0, 0])
    _raises(S.SP_ERR_INVALID_ARG, S.segpaged_tree_workspace, prefill, 8)
    _raises(S.SP_ERR_INVALID_ARG, S.segpaged_tree_attention, *args(plan=prefill))
    S.segpaged_plan_destroy(prefill)


def test_tree_commit_refusals():
    plan = _plan()

    def args(**change):
        a = dict(plan=plan, table=P, kd=P, vd=P, ss=2048, st=256, sh=128, nodes=8, path=P, path_len=P, max_path=4,
                 k=P, v=P, ws=P, stream=0)
        a.update(change)
        return list(a.values())

    for change in (dict(table=None), dict(kd=None), dict(vd=P + 4), dict(ss=-8), dict(st=4), dict(nodes=0),
                   dict(path=None), dict(path=P + 2), dict(path_len=None), dict(path_len=P + 3), dict(max_path=0),
                   dict(k=None), dict(v=P + 8), dict(ws=None), dict(ws=P + 64), dict(plan=None)):
        _raises(S.SP_ERR_INVALID_ARG, S.segpaged_tree_commit, *args(**change))
    _raises(S.SP_ERR_UNSUPPORTED, S.segpaged_tree_commit, *args(nodes=65))
    _raises(S.SP_ERR_UNSUPPORTED, S.segpaged_tree_commit, *args(max_path=65))
    S.segpaged_plan_destroy(plan)
    fixed = _plan(ring=False)
    _raises(S.SP_ERR_INVALID_ARG, S.segpaged_tree_commit, *args(plan=fixed))
    S.segpaged_plan_destroy(fixed)


def test_reorder_refusals():
    plan = _plan()

    def args(**change):
        a = dict(plan=plan, table=P, parents=P, common=None, k=P, v=P, ws=P, stream=0)
        a.update(change)
        return list(a.values())

    for change in (dict(table=None), dict(parents=None), dict(parents=P + 2), dict(common=P + 1), dict(k=None),
                   dict(v=P + 8), dict(ws=None), dict(ws=P + 32), dict(plan=None)):
        _raises(S.SP_ERR_INVALID_ARG, S.segpaged_reorder, *args(**change))
    S.segpaged_plan_destroy(plan)
    fixed = _plan(ring=False)
    _raises(S.SP_ERR_INVALID_ARG, S.segpaged_reorder, *args(plan=fixed))
    S.segpaged_plan_destroy(fixed)
    many = S.segpaged_plan_create(S.make_problem(2049, 1, 1, 64, 16, "f32", [1] * 2049, [0] * 2049,
                                                 [("global", 0, 0)] * 2049, flags=S.SP_FLAG_RING, append_capacity=1))
    _raises(S.SP_ERR_UNSUPPORTED, S.segpaged_reorder, *args(plan=many))
    S.segpaged_plan_destroy(many)


def _bf16(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def _i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


@pytest.mark.parametrize("change,error", [
    (dict(q=_bf16(2, 8, 4, 64)), ValueError), (dict(q=_bf16(3, 8, 4, 128)), ValueError),
    (dict(q=_bf16(2, 65, 4, 128)), ValueError), (dict(q=_bf16(2, 0, 4, 128)), ValueError),
    (dict(q=_bf16(2, 4, 8, 128).transpose(1, 2)), ValueError), (dict(q=_bf16(2, 8, 4, 128).float()), TypeError),
    (dict(k=_bf16(2, 7, 2, 128)), ValueError), (dict(v=_bf16(2, 8, 2, 64)), ValueError),
    (dict(k=_bf16(2, 2, 8, 128).transpose(1, 2)), ValueError), (dict(v=_bf16(2, 8, 2, 128).float()), TypeError),
    (dict(k=_bf16(2, 8, 2, 256)[..., ::2], v=_bf16(2, 8, 2, 256)[..., ::2]), ValueError),
    (dict(parents=_i32(2, 7)), ValueError), (dict(parents=_i32(2, 8).long()), TypeError),
    (dict(parents=_i32(8, 2).t()), ValueError), (dict(num=_i32(3)), ValueError), (dict(num=[8, 8]), TypeError)])
def test_layer_refuses_tree_tensors_that_do_not_fit(change, error):
    a = dict(q=_bf16(2, 8, 4, 128), k=_bf16(2, 8, 2, 128), v=_bf16(2, 8, 2, 128), parents=_i32(2, 8), num=_i32(2))
    a.update(change)
    with pytest.raises(error):
        fake_layer().tree_attention(a["q"], a["k"], a["v"], a["parents"], a["num"])


@pytest.mark.parametrize("change,error", [
    (dict(k=_bf16(2, 8, 2, 64)), ValueError), (dict(k=None), ValueError), (dict(v=_bf16(2, 7, 2, 128)), ValueError),
    (dict(path=_i32(3, 4)), ValueError), (dict(path=_i32(2)), ValueError), (dict(path=_i32(4, 2).t()), ValueError),
    (dict(path=_i32(2, 4).long()), TypeError), (dict(n=_i32(3)), ValueError), (dict(n=2), TypeError)])
def test_layer_refuses_commit_tensors_that_do_not_fit(change, error):
    a = dict(k=_bf16(2, 8, 2, 128), v=_bf16(2, 8, 2, 128), path=_i32(2, 4), n=_i32(2))
    a.update(change)
    with pytest.raises(error):
        fake_layer().tree_commit(a["k"], a["v"], a["path"], a["n"])


@pytest.mark.parametrize("parents,common,error", [
    (_i32(3), None, ValueError), (_i32(2).long(), None, TypeError), ([0, 1], None, TypeError),
    (_i32(2), _i32(1), ValueError), (_i32(2), _i32(2).float(), TypeError)])
def test_layer_refuses_reorder_tensors_that_do_not_fit(parents, common, error):
    with pytest.raises(error):
        fake_layer().reorder(parents, common)
