"""The stored runs of RETRIEVAL heads (host logic, CPU only).

Every page of a retrieval head is seen either causally, whatever the window
(kept blocks), or by the local rule (the sink and the window).  A call whose
queries stand behind the plan's last position (drafted tokens) or at several
positions needs that difference, so no run may mix the two.  The sink is seen
either way and may join any run.
"""
from __future__ import annotations

import random

import numpy as np
import pytest

from head_aware_paged_build_b200 import segpaged as S


def _runs(dtype, page, lens, q_start, sink, window, kept):
    """(plan, mask of the positions in kept blocks) of one retrieval head a sequence."""
    masses, seen = [], []
    for L, keep in zip(lens, kept):
        nb = -(-L // page)
        masses.append([1.0 if i in keep else 0.0 for i in range(nb)])
        seen.append(np.isin(np.arange(L) // page, sorted(keep)))
    p = S.make_problem(len(lens), 2, 1, 64, page, dtype, lens, q_start,
                       [("retrieval", sink, window, 0.9999)] * len(lens), block_mass=masses)
    return S.segpaged_plan_create(p), seen


def _check(dtype, page, lens, q_start, sink, window, kept):
    plan, seen = _runs(dtype, page, lens, q_start, sink, window, kept)
    try:
        for b, L in enumerate(lens):
            held = np.zeros(L, bool)
            for start, length, _, _ in S.segpaged_plan_head_segments(plan, b, 0):
                part = seen[b][max(start, sink):start + length]
                assert part.all() or not part.any(), (b, start, length)
                held[start:start + length] = True
            j = np.arange(L)
            assert np.array_equal(held, seen[b] | (j < sink) | (j >= max(sink, q_start[b] - window + 1)))
    finally:
        S.segpaged_plan_destroy(plan)


@pytest.mark.parametrize("L,sink,window,kept", [
    (704, 4, 320, set(range(10))),   # every block but the newest
    (700, 4, 300, {6}),              # the window starts inside the kept block
    (768, 4, 128, {9}),              # the window starts where the kept block ends
    (700, 4, 300, {0, 10}),          # the newest block kept
    (700, 130, 300, {2, 7}),         # a kept block that begins in the sink
    (65, 0, 1, {0}), (64, 4, 64, set())])
def test_kept_blocks_next_to_the_window(L, sink, window, kept):
    _check("bf16", 64, [L], [L - 1], sink, window, [kept])
    _check("bf16", 64, [L, 300], [L - 1, 200], sink, window, [kept, {1}])  # one query next to a hundred


@pytest.mark.parametrize("dtype,page", [("bf16", 64), ("f32", 16)])
def test_random_kept_blocks(dtype, page):
    rng = random.Random(page)
    for _ in range(60):
        lens = [rng.randint(1, 900) for _ in range(3)]
        kept = [{i for i in range(-(-L // page)) if rng.random() < 0.5} for L in lens]
        _check(dtype, page, lens, [L - 1 for L in lens], rng.choice([0, 4, 70, 130]), rng.randint(1, 700), kept)
