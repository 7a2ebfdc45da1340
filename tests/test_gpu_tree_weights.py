"""Tree attention over E4M3 pages where small softmax weights carry the result."""
from __future__ import annotations

import math

import pytest
import torch

from head_aware_paged_build_b200 import segpaged as S
from test_gpu_tree import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    S.load()


@pytest.mark.parametrize("log2_below", [10.5, 20.25, 26.5, 29.5])
@pytest.mark.parametrize("d,g,T", [(128, 4, 3), (64, 4, 3), (128, 4, 8), (64, 4, 8), (128, 8, 16), (64, 8, 16),
                                   (128, 8, 40), (64, 8, 40)])
def test_small_weights_beside_a_dominant_key(log2_below, d, g, T):
    """Every 16th key has a score `log2_below` powers of two above the others and a value of zero, the others a
    value of one: the result is the others' share alone.

    A weight is rounded to f16 when it is 2^7 times its share of the running maximum, which the row's own maximum
    M is never below: by 2^-11 of itself, or by half an f16 subnormal step, 2^-25, which is 2^-32 at the scale of
    the maximum.  So beyond the relative roundings (weights 2^-11; result 2^-8; 6e-4 of the mean of |v| for scores,
    exponentials and sums) the result is off by at most 2^-32 sum |v_j| / sum 2^(s_j - M)."""
    c = Case("e4m3", d, g, T, (2400, 1100), policy=[("global", 0, 0), ("local", 4, 900)], hkv=2)
    c.k.zero_()
    c.k[:, :, ::16, 0] = 1
    c.v.fill_(1)
    c.v[:, :, ::16] = 0
    c.q.zero_()
    c.q[..., 0] = 1
    c.kd.zero_()
    c.vd.fill_(1)
    stored = (torch.tensor(1.0 / 0.01).to(torch.float8_e4m3fn).float() * 0.01).item()
    c.scale = log2_below * math.log(2) / stored
    c.layer.build(c.k, c.v)
    out, lse = c.call()
    torch.cuda.synchronize()
    assert c.layer.device_status() == 0
    ref, lse_ref, mag = c.reference()
    # sum 2^(s_j - M) from the reference's log-sum-exp: M is the dominant keys' score
    total = torch.exp(lse_ref - c.scale * stored)
    others = mag * total[..., None]  # sum |v_j| 2^(s_j - M)
    count = others * 2.0 ** log2_below  # sum |v_j| over the keys that a row sees
    bound = (2.0 ** -11 * 1.01 + 2.0 ** -8 * 1.01 + 6e-4) * mag + 2.0 ** -32 * count / total[..., None]
    worst = ((out.double() - ref).abs() / bound).max().item()
    assert worst <= 1, worst
    # the sums are of unrounded weights
    assert (lse.double() - lse_ref).abs().max() <= 3e-4
