"""Layer norm: whole rows that hold an infinity, rows whose squares pass fp32's range, values
around the statistics."""
import math

import pytest
import torch

import mixture_experts_routing_gb300 as moe
from test_gpu_norm import KINDS, Rows
from test_gpu_w4 import DEV, ok

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("h", [8, 24, 64, 520, 2056, 7168, 8200, 16384])
@pytest.mark.parametrize("add,bias", [(False, False), (True, True)])
def test_a_row_with_an_infinity_is_nan_throughout(h, kind, add, bias):
    r = Rows(9, h, kind, add=add, bias=bias)
    r.forward()
    ok()
    y, rstd = r.y.clone(), r.rstd.clone()
    r.x[1, h // 2], r.x[3, h - 1], r.x[4, 0], r.x[6, 1] = math.inf, -math.inf, math.inf, math.nan
    bad = [1, 3, 4, 6]
    if add:  # finite values whose sum is not
        r.x[7, 5] = r.add[7, 5] = 3e38
        bad.append(7)
    r.forward()
    ok()
    for t in range(9):
        if t in bad:
            assert r.y[t].isnan().all() and r.rstd[t].isnan(), t
        else:
            assert torch.equal(r.y[t], y[t]) and r.rstd[t] == rstd[t], t


@pytest.mark.parametrize("h", [8, 64, 2056, 8200])
def test_a_row_whose_squares_pass_the_range(h):
    r = Rows(4, h, moe.NORM_RMS, add=False)
    r.x[2] = 1e30
    r.forward()
    ok()
    assert r.rstd[2] == 0 and torch.equal(r.y[2], r.b.to(torch.bfloat16))


@pytest.mark.parametrize("n,h", [(19, 1096), (5, 64), (3, 8200)])
def test_values_behind_the_statistics_are_left(n, h):
    r = Rows(n, h, moe.NORM_LAYER)
    r.forward()
    mean, rstd = (torch.full((n + 16,), 7.0, device=DEV) for _ in range(2))
    moe.norm_forward(r.cfg, r.x, r.w, r.y, bias=r.b, add=r.add, sum=r.sum, mean=mean[:n], rstd=rstd[:n])
    ok()
    assert (mean[n:] == 7).all() and (rstd[n:] == 7).all()
    assert torch.equal(mean[:n], r.mean) and torch.equal(rstd[:n], r.rstd)
