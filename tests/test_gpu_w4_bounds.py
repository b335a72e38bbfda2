"""The 4-bit products against their formulas in 64 bits, element by element, with
bounds that an output of zeros does not meet.

The codes enter the tensor cores as code - 8, exactly, and a group's products (of 8
significant bits by 4) are exact in fp32. So a sum over C columns takes at most
`group` additions within each group, one scaled addition for each of the C / group
groups and one for each of the 8 warps that may share the columns:
(group + C / group + 8) 2^-23 of the sum of the magnitudes, truncation included. A
rounding to bf16 takes 2^-8, the activation 2^-18."""
import math

import pytest
import torch

import mixture_experts_routing_gb300 as moe
from test_gpu_w4 import DEV, F64, MATVEC, Batch, act64, codes, gen, normal, ok, weights, within

pytestmark = pytest.mark.gpu


def sum_error(cols, group):
    return (group + cols / group + 8) * 2.0 ** -23


def rms(t):
    return t.square().mean(1, keepdim=True).sqrt()


def near(got, ref, routed, what):
    """The roundings of the hidden values (at most 2^-8 of each) are independent, so over
    a long sum they are a small part of 2^-8 of the row's size; 2^-5 of it leaves room
    for a sum that one term dominates, times the largest weight of a row."""
    d = (got.to(F64) - ref).abs()
    over = d - 2.0 ** -8 * ref.abs() - 2.0 ** -5 * rms(routed)
    assert torch.isfinite(d).all() and over.max().item() <= 0, "%s: %d elements off" % (what, (over > 0).sum().item())


def tells(part, bound):
    """The part that the kernel computes is over the bound on most elements."""
    assert (part.abs() > bound).double().mean().item() > 0.5


@pytest.mark.parametrize("n,rows,cols,group", MATVEC + [(1, 4104, 7168, 64), (6, 520, 7168, 32), (13, 4104, 4096, 32), (20, 1032, 6144, 128)])
def test_matvec(n, rows, cols, group):
    g = gen(n + rows + cols)
    x, q, s = normal(g, n, cols), codes(g, rows, cols // 2), normal(g, rows, cols // group, std=0.02)
    y = torch.full((n, rows), math.nan, dtype=torch.bfloat16, device=DEV)
    moe.w4_matvec(x, q, s, y)
    ok()
    w = weights(q, s)
    ref = x.to(F64) @ w.t()
    bound = 2.0 ** -8 * ref.abs() + sum_error(cols, group) * (x.to(F64).abs() @ w.abs().t())
    if n * rows > 16:
        tells(ref, bound)
    within(y, ref, bound, "y")


def reference(b):
    """y, the routed experts' part of it, and the bound."""
    group = b.cfg.group
    part = torch.zeros((b.n, b.h), dtype=F64, device=DEV)
    bound = torch.zeros_like(part)
    for e in range(b.e):
        t, k = (b.ids == e).nonzero(as_tuple=True)
        if not len(t):
            continue
        x = b.x[t].to(F64)
        w13, w2 = weights(b.q13[e], b.s13[e]), weights(b.q2[e], b.s2[e])
        (g, u), (eg, eu) = ((v.split(b.i, 1)) for v in (x @ w13.t(), sum_error(b.h, group) * (x.abs() @ w13.abs().t())))
        a = act64(g, b.act)
        hid = a * u
        eh = (2.0 ** -8 + 2.0 ** -18) * hid.abs() + 1.15 * eg * u.abs() + a.abs() * eu + 1.15 * eg * eu
        p = b.p[t, k].to(F64).unsqueeze(1)
        part.index_add_(0, t, p * (hid @ w2.t()))
        # 8 more additions, of the products' parts and of the token's routes
        bound.index_add_(0, t, p * (1.01 * eh @ w2.abs().t() + (sum_error(b.i, group) + (8 + b.k) * 2.0 ** -23) * (hid.abs() @ w2.abs().t())))
    y = part if b.add is None else part + b.add.to(F64)
    return y, part, bound + 2.0 ** -8 * y.abs() + b.k * 2.0 ** -23 * (0 if b.add is None else b.add.to(F64).abs())


@pytest.mark.parametrize("act", [moe.ACT_SWIGLU, moe.ACT_GEGLU])
@pytest.mark.parametrize("n,h,e,k,i,group", [
    (1, 128, 1, 1, 128, 128), (1, 32, 3, 2, 64, 32), (1, 1024, 16, 8, 512, 128), (2, 96, 4, 2, 160, 32), (3, 640, 5, 5, 192, 64), (5, 2048, 128, 8, 768, 64),
    (8, 256, 8, 4, 384, 128), (9, 128, 2, 1, 256, 32), (16, 512, 256, 16, 128, 64), (33, 384, 4, 3, 128, 128), (64, 256, 64, 16, 128, 32),
    (100, 128, 1, 1, 96, 32), (128, 256, 16, 8, 192, 64), (1024, 64, 8, 1, 64, 64), (1, 7168, 8, 8, 2048, 128), (40, 4096, 3, 2, 1408, 128),
    (24, 2080, 40, 4, 1056, 32), (32, 1056, 20, 8, 2080, 32), (32, 1088, 24, 8, 1088, 64), (25, 2112, 70, 3, 1088, 64), (32, 1152, 60, 4, 1280, 128),
    (4, 7168, 16, 8, 2048, 64), (33, 2048, 128, 8, 768, 64),
])
def test_experts(n, h, e, k, i, group, act):
    b = Batch(n, h, e, k, i, group, act, add=n % 2 == 0)
    b.y.fill_(math.nan)
    b.run()
    ok()
    y, part, bound = reference(b)
    if b.add is None:
        tells(part, bound)
    else:  # the addend's own rounding is not the experts'
        tells(part, bound - 2.0 ** -8 * y.abs() + 2.0 ** -8 * part.abs())
    within(b.y, y, bound, "y")
    near(b.y, y, part, "y")
