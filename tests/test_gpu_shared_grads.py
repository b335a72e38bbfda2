"""The shared expert's backward where one pair of CTAs takes tiles of more than one
gradient, fp32 ones among them: batches longer than wide, whose dx tiles come after
the weight gradients' in a pair's list. And every output at every size, element by
element, with a bound that follows the size of its row."""
import math

import pytest
import torch

import mixture_experts_routing_gb300 as moe
from test_gpu_shared import SIZES, Block, fro, ok, reference_backward, reference_forward, within

pytestmark = pytest.mark.gpu

# 2i < n, and more tiles of 256 rows than pairs of CTAs
LONG = [(2500, 2056, 32), (4096, 2048, 64), (3000, 5000, 96), (6000, 4096, 64), (8192, 4096, 64), (8192, 2048, 768)]


def near(got, ref, what, add=None):
    """Off by a rounding to bf16 (2^-8 of the value, and as much again for a sum of one
    term) and by the operands' roundings: at most 2^-8 of each and independent, so over
    a sum of many terms a small part of 2^-8 of the row's size; 2^-5 of it leaves room
    for a sum that one term dominates, times the largest weight of a row. What is added
    is exact and does not count to the row's size."""
    d = (got.double() - ref).abs()
    row = ref if add is None else ref - add.double()
    over = d - 2.0 ** -7 * ref.abs() - 2.0 ** -5 * row.square().mean(1, keepdim=True).sqrt()
    assert torch.isfinite(d).all() and over.max().item() <= 0, "%s: %d elements off" % (what, (over > 0).sum().item())


@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("grad_f32", [1, 0])
@pytest.mark.parametrize("n,h,i", LONG)
def test_long_batches(n, h, i, grad_f32, add):
    b = Block(n, h, i, moe.ACT_SWIGLU, add=add, grad_f32=grad_f32)
    b.forward()
    b.backward()
    ok()
    for name, got, (ref, bound) in zip(("dx", "dw13", "dw2"), (b.dx, b.dw13, b.dw2), reference_backward(b)):
        within(got, ref, bound, name)
        near(got, ref, name, b.add if name == "dx" else None)
        fro(got, ref, 5e-3, name)
    first = [t.clone() for t in (b.dx, b.dw13, b.dw2)]
    for _ in range(20):
        for t in (b.dx, b.dw13, b.dw2):
            t.fill_(math.nan)
        b.backward()
        ok()
        assert all(torch.equal(t, f) for t, f in zip((b.dx, b.dw13, b.dw2), first))


@pytest.mark.parametrize("act", [moe.ACT_SWIGLU, moe.ACT_GEGLU])
@pytest.mark.parametrize("n,h,i", SIZES + [(64, 4096, 2048), (130, 1032, 1408), (700, 264, 2048), (500, 4096, 1408), (1935, 304, 256)])
def test_every_element(n, h, i, act):
    b = Block(n, h, i, act, add=(n + i) % 3 == 0, grad_f32=(n + h // 8 + 1) % 2)
    for t in (b.y, b.dx, b.dw13, b.dw2):
        t.fill_(math.nan)
    b.forward()
    b.backward()
    ok()
    near(b.y, reference_forward(b)[0], "y", b.add)
    for name, got, (ref, _) in zip(("dx", "dw13", "dw2"), (b.dx, b.dw13, b.dw2), reference_backward(b)):
        near(got, ref, name, b.add if name == "dx" else None)
