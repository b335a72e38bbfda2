"""The example's training and decode steps against the layer's formulas in 64 bits."""
import os
import sys

import pytest
import torch

import mixture_experts_routing_gb300 as moe
from conftest import ROOT

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(ROOT, "examples"))


@pytest.mark.parametrize("activation", ["swiglu", "geglu"])
@pytest.mark.parametrize("decode", [1, 6])
def test_example(activation, decode):
    import moe_layer
    layer, y, dx, grads, d = moe_layer.main(["--tokens", "300", "--decode", str(decode), "--activation", activation])
    act = layer.cfg.activation

    def f(t):
        return t.double().detach().requires_grad_()

    x, wr, w13, w2, sw13, sw2 = (f(t) for t in (layer.x, layer.w_router, layer.w13, layer.w2, layer.sw13, layer.sw2))

    def ffn(x, w13, w2):
        g, u = (x @ w13.t()).chunk(2, 1)
        a = g * torch.sigmoid(g) if act == moe.ACT_SWIGLU else 0.5 * g * (1 + torch.erf(g * 0.5 ** 0.5))
        return (a * u) @ w2.t()

    p = torch.softmax(x @ wr, 1)
    top = p.topk(layer.cfg.top_k, 1)
    q = top.values / top.values.sum(1, keepdim=True)
    out = ffn(x, sw13, sw2)
    for e in range(layer.cfg.n_experts):
        w = (q * (top.indices == e)).sum(1, keepdim=True)
        out = out + w * ffn(x, w13[e], w2[e])
    (out * layer.dy.double()).sum().backward()

    def rel(a, b):
        return ((a.double() - b).norm() / b.norm()).item()

    # bf16 operands and results: 2^-8 of a value at most, a few of them in a row
    assert rel(y, out.detach()) < 1e-2
    for name, got, want in (("w13", grads["w13"], w13.grad), ("w2", grads["w2"], w2.grad), ("router", grads["router"], wr.grad)):
        assert rel(got, want) < 1e-2, name
    # the shared expert's gradients come from activations kept in 8 bits: each is off by
    # up to 2^-4 of itself, 0.026 in the mean square, in two factors
    for name, got, want in (("dx", dx, x.grad), ("shared_w13", grads["shared_w13"], sw13.grad), ("shared_w2", grads["shared_w2"], sw2.grad)):
        assert rel(got, want) < 6e-2, name
    # 4-bit weights: half a step of max/7 over 128 normal values, 0.11 of a weight in the mean square, in three factors
    assert rel(d, out.detach()[:decode]) < 0.3
