"""A Mixture-of-Experts layer with a shared expert: one training step, then decode
steps with the routed experts in 4 bits.

    python examples/moe_layer.py [--tokens 1024] [--decode 4] [--activation swiglu] [--block]

Training: routed experts and shared expert forward, the shared expert's activations
kept in 8 bits, and both backwards; the layer's output and input gradient are built
up in place (`add=y`, `dx_add=dx`). Decode: router, 4-bit experts, shared expert on
a few tokens. --block puts the layer between two norms with residual sums, updates its
weights with AdamW (states in 8 bits) and decodes in bf16 with the updated weights.
Sizes are those of the small Qwen3-style layer of the benchmarks.
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import mixture_experts_routing_gb300 as moe  # noqa: E402


class Layer:
    """Random weights of one layer and the buffers of a training step of n tokens."""

    def __init__(self, n=1024, hidden=512, experts=8, top_k=2, inter=1024, shared_inter=1024,
                 activation=moe.ACT_SWIGLU, seed=0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def normal(*shape, std=1.0, dtype=torch.bfloat16):
            return (torch.randn(shape, device=device, generator=g) * std).to(dtype)

        self.device = device
        self.cfg = moe.Config(n, hidden, experts, top_k, inter, cap_num=0, cap_den=1, block_m=32,
                              ladder=[1, 2, 4], ladder_den=2, activation=activation)
        self.shared = moe.SharedConfig(n, hidden, shared_inter, activation=activation, grad_f32=1)
        self.w_router = normal(hidden, experts, std=0.02, dtype=torch.float32)
        self.w13, self.w2 = normal(experts, 2 * inter, hidden, std=hidden ** -0.5), normal(experts, hidden, inter, std=inter ** -0.5)
        self.sw13, self.sw2 = normal(2 * shared_inter, hidden, std=hidden ** -0.5), normal(hidden, shared_inter, std=shared_inter ** -0.5)
        self.x, self.dy = normal(n, hidden), normal(n, hidden)

    def train_step(self):
        """y, dx and every weight gradient of x and dy."""
        y = self.forward()
        return (y, *self.backward())

    def forward(self):
        """y of x; what the backward needs is kept."""
        c, s, dev = self.cfg, self.shared, self.device
        routes, ws = moe.alloc_routes(c, dev), moe.alloc_workspace(c, dev)
        h, o, y = moe.alloc_buffers(c, dev)
        preact = torch.empty((h.shape[0], 2 * c.inter), dtype=torch.bfloat16, device=dev)
        sh, _ = moe.alloc_shared_buffers(s, dev)
        ck, ck_sf = moe.alloc_shared_checkpoint(s, dev)
        moe.route_align(c, self.x, self.w_router, None, routes, ws)
        moe.ffn_forward_train(c, routes, self.x, self.w13, self.w2, h, o, preact)
        moe.combine(c, routes, o, y)
        moe.shared_forward_train(s, self.x, self.sw13, self.sw2, sh, y, ck, ck_sf, add=y)
        self.kept = routes, ws, preact, ck, ck_sf
        return y

    def backward(self):
        """dx and every weight gradient of dy."""
        c, s, dev = self.cfg, self.shared, self.device
        f32 = dict(dtype=torch.float32, device=dev)
        routes, ws, preact, ck, ck_sf = self.kept
        dx = torch.empty_like(self.x)
        grads = {"w13": torch.empty(self.w13.shape, **f32), "w2": torch.empty(self.w2.shape, **f32),
                 "router": torch.empty(self.w_router.shape, **f32),
                 "shared_w13": torch.empty(self.sw13.shape, **f32), "shared_w2": torch.empty(self.sw2.shape, **f32)}
        dprob = torch.empty((c.n_tokens, c.top_k), **f32)
        moe.ffn_backward(c, routes, self.x, self.w13, self.w2, preact, self.dy, dx, grads["w13"],
                         grads["w2"], dprob, moe.alloc_backward_workspace(c, dev))
        moe.router_backward(c, routes, self.x, self.w_router, None, dprob, dx, grads["router"], None,
                            moe.alloc_router_backward_workspace(c, dev),
                            logits=moe.route_workspace_logits(c, ws))
        moe.shared_backward(s, self.x, self.sw13, self.sw2, ck, ck_sf, self.dy, dx,
                            grads["shared_w13"], grads["shared_w2"],
                            moe.alloc_shared_backward_workspace(s, dev), dx_add=dx)
        return dx, grads

    def pack_for_decode(self, group=128):
        """The routed experts in 4 bits, once."""
        self.w4 = moe.W4Weights(self.w13, self.w2, group)

    def decode(self, x):
        """The layer's output for a few tokens x [n, hidden]."""
        n, c, dev = x.shape[0], self.cfg, self.device
        route = moe.Config(n, c.hidden, c.n_experts, c.top_k, c.inter, cap_num=0, cap_den=1,
                           block_m=16, activation=c.activation)
        routes, ws = moe.alloc_routes(route, dev), moe.alloc_workspace(route, dev)
        w4 = moe.W4Config(n, c.hidden, c.n_experts, c.top_k, c.inter, self.w4.group, activation=c.activation)
        shared = moe.SharedConfig(n, c.hidden, self.shared.inter, activation=c.activation)
        sh, y = moe.alloc_shared_buffers(shared, dev)
        moe.route_align(route, x, self.w_router, None, routes, ws)
        moe.w4_ffn_forward(w4, routes.topk_ids, routes.topk_p, x, self.w4.w13q, self.w4.w13_scale,
                           self.w4.w2q, self.w4.w2_scale, y, moe.alloc_w4_workspace(w4, dev))
        moe.shared_forward(shared, x, self.sw13, self.sw2, sh, y, add=y)
        return y


class Block(Layer):
    """The layer in a pre-norm block: s = x + r, a = norm(s), y = layer(a), t = s + y,
    z = norm(t); RMS norms, as such layers have them. Every weight is trained."""

    def __init__(self, n=1024, lr=1e-2, **kw):
        super().__init__(n, **kw)
        h = self.cfg.hidden
        g = torch.Generator(device=self.device)
        g.manual_seed(kw.get("seed", 0) + 1)
        self.tokens = self.x
        self.residual, self.dz = (torch.randn((n, h), device=self.device, generator=g).bfloat16() for _ in range(2))
        self.norm_w = [1 + 0.1 * torch.randn(h, device=self.device, generator=g) for _ in range(2)]
        self.weights = {"router": self.w_router, "w13": self.w13, "w2": self.w2, "shared_w13": self.sw13, "shared_w2": self.sw2,
                        "norm0": self.norm_w[0], "norm1": self.norm_w[1]}
        self.grads = {k: torch.empty(w.shape, dtype=torch.float32, device=self.device) for k, w in self.weights.items()}
        self.opt = moe.AdamW(list(self.weights.values()), list(self.grads.values()), lr=lr, betas=(0.9, 0.95), state_bits=8,
                             weight_decay=[0.0 if k.startswith("norm") else 0.1 for k in self.weights])

    def norm(self, i, x, add):
        """The residual sum, its norm, and 1 / rms of its rows."""
        cfg = moe.NormConfig(x.shape[0], x.shape[1], kind=moe.NORM_RMS)
        s, y, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(x.shape[0], device=x.device)
        moe.norm_forward(cfg, x, self.norm_w[i], y, add=add, sum=s, rstd=rstd)
        return s, y, rstd

    def norm_grad(self, i, s, rstd, dy, dx_add=None):
        cfg = moe.NormConfig(s.shape[0], s.shape[1], kind=moe.NORM_RMS)
        dx = torch.empty_like(s)
        moe.norm_backward(cfg, s, self.norm_w[i], None, rstd, dy, dx, self.grads["norm%d" % i],
                          moe.alloc_norm_backward_workspace(cfg, self.device), dx_add=dx_add)
        return dx

    def block_step(self):
        """Forward, gradients of x (and of r alike) and of every weight, update."""
        s, a, rstd0 = self.norm(0, self.tokens, self.residual)
        self.x = a
        y = self.forward()
        t, z, rstd1 = self.norm(1, s, y)
        self.dy = self.norm_grad(1, t, rstd1, self.dz)  # the gradient of t, hence of y and of s
        da, grads = self.backward()
        for k, g in grads.items():
            self.grads[k].copy_(g)
        dx = self.norm_grad(0, s, rstd0, da, dx_add=self.dy)
        self.opt.step()
        return z, dx

    def block_decode(self, x, residual):
        """z for a few tokens, with the routed experts' layer in one call."""
        n, c, dev = x.shape[0], self.cfg, self.device
        few = moe.FewConfig(n, c.hidden, c.n_experts, c.top_k, c.inter, activation=c.activation)
        shared = moe.SharedConfig(n, c.hidden, self.shared.inter, activation=c.activation)
        h, y = moe.alloc_shared_buffers(shared, dev)
        s, a, _ = self.norm(0, x, residual)
        moe.shared_forward(shared, a, self.sw13, self.sw2, h, y)
        moe.few_forward(few, a, self.w_router, None, self.w13, self.w2, y, moe.alloc_few_workspace(few, dev), add=y)
        return self.norm(1, s, y)[1]


def main_block(a, activation):
    block = Block(a.tokens, activation=activation)
    before = {k: w.clone() for k, w in block.weights.items()}
    z, dx = block.block_step()
    print("block: z rms %.3f, dx rms %.3f, weights moved by %s" % (
        z.float().square().mean().sqrt(), dx.float().square().mean().sqrt(),
        ", ".join("%s %.2g" % (k, (w.float() - before[k].float()).abs().mean()) for k, w in block.weights.items())))
    n = min(a.decode, 64)
    d = block.block_decode(block.tokens[:n].contiguous(), block.residual[:n].contiguous())
    print("block decode: %d tokens with the updated weights, rms %.3f" % (n, d.float().square().mean().sqrt()))
    torch.cuda.synchronize()
    err = moe.device_error()
    if err:
        raise RuntimeError("device error word %d" % err)
    return block, before, z, dx, d


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=1024)
    ap.add_argument("--decode", type=int, default=4, help="tokens of a decode step")
    ap.add_argument("--activation", choices=("swiglu", "geglu"), default="swiglu")
    ap.add_argument("--block", action="store_true", help="the layer between norms: a training step with its update, decode in bf16")
    a = ap.parse_args(argv)
    activation = moe.ACT_GEGLU if a.activation == "geglu" else moe.ACT_SWIGLU
    if a.block:
        return main_block(a, activation)
    layer = Layer(a.tokens, activation=activation)
    y, dx, grads = layer.train_step()
    print("train: y rms %.3f, dx rms %.3f, gradients %s" % (
        y.float().square().mean().sqrt(), dx.float().square().mean().sqrt(),
        ", ".join("%s %.3f" % (k, v.square().mean().sqrt()) for k, v in grads.items())))
    layer.pack_for_decode()
    d = layer.decode(layer.x[: a.decode].contiguous())
    off = (d.float() - y[: a.decode].float()).norm() / y[: a.decode].float().norm()
    print("decode: %d tokens, %.3f from the training forward (what 4 bits lose)" % (a.decode, off))
    torch.cuda.synchronize()
    err = moe.device_error()
    if err:
        raise RuntimeError("device error word %d" % err)
    return layer, y, dx, grads, d


if __name__ == "__main__":
    main()
