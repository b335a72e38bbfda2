"""AdamW over many tensors, states in 32 and in 8 bits, against its formula in 64 bits.

Bounds: m and v are two products and a sum in fp32: 2 2^-24 of each term's size, 4 2^-24
with the scaled gradient. The update has a square root, a division and the corrections
1 - b^t, each within a few roundings: 2^-19 of itself; where v is a difference of nothing,
its own error enters as half of itself. An 8-bit code is one of the two next to the value."""
import math

import numpy as np
import pytest
import torch

import mixture_experts_routing_gb300 as moe
from test_gpu_w4 import DEV, F64, gen, ok, within

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
SIZES = [[1], [7, 8, 9], [255, 256, 257], [1000, 1, 4096, 100003], [64] * 239, [65] * 240, [300] * 241, [17] * 481 + [70000], [2500000]]


def decode(codes, scale):
    """Values of 8-bit states."""
    v = codes.view(torch.float8_e4m3fn).to(F64).view(-1, 256)
    return (v * scale.to(F64).unsqueeze(1)).view(-1)


class Set:
    """Tensors with gaps behind them, their gradients and an optimizer; the same flat layout in 64 bits."""

    def __init__(self, sizes, wide, grad32, bits, decay=0.1, **kw):
        g = gen(sum(sizes))
        self.sizes, self.wide, self.bits = sizes, wide, bits
        pt, gt = torch.float32 if wide else torch.bfloat16, torch.float32 if grad32 else torch.bfloat16
        self.params, self.grads, self.guards = [], [], []
        for n in sizes:
            room = torch.full((n + 24,), 5.0, dtype=pt, device=DEV)
            room[:n] = torch.randn(n, device=DEV, generator=g) * 0.05
            self.guards.append(room[n:])
            self.params.append(room[:n])
            self.grads.append((torch.randn(n, device=DEV, generator=g) * torch.exp(torch.randn(n, device=DEV, generator=g))).to(gt))
        self.decay = [decay if i % 2 == 0 else 0.0 for i in range(len(sizes))]
        self.kw = dict(lr=1e-2, betas=(0.9, 0.99), eps=1e-8) | kw
        self.opt = moe.AdamW(self.params, self.grads, weight_decay=self.decay, state_bits=bits, **self.kw)

    def flat(self, tensors):
        out = torch.zeros(self.opt.m.numel(), dtype=F64, device=DEV)
        for a, t in zip(self.opt.offsets, tensors):
            out[a: a + t.numel()] = t.to(F64).view(-1)
        return out

    def state(self):
        o = self.opt
        m = o.m.to(F64) if self.bits == 32 else decode(o.m, o.m_scale)
        v = o.v.to(F64) if self.bits == 32 else decode(o.v, o.v_scale).square()
        return (self.flat(self.params) if self.wide else o.master.to(F64)), m, v

    def reference(self, before, t, scale=1.0, lr=None):
        """The state after step t, and how far it may be off, before any rounding to 8 bits."""
        p, m, v = before
        lr, (b1, b2), eps = self.kw["lr"] if lr is None else lr, self.kw["betas"], self.kw["eps"]
        g = self.flat(self.grads) * scale
        wd = self.flat([torch.full((n,), float(d), device=DEV) for n, d in zip(self.sizes, self.decay)])
        m2, v2 = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
        dm, dv = 4 * U * ((b1 * m).abs() + ((1 - b1) * g).abs()), 8 * U * v2
        up = m2 / (1 - b1 ** t) / (torch.sqrt(v2 / (1 - b2 ** t)) + eps)
        dup = 2.0 ** -19 * up.abs() + dm / (1 - b1 ** t) / (torch.sqrt(v2 / (1 - b2 ** t)) + eps)
        p2 = p - lr * (up + wd * p)
        return (p2, m2, v2), (4 * U * (p.abs() + (lr * up).abs()) + lr * dup, dm, dv + 1e-44)


def codes_next_to(got, scale, want, tol, what):
    """Every code is one of the two around the value that it stands for, the scale that of the block's largest."""
    b = want.view(-1, 256)
    top = b.abs().amax(1)
    zero = top < 2.0 ** -100
    assert (scale[zero] == 0).all() and (got.view(-1, 256)[zero] & 127 == 0).all()
    assert ((scale.to(F64) - top / 448).abs() <= tol * top + 1e-44)[~zero].all(), what
    a = torch.where(zero.unsqueeze(1), 0, b / (top / 448).clamp(min=1e-300).unsqueeze(1))
    step = torch.exp2(torch.floor(torch.log2(a.abs().clamp(min=2.0 ** -30))).clamp(min=-6) - 3)
    d = (got.view(torch.float8_e4m3fn).to(F64).view(-1, 256) - a).abs()
    assert (d < step * (1 + 1e-9) + 2 * tol * 448).all(), what


def check(s, before, t, **kw):
    want, room = s.reference(before, t, **kw)
    p, m, v = s.state()
    within(p, want[0], room[0], "p")
    if not s.wide:  # a weight is the rounding of its master
        flat = s.flat(s.params)
        assert torch.equal(flat, s.opt.master.to(torch.bfloat16).to(F64))
    if s.bits == 32:
        within(m, want[1], room[1], "m")
        within(v, want[2], room[2], "v")
    else:
        codes_next_to(s.opt.m, s.opt.m_scale, want[1], 8 * U, "m")
        codes_next_to(s.opt.v, s.opt.v_scale, want[2].sqrt(), 8 * U, "v")
    gap = s.flat([torch.ones(n, device=DEV) for n in s.sizes]) == 0
    assert (s.opt.m[gap] == 0).all() and (s.opt.v[gap] == 0).all()
    assert all((g == 5).all() for g in s.guards)
    assert s.opt.steps.tolist() == [t, 0]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("wide,grad32", [(True, True), (False, True), (False, False), (True, False)])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: "%dx%d" % (len(s), max(s)))
def test_steps(sizes, wide, grad32, bits):
    s = Set(sizes, wide, grad32, bits)
    for t in (1, 2, 3):
        before = s.state()
        s.opt.step()
        ok()
        check(s, before, t)
        for i, g in enumerate(s.grads):
            g.mul_(-0.7 if i % 2 else 0.01)


@pytest.mark.parametrize("bits", [32, 8])
def test_gradient_scale_and_rate_from_the_device(bits):
    s = Set([1000, 5000], False, True, bits)
    scale, lr = torch.tensor([0.125], device=DEV), torch.tensor([3e-3], device=DEV)
    before = s.state()
    s.opt.step(grad_scale=scale, lr=lr)
    ok()
    check(s, before, 1, scale=0.125, lr=float(lr))
    before = s.state()
    s.opt.step(lr=5e-4)
    ok()
    check(s, before, 2, lr=5e-4)
    kept = [t.clone() for t in (s.opt.m, s.opt.v, s.opt.master, *s.params)]
    for bad in (math.nan, math.inf, -math.inf):
        scale.fill_(bad)
        s.opt.step(grad_scale=scale)
        ok()
        assert s.opt.steps.tolist() == [2, 0]
        assert all(torch.equal(a, b) for a, b in zip(kept, (s.opt.m, s.opt.v, s.opt.master, *s.params)))
    scale.fill_(0.0)
    before = s.state()
    s.opt.step(grad_scale=scale)
    ok()
    check(s, before, 3, scale=0.0, lr=5e-4)


@pytest.mark.parametrize("betas", [(0.0, 0.0), (0.0, 0.999), (0.9999, 0.99999), (0.9, 0.95)])
def test_corrections_of_early_and_late_steps(betas):
    s = Set([3000], True, True, 32, betas=betas)
    for t in (1, 2, 1000, 1000000):
        s.opt.steps[0] = t - 1
        before = s.state()
        s.opt.step()
        ok()
        check(s, before, t)


def test_an_empty_tensor_and_an_empty_list_of_values():
    s = Set([0, 513, 0], True, True, 8)
    before = s.state()
    s.opt.step()
    ok()
    check(s, before, 1)
    e = Set([0, 0], False, True, 32)
    e.opt.step()
    ok()
    assert e.opt.steps.tolist() == [1, 0]


@pytest.mark.parametrize("bits", [32, 8])
def test_zero_tiny_huge_and_non_finite_gradients(bits):
    s = Set([256 * 6], True, True, bits)
    g = s.grads[0]
    g[:256] = 0
    g[256:512] *= 1e-18
    g[512:768] *= 1e12
    before = s.state()
    s.opt.step()
    ok()
    check(s, before, 1)
    g[800], g[1100] = math.nan, math.inf
    before, weights = s.state(), s.params[0].clone()
    s.opt.step()
    ok()
    want, room = s.reference(before, 2)
    p, m, v = s.state()
    clean = torch.ones(1536, dtype=torch.bool, device=DEV)
    clean[800] = clean[1100] = False
    within(p[:1536][clean], want[0][:1536][clean], room[0][:1536][clean], "p")
    assert p[800].isnan() and p[1100].isnan()
    if bits == 32:
        assert m[800].isnan() and m[1100].isinf()
        within(m[:1536][clean], want[1][:1536][clean], room[1][:1536][clean], "m")
    else:  # the blocks that hold them read as NaN, the others do not
        bad = torch.zeros(6, dtype=torch.bool, device=DEV)
        bad[3] = bad[4] = True
        assert torch.equal(m.view(-1, 256).isnan().all(1), bad) and torch.equal(m.view(-1, 256).isnan().any(1), bad)


def test_8_bit_states_keep_their_mean():
    """v decays by 1 % a step, 0.5 % in sqrt(v), against codes 6 to 12 % apart. Over t steps the rounding of
    each value adds a variance of at most its code step times its change: 0.005 * 0.125 r^2 a step, 0.25 r
    over 100 steps before decay; over 25600 values the mean is off by 0.25 / 160 = 0.0016, six of which are 0.01."""
    n = 25600
    s = Set([n], True, True, 8, betas=(0.9, 0.99))
    s.grads[0].copy_(0.5 + torch.rand(n, device=DEV, generator=gen(1)))
    s.grads[0].view(-1, 256)[:, 0] = 2.0  # the blocks' largest
    s.opt.step()
    s.grads[0].view(-1, 256)[:, 1:] = 0
    start = decode(s.opt.v, s.opt.v_scale).view(-1, 256)[:, 1:].mean()
    for _ in range(100):
        s.opt.step()
    ok()
    now = decode(s.opt.v, s.opt.v_scale).view(-1, 256)[:, 1:].mean()
    assert abs((now / start).item() / 0.99 ** 50 - 1) < 0.01


def test_the_rounding_is_that_of_the_hash():
    """Codes of a step from zero states, value by value: v = 0.01 g^2, m = 0.1 g, so sqrt(v) = 0.1 |g|."""
    n, first = 70000, 0
    s = Set([n], True, True, 8, betas=(0.9, 0.99), seed=77)
    g = s.grads[0].clone()
    s.opt.step()
    ok()

    def mix(v):
        v = (v ^ (v >> np.uint32(16))) * np.uint32(0x7FEB352D)
        v = (v ^ (v >> np.uint32(15))) * np.uint32(0x846CA68B)
        return v ^ (v >> np.uint32(16))

    with np.errstate(over="ignore"):
        key = mix(np.array([0x9E3779B1 + 77], dtype=np.uint32))
        d = mix((np.arange(n, dtype=np.uint32) + np.uint32(first)) * np.uint32(0x9E3779B1) + key)
    m = np.zeros(-(-n // 256) * 256)
    m[:n] = 0.1 * g.double().cpu().numpy()
    b = m.reshape(-1, 256)
    a = np.abs(b) / (np.abs(b).max(1, keepdims=True) / 448)
    step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(a, 2.0 ** -30))), -6) - 3)
    frac = np.zeros_like(m)
    frac[:n] = ((d & np.uint32(0xFFFF)).astype(np.float64) + 0.5) / 65536
    want = np.sign(b) * np.minimum(np.floor(a / step + frac.reshape(-1, 256)) * step, 448)
    got = s.opt.m.view(torch.float8_e4m3fn).double().cpu().numpy().reshape(-1, 256)
    # fp32 puts a value on the other side of its dither with a probability of 2^-20 or so
    assert (got != want).mean() < 1e-4


def test_many_small_codes_do_not_pass_the_largest():
    s = Set([256 * 40], True, True, 8)
    for _ in range(20):
        s.opt.step()
    ok()
    assert (s.opt.m & 127).max().item() <= 126 and s.opt.v.max().item() <= 126
    assert ((s.opt.m & 127).view(-1, 256).amax(1) == 126).all() and (s.opt.v.view(-1, 256).amax(1) == 126).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_replayed_and_resumed(bits):
    a, b, c = (Set([5000, 33, 70001], False, True, bits) for _ in range(3))
    for _ in range(4):
        a.opt.step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.opt.step()
    for _ in range(3):
        graph.replay()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b.opt.step(stream=side)
    c.opt.step()
    c.opt.step()
    d = Set([5000, 33, 70001], False, True, bits)
    for n in ("m", "v", "master", "steps") + (("m_scale", "v_scale") if bits == 8 else ()):
        getattr(d.opt, n).copy_(getattr(c.opt, n))
    d.opt.step()
    d.opt.step()
    ok()
    for s in (b, d):
        assert s.opt.steps.tolist() == [4, 0]
        for n in ("m", "v", "master"):
            assert torch.equal(getattr(s.opt, n), getattr(a.opt, n))
        assert all(torch.equal(p, q) for p, q in zip(s.params, a.params))


@pytest.mark.parametrize("bits", [32, 8])
def test_weights_and_gradients_of_both_types_in_one_list(bits):
    """Each tensor moves as it does in a list of its own type (8 bits: but for the places in the hash)."""
    g = gen(11)
    shapes = [(64, 33), (1000,), (2, 3, 50), (7,), (300, 300)]
    types = [(torch.bfloat16, torch.float32), (torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16), (torch.float32, torch.bfloat16), (torch.bfloat16, torch.float32)]
    params = [(torch.randn(s, device=DEV, generator=g) * 0.1).to(p).requires_grad_(p is torch.float32) for s, (p, _) in zip(shapes, types)]
    grads = [torch.randn(s, device=DEV, generator=g).to(t) for s, (_, t) in zip(shapes, types)]
    old = [p.detach().clone() for p in params]
    opt = moe.AdamW(params, grads, lr=1e-2, betas=(0.9, 0.99), weight_decay=[0.1, 0, 0.2, 0, 0.3], state_bits=bits)
    opt.step()
    ok()
    for i, (p, q, gr) in enumerate(zip(params, old, grads)):
        alone = q.clone()
        one = moe.AdamW([alone], [gr], lr=1e-2, betas=(0.9, 0.99), weight_decay=[0.1, 0, 0.2, 0, 0.3][i], state_bits=bits)
        one.step()
        ok()
        assert torch.equal(alone, p.detach()), i
        a, n = opt.offsets[i], q.numel()
        if bits == 32:
            assert torch.equal(opt.m[a: a + n], one.m[:n]) and torch.equal(opt.v[a: a + n], one.v[:n])
        else:
            assert torch.equal(opt.m_scale[a // 256: -(-(a + n) // 256)], one.m_scale)


def test_more_than_2_31_values():
    n = (1 << 31) + 1000  # 8-bit states, bf16 gradients: values on both sides of the border
    p = torch.zeros(n, dtype=torch.float32, device=DEV)
    g = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    tail = 3000
    g[-tail:] = torch.randn(tail, device=DEV, generator=gen(3)).to(torch.bfloat16)
    opt = moe.AdamW([p], [g], lr=1e-2, weight_decay=0.0, state_bits=8)
    opt.step()
    ok()
    # the first step moves each weight by lr against the sign of its gradient
    assert torch.allclose(p[-tail:], -1e-2 * torch.sign(g[-tail:].float()), rtol=1e-4, atol=1e-7)
    assert (p[:tail] == 0).all() and not p[: n - tail].any()
    m = decode(opt.m[-4096:], opt.m_scale[-16:])
    at = opt.m.numel() - n
    got = m[m.numel() - at - tail: m.numel() - at]
    want = 0.1 * g[-tail:].to(F64)
    assert ((got - want).norm() / want.norm()).item() < 0.08  # a code is 2^-3 of its value apart at most


def test_refusals():
    p, g = torch.zeros(64, device=DEV), torch.zeros(64, device=DEV)
    for bad in (dict(params=[p], grads=[g[:63]]), dict(params=[p.half()], grads=[g]), dict(params=[p[::2]], grads=[g[:32]]), dict(params=[p], grads=[g.cpu()])):
        with pytest.raises(ValueError):
            moe.AdamW(lr=1e-3, **bad)
    with pytest.raises(ValueError, match="twice"):
        moe.AdamW([p, p], [g, g.clone()], lr=1e-3)
    opt = moe.AdamW([torch.zeros(65, device=DEV)[1:]], [g], lr=1e-3)
    with pytest.raises(moe.MoEError):  # not 16-byte aligned
        opt.step()
    opt = moe.AdamW([p], [g], lr=1e-3)
    with pytest.raises(ValueError, match="grad_scale"):
        opt.step(grad_scale=torch.tensor([1.0]))
    with pytest.raises(moe.MoEError):
        opt.step(lr=math.nan)


def test_a_refused_step_keeps_the_rate():
    p, g = torch.zeros(64, device=DEV), torch.ones(64, device=DEV)
    opt = moe.AdamW([p], [g], lr=0.25, weight_decay=0.0)
    with pytest.raises(ValueError, match="grad_scale"):
        opt.step(grad_scale=torch.tensor([1.0]), lr=0.5)
    with pytest.raises(moe.MoEError):
        opt.step(lr=math.inf)
    opt.step()
    # the first step is lr g / (|g| + eps): -0.25 up to roundings of m, v and their corrections
    assert (p + 0.25).abs().max().item() < 0.25 * 2.0 ** -20


def test_overlapping_tensors_are_refused():
    p, g = torch.zeros(1024, device=DEV), torch.zeros(512, device=DEV)
    with pytest.raises(ValueError, match="overlap"):
        moe.AdamW([p[256:768], p[:512]], [g, g], lr=1e-3)
    with pytest.raises(ValueError, match="overlap"):
        moe.AdamW([p[:512], p[256:256 + 64].view(torch.bfloat16)], [g, g[:128]], lr=1e-3)
    moe.AdamW([p[512:], p[:512], p[:0]], [g, g, g[:0]], lr=1e-3)
