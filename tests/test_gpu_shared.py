"""The shared expert (forward, 8-bit checkpoint, backward) against its formulas
in 64 bits.

Every bound is worked out element by element from the roundings that the
interface states: a sum of K products in fp32 is off by at most K 2^-23 of the
sum of their magnitudes (any order, truncation included), a rounding to bf16 (8
significant bits, to nearest) by 2^-8 of the value, the activation and its
derivative by 2^-18 of theirs; the operands rounded to bf16 between two products
carry their error through the second one."""
import math

import pytest
import torch

import mixture_experts_routing_gb300 as moe

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F64 = torch.float64
SIZES = [  # n, h, i
    (1, 8, 32), (1, 520, 160), (2, 72, 96), (7, 128, 64), (16, 264, 288), (17, 1024, 416), (31, 64, 544),
    (37, 520, 128), (64, 256, 256), (65, 136, 32), (128, 512, 1024), (129, 1032, 160), (200, 2048, 768), (257, 328, 320),
    (300, 4096, 1408), (513, 640, 96), (1000, 200, 672), (1, 7168, 2048), (4, 5120, 896), (600, 5120, 896), (1300, 1000, 1888),
]


def act64(g, act):
    if act == moe.ACT_SWIGLU:
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    phi = 0.5 * (1 + torch.erf(g / math.sqrt(2)))
    return g * phi, phi + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)


def kept_values(ck, sf):
    """The 64-bit values of a checkpoint."""
    v = ck.view(torch.float8_e4m3fn).to(F64).view(ck.shape[0], -1, 32)
    s = torch.where(sf == 255, torch.full_like(sf, 0).to(F64) + math.nan, torch.exp2(sf.to(F64) - 127))
    return (v * s.unsqueeze(2)).view(ck.shape)


class Block:
    def __init__(self, n, h, i, act, seed=0, add=True, grad_f32=0, scale=1.0):
        g = torch.Generator(device=DEV)
        g.manual_seed(1000 * n + 10 * h + i + seed)

        def normal(*shape, std=1.0):
            return (torch.randn(shape, device=DEV, generator=g) * std).to(torch.bfloat16)

        self.cfg = moe.SharedConfig(n, h, i, activation=act, grad_f32=grad_f32)
        self.n, self.h, self.i, self.act = n, h, i, act
        self.x, self.dy = normal(n, h, std=scale), normal(n, h)
        self.w13, self.w2 = normal(2 * i, h, std=h ** -0.5), normal(h, i, std=i ** -0.5)
        self.add = normal(n, h) if add else None
        self.hid, self.y = moe.alloc_shared_buffers(self.cfg, DEV)
        self.ck, self.sf = moe.alloc_shared_checkpoint(self.cfg, DEV)
        gt = torch.float32 if grad_f32 else torch.bfloat16
        self.dx = torch.empty_like(self.dy)
        self.dw13 = torch.empty((2 * i, h), dtype=gt, device=DEV)
        self.dw2 = torch.empty((h, i), dtype=gt, device=DEV)
        self.ws = moe.alloc_shared_backward_workspace(self.cfg, DEV)

    def forward(self, train=True, stream=None):
        if train:
            moe.shared_forward_train(self.cfg, self.x, self.w13, self.w2, self.hid, self.y, self.ck, self.sf, add=self.add, stream=stream)
        else:
            moe.shared_forward(self.cfg, self.x, self.w13, self.w2, self.hid, self.y, add=self.add, stream=stream)

    def backward(self, stream=None):
        moe.shared_backward(self.cfg, self.x, self.w13, self.w2, self.ck, self.sf, self.dy, self.dx, self.dw13, self.dw2, self.ws,
                            dx_add=self.add, stream=stream)


def ok():
    torch.cuda.synchronize()
    assert moe.device_error() == 0


def within(got, ref, bound, what):
    d = (got.to(F64) - ref).abs()
    worst = (d - bound).max().item() if d.numel() else 0.0
    assert torch.isfinite(d).all() and worst <= 0, "%s: %.3g over its bound of %.3g" % (what, worst, bound.flatten()[(d - bound).argmax()].item())


def fro(got, ref, limit, what):
    rel = ((got.to(F64) - ref).norm() / ref.norm().clamp(min=1e-300)).item()
    assert rel <= limit, "%s: relative error %.3g" % (what, rel)


def reference_forward(b):
    """y and its bound; g, u and theirs."""
    x, wg, wu, w2 = b.x.to(F64), b.w13[: b.i].to(F64), b.w13[b.i:].to(F64), b.w2.to(F64)
    g, u = x @ wg.t(), x @ wu.t()
    eg, eu = (b.h * 2.0 ** -23 * (x.abs() @ w.abs().t()) for w in (wg, wu))
    a, da = act64(g, b.act)
    h = a * u
    eh = 2.0 ** -8 * h.abs() + 2.0 ** -18 * h.abs() + 1.15 * eg * u.abs() + a.abs() * eu + 1.15 * eg * eu
    y = h @ w2.t()
    ey = eh @ w2.abs().t() + b.i * 2.0 ** -23 * (h.abs() @ w2.abs().t())
    if b.add is not None:
        y = y + b.add.to(F64)
    return y, 2.0 ** -8 * y.abs() + 1.01 * ey, g, eg, u, eu


def check_kept(b, g, eg, u, eu):
    """Every kept value is the nearest one of its block's grid, up to the sum's
    error; the scale is that of the largest value."""
    v, e = torch.cat([g, u], 1).view(b.n, -1, 32), torch.cat([eg, eu], 1).view(b.n, -1, 32)
    top, et = v.abs().amax(2), e.amax(2)

    def exponent(t):
        return (torch.floor(torch.log2(t.clamp(min=1e-300))) - 8).clamp(-127, 127) + 127

    sf = b.sf.to(F64)
    assert ((sf >= exponent((top - et).clamp(min=0))) & (sf <= exponent(top + et))).all()
    s = torch.exp2(sf - 127).unsqueeze(2)
    k = kept_values(b.ck, b.sf).view(v.shape)
    step = torch.exp2(torch.floor(torch.log2((v.abs() / s).clamp(min=2.0 ** -6))) - 3) * s
    over = (v.abs() / s - 448).clamp(min=0) * s
    assert ((k - v).abs() <= 0.5 * step * (1 + 1e-9) + e + over).all()


@pytest.mark.parametrize("act", [moe.ACT_SWIGLU, moe.ACT_GEGLU])
@pytest.mark.parametrize("n,h,i", SIZES)
def test_forward_and_checkpoint(n, h, i, act):
    b = Block(n, h, i, act, add=(n + i) % 3 != 0)
    b.forward()
    ok()
    y, bound, g, eg, u, eu = reference_forward(b)
    within(b.y, y, bound, "y")
    fro(b.y, y, 5e-3, "y")
    check_kept(b, g, eg, u, eu)
    with_checkpoint = b.y.clone()
    b.y.fill_(math.nan)
    b.forward(train=False)
    ok()
    within(b.y, y, bound, "y without a checkpoint")
    fro(b.y, with_checkpoint.to(F64), 5e-3, "y with and without a checkpoint")


def reference_backward(b):
    x, w13, w2, dy = (t.to(F64) for t in (b.x, b.w13, b.w2, b.dy))
    g, u = kept_values(b.ck, b.sf).split(b.i, 1)
    a, s = act64(g, b.act)
    da = dy @ w2
    eda = b.h * 2.0 ** -23 * (dy.abs() @ w2.abs())
    d = torch.cat([da * u * s, da * a], 1)
    slack = 2.0 ** -8 + 2.0 ** -16
    # the derivative's own error, where it is small by cancellation: 2^-18 of its terms
    terms = 1 + g.abs()
    ed = torch.cat([eda * (u * s).abs() + 2.0 ** -18 * (da * u).abs() * terms, eda * a.abs() + 2.0 ** -18 * (da * g).abs()], 1) + slack * d.abs()
    h = a * u
    eh = (slack + 2.0 ** -18) * h.abs()
    dx = d @ w13
    ex = ed @ w13.abs() + 2 * b.i * 2.0 ** -23 * (d.abs() @ w13.abs())
    if b.add is not None:
        dx = dx + b.add.to(F64)
    dw13, dw2 = d.t() @ x, dy.t() @ h
    e13 = ed.t() @ x.abs() + b.n * 2.0 ** -23 * (d.abs().t() @ x.abs())
    e2 = dy.abs().t() @ eh + b.n * 2.0 ** -23 * (dy.abs().t() @ h.abs())
    r = 0.0 if b.cfg.grad_f32 else 2.0 ** -8
    return ((dx, 2.0 ** -8 * dx.abs() + 1.01 * ex), (dw13, r * dw13.abs() + 1.01 * e13), (dw2, r * dw2.abs() + 1.01 * e2))


@pytest.mark.parametrize("act", [moe.ACT_SWIGLU, moe.ACT_GEGLU])
@pytest.mark.parametrize("n,h,i", SIZES)
def test_backward(n, h, i, act):
    b = Block(n, h, i, act, add=(n + i) % 3 != 0, grad_f32=(n + h // 8) % 2)
    b.forward()
    b.backward()
    ok()
    for name, got, (ref, bound) in zip(("dx", "dw13", "dw2"), (b.dx, b.dw13, b.dw2), reference_backward(b)):
        within(got, ref, bound, name)
        fro(got, ref, 5e-3, name)


@pytest.mark.parametrize("grad_f32", [0, 1])
@pytest.mark.parametrize("n,h,i", [
    (1, 5120, 896), (5, 7168, 64), (64, 4096, 2048), (77, 2056, 160), (130, 1032, 1408), (300, 4096, 1408), (1000, 4096, 1408), (700, 264, 2048),
    (1935, 304, 256), (4000, 256, 128), (2001, 520, 512),
])
def test_backward_of_long_contractions(n, h, i, grad_f32):
    """Tiles too few for the SMs: a cluster's pairs share their contractions."""
    b = Block(n, h, i, moe.ACT_SWIGLU, add=n % 2 == 0, grad_f32=grad_f32)
    b.forward()
    b.backward()
    ok()
    for name, got, (ref, bound) in zip(("dx", "dw13", "dw2"), (b.dx, b.dw13, b.dw2), reference_backward(b)):
        within(got, ref, bound, name)
        fro(got, ref, 5e-3, name)
    first = [t.clone() for t in (b.dx, b.dw13, b.dw2)]
    for _ in range(3):
        for t in (b.dx, b.dw13, b.dw2):
            t.fill_(math.nan)
        b.backward()
        ok()
        assert all(torch.equal(t, f) for t, f in zip((b.dx, b.dw13, b.dw2), first))


@pytest.mark.parametrize("act", [moe.ACT_SWIGLU, moe.ACT_GEGLU])
def test_gradients_against_differences(act):
    """Inputs whose pre-activations are whole 8-bit values (few significant
    bits), so that the checkpoint is exact and the gradients are those of the
    forward: each must match the central difference of the loss sum(y dy)."""
    n, h, i = 5, 16, 32
    b = Block(n, h, i, act, add=False, grad_f32=1)
    g = torch.Generator(device=DEV)
    g.manual_seed(7)
    b.x.zero_()
    b.x[:, 0], b.x[:, 1] = 1, torch.tensor([1, -1, 2, 1, -2], device=DEV, dtype=torch.bfloat16)
    b.w13.copy_(torch.randint(-2, 3, b.w13.shape, device=DEV, generator=g) / 4)
    b.forward()
    b.backward()
    ok()
    x, w13, w2, dy = (t.to(F64) for t in (b.x, b.w13, b.w2, b.dy))
    assert torch.equal(kept_values(b.ck, b.sf), x @ w13.t())

    def loss(x, w13, w2):
        p = x @ w13.t()
        return ((act64(p[:, :i], act)[0] * p[:, i:]) @ w2.t() * dy).sum()

    step = 1e-5
    for got, at in ((b.dx, 0), (b.dw13, 1), (b.dw2, 2)):
        args = [x, w13, w2]
        num = torch.zeros_like(args[at])
        for j in range(num.numel()):
            lo, hi = args[at].clone(), args[at].clone()
            lo.view(-1)[j] -= step
            hi.view(-1)[j] += step
            num.view(-1)[j] = (loss(*args[:at], hi, *args[at + 1:]) - loss(*args[:at], lo, *args[at + 1:])) / (2 * step)
        # bf16 operands between the products and, for dx, the result: 2^-8 of the value each; sums whose terms cancel
        # are off by as much of the largest value
        assert ((got.to(F64) - num).abs() <= 2.0 ** -7 * num.abs() + 2.0 ** -7 * num.abs().max()).all()
        fro(got, num, 5e-3, "argument %d" % at)


def test_add_may_be_the_output():
    for n in (3, 70, 300):
        b = Block(n, 264, 96, 0)
        b.forward()
        b.backward()
        y, dx = b.y.clone(), b.dx.clone()
        b.y.copy_(b.add)
        b.dx.copy_(b.add)
        moe.shared_forward(b.cfg, b.x, b.w13, b.w2, b.hid, b.y, add=b.y)
        moe.shared_backward(b.cfg, b.x, b.w13, b.w2, b.ck, b.sf, b.dy, b.dx, b.dw13, b.dw2, b.ws, dx_add=b.dx)
        ok()
        fro(b.y, y.to(F64), 5e-3, "y")
        assert torch.equal(b.dx, dx)


@pytest.mark.parametrize("n,h,i", [(1, 520, 160), (4, 5120, 896), (37, 2048, 768), (100, 512, 416), (1000, 1032, 288), (700, 2048, 1408)])
def test_same_result_every_time_and_on_another_stream(n, h, i):
    b = Block(n, h, i, 1)
    b.forward()
    b.backward()
    ok()
    first = [t.clone() for t in (b.y, b.ck, b.sf, b.dx, b.dw13, b.dw2)]
    s = torch.cuda.Stream()
    for t in (b.y, b.dx, b.dw13, b.dw2):
        t.zero_()
    for t in (b.ck, b.sf):
        t.zero_()
    torch.cuda.synchronize()
    for _ in range(12):
        for _ in range(3):
            b.forward(stream=s)
            b.backward(stream=s)
        ok()
        for got, want in zip((b.y, b.ck, b.sf, b.dx, b.dw13, b.dw2), first):
            assert torch.equal(got, want)


@pytest.mark.parametrize("n,h,i", [(1, 8, 32), (5, 24, 32), (33, 520, 160), (130, 136, 288), (259, 1000, 352)])
def test_nothing_is_written_past_the_outputs(n, h, i):
    b = Block(n, h, i, 0)
    pads = {}

    def padded(t):
        full = torch.full((t.numel() + 4096,), 77, dtype=t.dtype, device=DEV)
        view = full[: t.numel()].view(t.shape)
        pads[id(view)] = (full, t.numel())
        return view

    for name in ("y", "hid", "ck", "sf", "dx", "dw13", "dw2", "ws"):
        setattr(b, name, padded(getattr(b, name)))
    b.forward()
    b.backward()
    ok()
    for full, used in pads.values():
        assert (full[used:] == 77).all()


@pytest.mark.parametrize("n", [2, 20, 90, 300])
def test_a_row_that_is_not_finite_stays_in_its_row(n):
    b = Block(n, 264, 160, 0, add=False)
    b.forward()
    ok()
    y, ck, sf = b.y.clone(), b.ck.clone(), b.sf.clone()
    b.x[n // 2, 3] = math.nan
    b.x[0, 5] = math.inf
    b.forward()
    ok()
    keep = torch.ones(n, dtype=torch.bool, device=DEV)
    keep[[0, n // 2]] = False
    assert torch.equal(b.y[keep], y[keep]) and torch.equal(b.ck[keep], ck[keep]) and torch.equal(b.sf[keep], sf[keep])
    assert torch.isnan(b.y[n // 2]).all() and not torch.isfinite(b.y[0]).any()
    assert (b.sf[n // 2] == 255).all() and (b.sf[0] == 255).all()
    b.backward()
    ok()
    assert torch.isfinite(b.dx[keep]).all() and torch.isnan(b.dx[n // 2]).all()


def test_zero_blocks_and_large_values():
    """Rows of zeros keep the smallest scale and give zero gradients; large
    activations saturate neither the sums nor the scale."""
    b = Block(40, 256, 96, 0, add=False, scale=1e4)
    b.x[3] = 0
    b.forward()
    b.backward()
    ok()
    y, bound, g, eg, u, eu = reference_forward(b)
    within(b.y, y, bound, "y")
    check_kept(b, g, eg, u, eu)
    assert (b.sf[3] == 0).all() and (b.ck[3] & 127 == 0).all() and (b.y[3] == 0).all() and (b.dx[3] == 0).all()


def test_no_token():
    b = Block(0, 72, 96, 0, add=False)
    b.dw13.fill_(5)
    b.dw2.fill_(5)
    b.forward()
    b.forward(train=False)
    b.backward()
    ok()
    assert (b.dw13 == 0).all() and (b.dw2 == 0).all()


def test_offsets_past_32_bits():
    """More than 2^31 checkpoint values: rows at the far end are right."""
    n, h, i = 560_000, 64, 2048
    b = Block(n, h, i, 0, add=False)
    b.forward()
    b.backward()
    ok()
    rows = torch.tensor([0, 1, n // 2, n - 2, n - 1], device=DEV)
    c = Block(len(rows), h, i, 0, add=False)
    c.x, c.dy, c.w13, c.w2, c.ck, c.sf = b.x[rows], b.dy[rows], b.w13, b.w2, b.ck[rows], b.sf[rows]
    y, bound, g, eg, u, eu = reference_forward(c)
    within(b.y[rows], y, bound, "y")
    check_kept(c, g, eg, u, eu)
    dx, bound = reference_backward(c)[0]
    within(b.dx[rows], dx, bound, "dx")


def test_refusals():
    b = Block(4, 72, 96, 0)
    bad = moe.SharedConfig(4, 72, 96)
    with pytest.raises(ValueError):
        moe.shared_forward(b.cfg, b.x[:, ::2], b.w13, b.w2, b.hid, b.y)
    with pytest.raises(ValueError):
        moe.shared_forward(b.cfg, b.x.float(), b.w13, b.w2, b.hid, b.y)
    with pytest.raises(ValueError):
        moe.shared_forward(b.cfg, b.x, b.w13[:-1], b.w2, b.hid, b.y)
    with pytest.raises(ValueError):
        moe.shared_forward(b.cfg, b.x.cpu(), b.w13, b.w2, b.hid, b.y)
    with pytest.raises(ValueError):
        moe.shared_forward(b.cfg, b.x, b.w13, b.w2, b.hid, b.y, add=b.add[:2])
    with pytest.raises(ValueError):
        moe.shared_forward_train(b.cfg, b.x, b.w13, b.w2, b.hid, b.y, b.ck, b.sf[:, :-1])
    with pytest.raises(ValueError):  # f32 gradients need grad_f32
        moe.shared_backward(bad, b.x, b.w13, b.w2, b.ck, b.sf, b.dy, b.dx, b.dw13.float(), b.dw2.float(), b.ws)
    with pytest.raises(moe.MoEError) as e:
        moe.shared_backward(b.cfg, b.x, b.w13, b.w2, b.ck, b.sf, b.dy, b.dx, b.dw13, b.dw2, b.ws[:16])
    assert e.value.status == -3
    full = torch.zeros(4 * 72 + 8, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(moe.MoEError) as e:  # a contiguous view that starts off a 16-byte boundary
        moe.shared_forward(b.cfg, full[1: 1 + 4 * 72].view(4, 72), b.w13, b.w2, b.hid, b.y)
    assert e.value.status == -1
    ok()
