"""Layer norm and its RMS form, forward and backward, against their formulas in 64 bits.

Bounds: a row's sum is a chain of at most 16 columns a thread, 5 steps of lanes and 32 of
warps, 53 additions of half a step each; E = 64 2^-24 leaves room for the products' own
roundings. The mean is off by E times the mean magnitude; the variance by 2 E of itself and
by the square of the mean's error; r by half of that relative to var + eps and a few
roundings. A rounding to bf16 is off by 2^-8."""
import math

import pytest
import torch

import mixture_experts_routing_gb300 as moe
from test_gpu_w4 import DEV, F64, gen, normal, ok, within

pytestmark = pytest.mark.gpu

E = 64 * 2.0 ** -24
SHAPES = [(1, 8), (2, 8), (1, 7168), (3, 16), (5, 24), (7, 64), (4, 72), (33, 256), (9, 264), (300, 520), (65, 1000), (17, 1032), (1001, 2048),
          (40, 2056), (130, 4104), (600, 7168), (3, 8192), (50, 8200), (2, 16376), (400, 16384), (5000, 64), (3001, 128), (20000, 8)]
KINDS = [moe.NORM_LAYER, moe.NORM_RMS]


class Rows:
    def __init__(self, n, h, kind, add=True, bias=True, eps=1e-5, seed=0):
        g = gen(n * 7 + h + kind + seed)
        self.n, self.h, self.kind, self.eps = n, h, kind, eps
        self.cfg = moe.NormConfig(n, h, kind=kind, eps=eps)
        size = torch.exp(torch.randn((n, 1), device=DEV, generator=g))
        self.x = ((torch.randn((n, h), device=DEV, generator=g) + 0.3) * size).to(torch.bfloat16)
        self.add = normal(g, n, h) if add else None
        self.w = 1 + 0.3 * torch.randn(h, device=DEV, generator=g)
        self.b = torch.randn(h, device=DEV, generator=g) if bias else None
        self.dy, self.res = normal(g, n, h), normal(g, n, h)

    def forward(self, **kw):
        bf, f = dict(dtype=torch.bfloat16, device=DEV), dict(device=DEV)
        self.sum = torch.full((self.n, self.h), math.nan, **bf) if self.add is not None else None
        self.y = torch.full((self.n, self.h), math.nan, **bf)
        self.mean = torch.full((self.n,), math.nan, **f) if self.kind == moe.NORM_LAYER else None
        self.rstd = torch.full((self.n,), math.nan, **f)
        moe.norm_forward(self.cfg, self.x, self.w, self.y, bias=self.b, add=self.add, sum=self.sum, mean=self.mean, rstd=self.rstd, **kw)

    def backward(self, add=True, **kw):
        self.dx = torch.full((self.n, self.h), math.nan, dtype=torch.bfloat16, device=DEV)
        self.dw = torch.full((self.h,), math.nan, device=DEV)
        self.db = torch.full((self.h,), math.nan, device=DEV) if self.b is not None else None
        ws = moe.alloc_norm_backward_workspace(self.cfg, DEV)
        moe.norm_backward(self.cfg, self.x if self.sum is None else self.sum, self.w, self.mean, self.rstd, self.dy, self.dx, self.dw, ws,
                          dbias=self.db, dx_add=self.res if add else None, **kw)


def check_forward(r, ref_x=None):
    s = (r.x if ref_x is None else ref_x).to(F64)
    if r.add is not None:
        s = (s + r.add.to(F64)).to(torch.bfloat16)  # the sum of two bf16 values is exact in 64 bits
        assert torch.equal(r.sum, s)
        s = s.to(F64)
    c, dmean = s, torch.zeros((r.n, 1), dtype=F64, device=DEV)
    if r.kind == moe.NORM_LAYER:
        mean = s.mean(1, keepdim=True)
        dmean = E * s.abs().mean(1, keepdim=True)
        within(r.mean, mean[:, 0], dmean[:, 0], "mean")
        c = s - mean
    var = c.square().mean(1, keepdim=True)
    rs = 1 / torch.sqrt(var + r.eps)
    dr = rs * ((2 * E * var + dmean.square()) / (var + r.eps) + 2.0 ** -22)
    within(r.rstd, rs[:, 0], dr[:, 0], "rstd")
    y = c * rs * r.w.to(F64) + (0 if r.b is None else r.b.to(F64))
    err = r.w.to(F64).abs() * (rs * (dmean + 2.0 ** -23 * c.abs()) + c.abs() * dr) * 1.01 + 2.0 ** -23 * (c * rs * r.w.to(F64)).abs()
    within(r.y, y, 1.01 * err + (2.0 ** -8 + 2.0 ** -23) * y.abs() + 1e-38, "y")


def check_backward(r, add=True):
    s = (r.x if r.sum is None else r.sum).to(F64)
    rs, dy, w = r.rstd.to(F64).unsqueeze(1), r.dy.to(F64), r.w.to(F64)
    z = (s if r.mean is None else s - r.mean.to(F64).unsqueeze(1)) * rs
    g = dy * w
    mz, mg = (g * z).mean(1, keepdim=True), g.mean(1, keepdim=True) if r.kind == moe.NORM_LAYER else torch.zeros_like(rs)
    dx = rs * (g - z * mz - mg)
    err = rs * (2.0 ** -21 * (g.abs() + (z * mz).abs() + mg.abs()) + z.abs() * 2 * E * (g * z).abs().mean(1, keepdim=True)
                + (E * g.abs().mean(1, keepdim=True) if r.kind == moe.NORM_LAYER else 0))
    if add:
        dx = dx + r.res.to(F64)
        err = err + 2.0 ** -23 * r.res.to(F64).abs()
    within(r.dx, dx, 1.01 * err + (2.0 ** -8 + 2.0 ** -23) * dx.abs() + 1e-38, "dx")
    # a chain of a part's rows (128 parts or more where there are as many rows), then of at most 640 parts
    chain = (r.n / min(r.n, 128) + 640 + 8) * 2.0 ** -24
    within(r.dw, (dy * z).sum(0), (chain + 2.0 ** -22) * (dy * z).abs().sum(0) + 1e-38, "dw")
    if r.db is not None:
        within(r.db, dy.sum(0), chain * dy.abs().sum(0), "db")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n,h", SHAPES)
def test_forward_and_backward(n, h, kind):
    r = Rows(n, h, kind, add=(n + h // 8) % 2 == 0, bias=(n + h // 16) % 2 == 0)
    r.forward()
    ok()
    check_forward(r)
    add = n % 3 != 0
    r.backward(add)
    ok()
    check_backward(r, add)
    first = [t.clone() for t in (r.y, r.dx, r.dw)]
    r.forward()
    r.backward(add)
    ok()
    assert all(torch.equal(a, b) for a, b in zip(first, (r.y, r.dx, r.dw)))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("add,bias", [(False, False), (True, False), (False, True), (True, True)])
def test_every_optional_argument(kind, add, bias):
    r = Rows(37, 1040, kind, add=add, bias=bias)
    r.forward()
    r.backward(add=not add)
    ok()
    check_forward(r)
    check_backward(r, add=not add)
    y = torch.empty_like(r.y)  # without the statistics
    moe.norm_forward(r.cfg, r.x, r.w, y, bias=r.b, add=r.add, sum=torch.empty_like(y) if add else None)
    ok()
    assert torch.equal(y, r.y)


@pytest.mark.parametrize("kind", KINDS)
def test_outputs_in_place(kind):
    a, b = Rows(70, 2064, kind), Rows(70, 2064, kind)
    a.forward()
    a.backward()
    x = b.x.clone()
    b.y, b.mean, b.rstd = torch.empty_like(x), None if a.mean is None else torch.empty_like(a.mean), torch.empty_like(a.rstd)
    moe.norm_forward(b.cfg, b.x, b.w, b.y, bias=b.b, add=b.add, sum=b.x, mean=b.mean, rstd=b.rstd)  # the residual stream in place
    b.sum, dx, dw, db = b.x, b.dy.clone(), torch.empty_like(a.dw), torch.empty_like(a.db)
    moe.norm_backward(b.cfg, b.x, b.w, b.mean, b.rstd, dx, dx, dw, moe.alloc_norm_backward_workspace(b.cfg, DEV), dbias=db, dx_add=b.res)
    dx2 = b.res.clone()
    moe.norm_backward(b.cfg, b.x, b.w, b.mean, b.rstd, b.dy, dx2, dw, moe.alloc_norm_backward_workspace(b.cfg, DEV), dbias=db, dx_add=dx2)
    c = Rows(70, 2064, kind, add=False)
    c.forward()
    want, y = c.y.clone(), c.x.clone()
    moe.norm_forward(c.cfg, y, c.w, y, bias=c.b)
    add2 = b.add.clone()
    y2 = torch.empty_like(add2)
    moe.norm_forward(b.cfg, x, b.w, y2, bias=b.b, add=add2, sum=add2)
    ok()
    assert torch.equal(b.x, a.sum) and torch.equal(b.y, a.y)
    assert torch.equal(dx, a.dx) and torch.equal(dx2, a.dx) and torch.equal(dw, a.dw) and torch.equal(db, a.db)
    assert torch.equal(y, want) and torch.equal(add2, a.sum) and torch.equal(y2, a.y)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("eps", [0.0, 1e-6, 1.0])
def test_constant_tiny_and_unlike_rows(kind, eps):
    r = Rows(8, 1024, kind, add=False, eps=eps)
    r.x[0] = 3.0
    r.x[1] *= 1e-3
    r.x[2] *= 1e8
    r.x[3] = r.x[3] * 0.01 + 100  # a mean far larger than the deviation
    if eps == 0.0:
        r.x[0, ::2] = 1.0  # not constant: 0 / 0 otherwise
    r.forward()
    r.backward()
    ok()
    c = r.x.to(F64) - (r.x.to(F64).mean(1, keepdim=True) if kind == moe.NORM_LAYER else 0)
    none = c.square().mean(1) + eps == 0  # row 3 of the layer norm is 100 throughout in bf16: 0 / 0 without eps
    assert none.sum().item() == (eps == 0.0 and kind == moe.NORM_LAYER)
    assert r.y[none].isnan().all() and r.rstd[none].isinf().all()
    r.n, r.cfg.n_tokens = 8 - int(none.sum()), 8 - int(none.sum())
    for name in ("x", "y", "rstd", "dy", "res") + (("mean",) if kind == moe.NORM_LAYER else ()):
        setattr(r, name, getattr(r, name)[~none].contiguous())
    check_forward(r)
    r.backward()  # without that row, whose gradient would reach every column's sum
    ok()
    check_backward(r)


@pytest.mark.parametrize("kind", KINDS)
def test_infinities_and_nan_stay_in_their_rows(kind):
    r = Rows(6, 520, kind, add=False, bias=False)
    r.forward()
    clean = r.y.clone()
    r.x[1, 7], r.x[3, 500], r.x[4, 0] = math.nan, math.inf, -math.inf
    r.forward()
    ok()
    for t in (0, 2, 5):
        assert torch.equal(r.y[t], clean[t])
    assert r.y[1].isnan().all() and r.y[3, 500].isnan() and r.y[4, 0].isnan()


def test_no_rows():
    for kind in KINDS:
        r = Rows(0, 128, kind)
        r.forward()
        r.backward()
        ok()
        assert (r.dw == 0).all() and (r.db == 0).all()


@pytest.mark.parametrize("kind", KINDS)
def test_values_around_the_rows_are_left(kind):
    n, h = 19, 1096
    r = Rows(n, h, kind)
    r.forward()
    r.backward()
    ok()
    bufs = {k: torch.full((n * h + 64,), 7.0, dtype=torch.bfloat16, device=DEV) for k in ("sum", "y", "dx")}
    vecs = {k: torch.full((m + 16,), 7.0, device=DEV) for k, m in (("mean", n), ("rstd", n), ("dw", h), ("db", h))}
    v = {k: t[: n * h].view(n, h) for k, t in bufs.items()} | {k: vecs[k][:m] for k, m in (("mean", n), ("rstd", n), ("dw", h), ("db", h))}
    mean = v["mean"] if kind == moe.NORM_LAYER else None
    moe.norm_forward(r.cfg, r.x, r.w, v["y"], bias=r.b, add=r.add, sum=v["sum"], mean=mean, rstd=v["rstd"])
    need = moe.norm_backward_workspace_bytes(r.cfg)
    ws = torch.full((need + 256,), 9, dtype=torch.uint8, device=DEV)
    moe.norm_backward(r.cfg, v["sum"], r.w, mean, v["rstd"], r.dy, v["dx"], v["dw"], ws[:need], dbias=v["db"], dx_add=r.res)
    ok()
    assert all((t[n * h:] == 7).all() for t in bufs.values()) and (ws[need:] == 9).all()
    assert all((vecs[k][m:] == 7).all() for k, m in (("rstd", n), ("dw", h), ("db", h)))
    assert torch.equal(v["y"], r.y) and torch.equal(v["dx"], r.dx) and torch.equal(v["dw"], r.dw) and torch.equal(v["db"], r.db)


@pytest.mark.parametrize("kind", KINDS)
def test_gradient_against_differences(kind):
    """sum(dy * norm(x)) along a direction, by a central difference in 64 bits."""
    r = Rows(12, 256, kind)
    r.forward()
    r.backward(add=False)
    ok()
    g = gen(5)
    d, dw, db = (torch.randn(s, device=DEV, generator=g, dtype=F64) for s in ((12, 256), (256,), (256,)))

    def loss(t):
        c = r.sum.to(F64) + t * d
        if kind == moe.NORM_LAYER:
            c = c - c.mean(1, keepdim=True)
        y = c / torch.sqrt(c.square().mean(1, keepdim=True) + r.eps) * (r.w.to(F64) + t * dw) + r.b.to(F64) + t * db
        return (y * r.dy.to(F64)).sum()

    slope = (loss(1e-5) - loss(-1e-5)) / 2e-5
    got = (r.dx.to(F64) * d).sum() + (r.dw.to(F64) * dw).sum() + (r.db.to(F64) * db).sum()
    # each of dx's roundings is 2^-8 of it at most; their sum along d, and the difference's own error
    room = 2.0 ** -8 * (r.dx.to(F64) * d).abs().sum() + 1e-6 * slope.abs() + 1e-4
    assert (got - slope).abs() <= room


def test_captured_and_on_another_stream():
    r = Rows(90, 2048, moe.NORM_LAYER)
    r.forward()
    r.backward()
    ok()
    want = [t.clone() for t in (r.sum, r.y, r.mean, r.rstd, r.dx, r.dw, r.db)]
    ws = moe.alloc_norm_backward_workspace(r.cfg, DEV)

    def both(stream=None):
        moe.norm_forward(r.cfg, r.x, r.w, r.y, bias=r.b, add=r.add, sum=r.sum, mean=r.mean, rstd=r.rstd, stream=stream)
        moe.norm_backward(r.cfg, r.sum, r.w, r.mean, r.rstd, r.dy, r.dx, r.dw, ws, dbias=r.db, dx_add=r.res, stream=stream)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    side = torch.cuda.Stream()
    for go in (graph.replay, graph.replay, lambda: both(side)):
        for t in (r.sum, r.y, r.dx, r.dw):
            t.fill_(math.nan)
        torch.cuda.synchronize()
        go()
        ok()
        assert all(torch.equal(a, b) for a, b in zip(want, (r.sum, r.y, r.mean, r.rstd, r.dx, r.dw, r.db)))


def test_more_than_2_31_values():
    n, h = 262400, 8192  # 2.15e9 values; rows past the border are checked
    x = torch.zeros((n, h), dtype=torch.bfloat16, device=DEV)
    tail = Rows(64, h, moe.NORM_RMS, add=False, bias=False)
    x[-64:] = tail.x
    y, rstd = torch.zeros_like(x), torch.empty(n, device=DEV)
    cfg = moe.NormConfig(n, h, kind=moe.NORM_RMS)
    moe.norm_forward(cfg, x, tail.w, y, rstd=rstd)
    tail.forward()
    ok()
    assert torch.equal(y[-64:], tail.y) and torch.equal(rstd[-64:], tail.rstd) and (y[:100] == 0).all()
    dy = torch.zeros_like(x)
    dy[-64:] = tail.dy
    dw = torch.empty(h, device=DEV)
    moe.norm_backward(cfg, x, tail.w, None, rstd, dy, y, dw, moe.alloc_norm_backward_workspace(cfg, DEV))
    tail.backward(add=False)
    ok()
    assert torch.equal(y[-64:], tail.dx) and (y[:100] == 0).all()
    z = tail.x.to(F64) * tail.rstd.to(F64).unsqueeze(1)
    within(dw, (tail.dy.to(F64) * z).sum(0), (n / 128 + 700) * 2.0 ** -24 * (tail.dy.to(F64) * z).abs().sum(0), "dw")


def test_refusals():
    r = Rows(4, 64, moe.NORM_LAYER)
    y = torch.empty_like(r.x)
    with pytest.raises(ValueError, match="y must be"):
        moe.norm_forward(r.cfg, r.x, r.w, y.float())
    with pytest.raises(ValueError, match="weight must be"):
        moe.norm_forward(r.cfg, r.x, r.w.to(torch.bfloat16), y)
    with pytest.raises(ValueError, match="x must be"):
        moe.norm_forward(r.cfg, r.x.t().contiguous().t(), r.w, y)
    with pytest.raises(moe.MoEError):
        moe.norm_forward(r.cfg, r.x, r.w, y, add=r.add)
