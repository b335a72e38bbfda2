"""The whole layer for a few tokens against its formulas in 64 bits, element by element.

A sum of C products in fp32 is a chain of at most C / 16 steps of the tensor cores (each
within 17 2^-23 of its 16 products' magnitudes, which the C / 16 steps share) and of 40
more additions: (C / 16 + 57) 2^-23 of the sum of magnitudes, truncation included. A logit
is a chain of at most H / 8 + 24 fp32 additions of half a step each. A rounding to bf16
takes 2^-8, the activation 2^-18."""
import math

import pytest
import torch

import mixture_experts_routing_gb300 as moe
from test_gpu_w4 import DEV, F64, act64, gen, normal, ok, within

pytestmark = pytest.mark.gpu


def sum_error(c):
    return (c / 16 + 57) * 2.0 ** -23


class Layer:
    def __init__(self, n, h, e, k, i, act=0, renorm=1, bias=True, add=True, seed=0):
        g = gen(n + h + e + i + 13 * k + seed)
        self.n, self.h, self.e, self.k, self.i, self.act, self.renorm = n, h, e, k, i, act, renorm
        self.cfg = moe.FewConfig(n, h, e, k, i, renorm=renorm, activation=act)
        self.x = normal(g, n, h)
        self.wr = torch.randn((h, e), device=DEV, generator=g) * h ** -0.5
        self.b = 0.3 * torch.randn(e, device=DEV, generator=g) if bias else None
        self.w13 = torch.empty((e, 2 * i, h), dtype=torch.bfloat16, device=DEV).normal_(std=h ** -0.5, generator=g)
        self.w2 = torch.empty((e, h, i), dtype=torch.bfloat16, device=DEV).normal_(std=i ** -0.5, generator=g)
        self.add = normal(g, n, h) if add else None
        self.y = torch.full((n, h), math.nan, dtype=torch.bfloat16, device=DEV)
        self.ids = torch.full((n, k), -7, dtype=torch.int32, device=DEV)
        self.p = torch.full((n, k), -7.0, device=DEV)
        self.ws = moe.alloc_few_workspace(self.cfg, DEV).fill_(0xFF)

    def run(self, **kw):
        kw = dict(add=self.add, topk_ids=self.ids, topk_p=self.p) | kw
        moe.few_forward(self.cfg, self.x, self.wr, self.b, self.w13, self.w2, self.y, self.ws, **kw)

    def check(self, live=None):
        """The choice, then the outputs of the experts that were chosen: against a bound of every rounding, and
        against the rows' size, which outputs of zeros do not meet."""
        n = self.n if live is None else live
        x, wr = self.x[:n].to(F64), self.wr.to(F64)
        logits = x @ wr + (0 if self.b is None else self.b.to(F64))
        dl = (self.h / 8 + 24) * 2.0 ** -24 * (x.abs() @ wr.abs()) + 2.0 ** -24 * logits.abs()
        ids, p = self.ids[:n].long(), self.p[:n].to(F64)
        assert (ids >= 0).all() and (ids < self.e).all() and all(len(set(r)) == self.k for r in ids.tolist())
        # the choice goes by probabilities: under exp(-87) of the largest they are 0 in fp32, hence equal
        logits = torch.maximum(logits, logits.amax(1, keepdim=True) - 87)
        chosen = logits.gather(1, ids)
        dc = dl.gather(1, ids)
        top = dl.amax(1, keepdim=True)
        if self.k < self.e:
            rest = logits.scatter(1, ids, -math.inf).amax(1, keepdim=True)
            assert (chosen >= rest - 2 * top - 2.0 ** -20).all(), "an expert of a smaller logit"
        assert (chosen[:, :-1] >= chosen[:, 1:] - 2 * top - 2.0 ** -20).all(), "not in descending order"
        q = torch.softmax(logits, 1).gather(1, ids)
        if self.renorm:
            q = q / q.sum(1, keepdim=True)
        dq = q * (torch.expm1(2 * (top + dc)) + 2.0 ** -18) + 1e-30
        within(p, q, dq, "p")
        part = torch.zeros((n, self.h), dtype=F64, device=DEV)
        bound = torch.zeros_like(part)
        for e in ids.unique().tolist():
            t, k = (ids == e).nonzero(as_tuple=True)
            w13, w2 = self.w13[e].to(F64), self.w2[e].to(F64)
            (g, u), (eg, eu) = ((v.split(self.i, 1)) for v in (x[t] @ w13.t(), sum_error(self.h) * (x[t].abs() @ w13.abs().t())))
            a = act64(g, self.act)
            hid = a * u
            eh = (2.0 ** -8 + 2.0 ** -18) * hid.abs() + 1.15 * eg * u.abs() + a.abs() * eu + 1.15 * eg * eu
            pe = p[t, k].unsqueeze(1)  # the probabilities as they are: their own error is checked above
            part.index_add_(0, t, pe * (hid @ w2.t()))
            m = hid.abs() @ w2.abs().t()
            bound.index_add_(0, t, pe * (1.01 * eh @ w2.abs().t() + (sum_error(self.i) + (8 + self.k) * 2.0 ** -23) * m))
        add = 0 if self.add is None else self.add[:n].to(F64)
        y = part + add
        total = bound + 2.0 ** -8 * y.abs() + self.k * 2.0 ** -23 * (0 if self.add is None else add.abs())
        within(self.y[:n], y, total, "y")
        # roundings of the hidden values are independent: a small part of the row's size in all
        d = (self.y[:n].to(F64) - y).abs()
        rms = part.square().mean(1, keepdim=True).sqrt()
        assert (d <= 2.0 ** -8 * y.abs() + 2.0 ** -5 * rms + 1e-30).all()


CASES = [
    (1, 64, 1, 1, 64), (1, 64, 3, 2, 128), (1, 128, 256, 16, 64), (1, 7168, 16, 8, 2048), (2, 192, 5, 5, 192), (3, 640, 33, 4, 320), (4, 1024, 8, 2, 512),
    (5, 2048, 128, 8, 768), (7, 4096, 64, 6, 1408), (8, 256, 9, 3, 448), (8, 512, 1, 1, 1024), (9, 512, 2, 1, 1024), (15, 576, 7, 7, 576), (16, 512, 8, 2, 1024),
    (17, 128, 3, 3, 64), (24, 1088, 40, 4, 1088), (31, 320, 256, 1, 64), (33, 2048, 128, 8, 768), (40, 4096, 3, 2, 1408), (48, 192, 31, 16, 960),
    (57, 960, 6, 2, 832), (63, 512, 100, 12, 128), (64, 512, 8, 2, 1024), (64, 64, 2, 2, 64), (64, 1024, 1, 1, 512), (64, 7168, 4, 4, 256), (2, 16384, 2, 1, 64),
    (2, 64, 2, 1, 16384), (64, 16384, 3, 1, 64), (64, 128, 16, 16, 4096),
]


@pytest.mark.parametrize("act", [moe.ACT_SWIGLU, moe.ACT_GEGLU])
@pytest.mark.parametrize("n,h,e,k,i", CASES)
def test_layer(n, h, e, k, i, act):
    s = Layer(n, h, e, k, i, act, renorm=(n + act) % 2, bias=(n + e + act) % 2 == 0, add=(n + k + act) % 2 == 0)
    s.run()
    ok()
    s.check()
    first = s.y.clone()
    s.y.fill_(math.nan)
    s.run()
    ok()
    assert torch.equal(first, s.y)
    s.run(topk_ids=None, topk_p=None)
    ok()
    assert torch.equal(first, s.y)


def test_one_expert_for_all_and_all_for_each():
    s = Layer(64, 512, 32, 1, 256, bias=True)
    s.b.fill_(0)
    s.b[17] = 1e4
    s.run()
    ok()
    assert (s.ids == 17).all() and (s.p == 1).all()
    s.check()
    s = Layer(64, 256, 16, 16, 128)
    s.run()
    ok()
    s.check()


@pytest.mark.parametrize("e", [6, 16, 200])
@pytest.mark.parametrize("live", [0, 1, 7, 8, 9, 20, 33])
def test_rows_behind_the_live_ones_are_left(live, e):
    s = Layer(33, 512, e, 4, 256)
    s.x[live:] = math.nan
    s.add[live:] = math.nan
    n = torch.tensor([live], dtype=torch.int32, device=DEV)
    s.y.fill_(3.0)
    s.run(n_valid=n)
    ok()
    assert (s.y[live:] == 3).all() and (s.ids[live:] == -7).all() and (s.p[live:] == -7).all()
    if live:
        s.check(live)
    for over, want in ((1000, 33), (-5, 0)):
        n.fill_(over)
        s.x.nan_to_num_(0.5)
        s.add.nan_to_num_(0.5)
        s.y.fill_(3.0)
        s.run(n_valid=n)
        ok()
        if want:
            s.check()
        else:
            assert (s.y == 3).all()


def test_the_addend_is_the_output():
    s = Layer(9, 640, 12, 3, 320)
    s.run()
    y = s.add.clone()
    want = s.y.clone()
    moe.few_forward(s.cfg, s.x, s.wr, s.b, s.w13, s.w2, y, s.ws, add=y)
    ok()
    assert torch.equal(y, want)


@pytest.mark.parametrize("n,h,e,k,i", [(1, 7168, 16, 8, 2048), (33, 2048, 128, 8, 768), (64, 512, 8, 2, 1024), (20, 1024, 2, 1, 64)])
def test_the_output_in_the_place_of_the_input(n, h, e, k, i):
    """x += layer(x): no block may write a row that another still reads."""
    s = Layer(n, h, e, k, i)
    s.add = s.x.clone()
    s.run()
    x = s.x.clone()
    for _ in range(20):
        x.copy_(s.x)
        moe.few_forward(s.cfg, x, s.wr, s.b, s.w13, s.w2, x, s.ws, add=x)
        ok()
        assert torch.equal(x, s.y)


@pytest.mark.parametrize("k", [2, 5])
def test_experts_shut_out_are_not_read(k):
    s = Layer(20, 256, 8, k, 128)
    s.b.zero_()
    s.b[[1, 2, 4, 6, 7]] = -math.inf  # three stay: with five picks two of no probability fill up
    s.w13[[1, 2, 4, 6, 7]] = math.nan
    s.w2[[1, 2, 4, 6, 7]] = math.inf
    s.run()
    ok()
    assert torch.isfinite(s.y).all()
    live = s.p > 0
    assert torch.isin(s.ids[live], torch.tensor([0, 3, 5], device=DEV)).all() and live.sum(1).eq(min(k, 3)).all()
    s.w13.nan_to_num_(0)
    s.w2[[1, 2, 4, 6, 7]] = 0
    s.b.masked_fill_(s.b == -math.inf, -1e3)
    before = s.y.clone()
    s.run()
    ok()
    s.check()
    assert torch.equal(before, s.y)


def test_a_bad_row_stays_alone():
    s = Layer(10, 256, 8, 2, 128)
    s.run()
    clean, ids = s.y.clone(), s.ids.clone()
    s.x[3, 5], s.x[6, 200] = math.nan, math.inf
    s.run()
    ok()
    keep = [0, 1, 2, 4, 5, 7, 8, 9]
    assert torch.equal(s.y[keep], clean[keep]) and torch.equal(s.ids[keep], ids[keep])
    assert s.y[3].isnan().all() and s.p[3].isnan().all() and s.y[6].isnan().any()
    assert (s.ids >= 0).all() and (s.ids < 8).all()
    s.b.fill_(-math.inf)  # nothing is left for any row
    s.run()
    ok()
    assert s.y.isnan().all() and s.p.isnan().all() and (s.ids >= 0).all() and (s.ids < 8).all()


def test_a_bad_weight_reaches_its_tokens_only():
    s = Layer(16, 256, 8, 2, 128, add=False)
    s.run()
    clean, ids = s.y.clone(), s.ids.clone()
    s.w2[5, 100, 3] = math.nan
    s.run()
    ok()
    hit = (ids == 5).any(1)
    assert hit.any() and not hit.all()
    assert s.y[hit, 100].isnan().all()
    s.y[hit, 100] = clean[hit, 100]
    assert torch.equal(s.y, clean)


@pytest.mark.parametrize("e", [7, 8, 40, 256])
def test_equal_logits_go_to_the_lower_experts(e):
    s = Layer(12, 128, e, 6, 64, bias=False)
    s.wr.zero_()
    s.run()
    ok()
    assert torch.equal(s.ids, torch.arange(6, dtype=torch.int32, device=DEV).expand(12, 6)) and torch.allclose(s.p, torch.full_like(s.p, 1 / 6))
    s.check()


def test_values_around_the_outputs_are_left():
    s = Layer(11, 192, 10, 3, 64)
    s.run()
    ok()
    y = torch.full((11 * 192 + 64,), 7.0, dtype=torch.bfloat16, device=DEV)
    ids, p = torch.full((33 + 16,), 7, dtype=torch.int32, device=DEV), torch.full((33 + 16,), 7.0, device=DEV)
    need = moe.few_workspace_bytes(s.cfg)
    ws = torch.full((need + 256,), 9, dtype=torch.uint8, device=DEV)
    moe.few_forward(s.cfg, s.x, s.wr, s.b, s.w13, s.w2, y[: 11 * 192].view(11, 192), ws[:need], add=s.add, topk_ids=ids[:33].view(11, 3), topk_p=p[:33].view(11, 3))
    ok()
    assert torch.equal(y[: 11 * 192].view(11, 192), s.y) and (y[11 * 192:] == 7).all() and (ids[33:] == 7).all() and (p[33:] == 7).all() and (ws[need:] == 9).all()


def test_captured_graphs_that_share_a_workspace():
    big, small = Layer(33, 512, 16, 4, 256), Layer(3, 512, 16, 4, 256, seed=1)
    small.wr, small.b, small.w13, small.w2 = big.wr, big.b, big.w13, big.w2
    small.ws = big.ws
    graphs = []
    live = torch.tensor([33], dtype=torch.int32, device=DEV)
    for s in (big, small):
        s.run(n_valid=live) if s is big else s.run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.run(n_valid=live) if s is big else s.run()
        graphs.append(g)
    for n in (33, 5, 33, 0, 12):
        live.fill_(n)
        big.y.fill_(math.nan)
        small.y.fill_(math.nan)
        for g in (graphs[0], graphs[1], graphs[0]):
            g.replay()
        ok()
        if n:
            big.check(n)
        assert big.y[n:].isnan().all()
        small.check()


def test_two_streams_at_once():
    a, b = Layer(8, 2048, 32, 8, 768), Layer(20, 1024, 64, 4, 512)
    a.run()
    b.run()
    torch.cuda.synchronize()
    ya, yb = a.y.clone(), b.y.clone()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(100):
        a.run(stream=s)
        b.run(stream=t)
    ok()
    assert torch.equal(a.y, ya) and torch.equal(b.y, yb)


def test_shared_workspace_from_call_to_call():
    """Calls of unlike shapes one after another through one workspace, as a model's layers do."""
    shapes = [(5, 512, 16, 4, 256), (64, 256, 8, 2, 128), (1, 1024, 32, 8, 512), (33, 192, 100, 3, 320), (1, 1024, 32, 8, 512)]
    layers = [Layer(*s) for s in shapes]
    ws = torch.full((max(moe.few_workspace_bytes(s.cfg) for s in layers),), 0xAB, dtype=torch.uint8, device=DEV)
    for s in layers:
        s.ws = ws
    for _ in range(3):
        for s in layers:
            s.run()
    ok()
    for s in layers:
        s.check()


def test_the_ordinary_forward_agrees():
    s = Layer(64, 512, 8, 2, 1024, add=False, bias=True)
    s.run()
    cfg = moe.Config(64, 512, 8, 2, 1024, cap_num=0, cap_den=1, block_m=16)
    routes, ws = moe.alloc_routes(cfg, DEV), moe.alloc_workspace(cfg, DEV)
    h, o, y = moe.alloc_buffers(cfg, DEV)
    moe.forward(cfg, s.x, s.wr, s.b, s.w13, s.w2, routes, ws, h, o, y)
    ok()
    assert torch.equal(routes.topk_ids, s.ids)  # no near ties among these inputs
    assert torch.allclose(routes.topk_p, s.p, rtol=1e-5)
    # two roundings of o and y there, one here, the same h up to summation order: 3 2^-8 of the rows' size
    assert ((s.y.double() - y.double()).norm() / y.double().norm()).item() < 3 * 2.0 ** -8


def test_weights_behind_2_32_bytes():
    n, h, e, k, i = 3, 7168, 256, 4, 2048  # 15 GB of w13, 7.5 GB of w2; the last experts are chosen
    s = Layer(n, h, 4, k, i)
    w13 = torch.zeros((e, 2 * i, h), dtype=torch.bfloat16, device=DEV)
    w2 = torch.zeros((e, h, i), dtype=torch.bfloat16, device=DEV)
    w13[-4:], w2[-4:] = s.w13, s.w2
    b = torch.full((e,), -math.inf, device=DEV)
    b[-4:] = s.b if s.b is not None else 0
    wr = torch.zeros((h, e), device=DEV)
    wr[:, -4:] = s.wr
    s.run()
    cfg = moe.FewConfig(n, h, e, k, i, renorm=s.renorm)
    y, ids = torch.empty_like(s.y), torch.empty_like(s.ids)
    moe.few_forward(cfg, s.x, wr, b, w13, w2, y, moe.alloc_few_workspace(cfg, DEV), add=s.add, topk_ids=ids)
    ok()
    assert torch.equal(ids, s.ids + 252)
    s.check()
    # the same sums but for the logits' order of columns
    assert ((y.double() - s.y.double()).norm() / s.y.double().norm()).item() < 2.0 ** -8


def test_a_router_that_lies_at_an_odd_place():
    s = Layer(5, 256, 12, 3, 128)
    s.run()
    want = s.y.clone()
    room = torch.zeros(256 * 12 + 1, device=DEV)
    room[1:] = s.wr.flatten()
    s.wr = room[1:].view(256, 12)  # 4-byte aligned alone
    bias = torch.zeros(13, device=DEV)
    bias[1:] = s.b if s.b is not None else 0
    s.b = bias[1:]
    s.y.fill_(math.nan)
    s.run()
    ok()
    assert torch.equal(s.y, want)
    s.check()


def test_the_current_stream_is_the_one_taken():
    s = Layer(9, 512, 16, 4, 256)
    s.run()
    torch.cuda.synchronize()
    want = s.y.clone()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        s.x.mul_(2)  # the call has to come after this and before the next
        s.run()
        doubled = s.y.clone()
        s.x.mul_(0.5)
        s.run()
    side.synchronize()
    ok()
    assert torch.equal(s.y, want) and not torch.equal(doubled, want)


def test_no_tokens():
    s = Layer(0, 128, 4, 2, 64)
    s.run()
    ok()


def test_refusals():
    s = Layer(4, 128, 8, 2, 64)
    y = s.y
    for match, kw in (("x must be", dict(x=s.x.float())), ("w_router must be", dict(wr=s.wr.t().contiguous().t())), ("bias must be", dict(b=s.b[:7] if s.b is not None else s.wr[0, :7])),
                      ("w13 must be", dict(w13=s.w13[:, :64])), ("w2 must be", dict(w2=s.w2[:7])), ("y must be", dict(y=y[:, :64]))):
        a = dict(x=s.x, wr=s.wr, b=s.b, w13=s.w13, w2=s.w2, y=y) | kw
        with pytest.raises(ValueError, match=match):
            moe.few_forward(s.cfg, a["x"], a["wr"], a["b"], a["w13"], a["w2"], a["y"], s.ws)
    for name, t in (("add", s.add.float() if s.add is not None else s.wr), ("n_valid", torch.tensor([4], device=DEV)), ("topk_ids", s.ids.long()), ("topk_p", s.p.double())):
        with pytest.raises(ValueError, match=name):
            moe.few_forward(s.cfg, s.x, s.wr, s.b, s.w13, s.w2, y, s.ws, **{name: t})
    with pytest.raises(moe.MoEError) as e:
        moe.few_forward(s.cfg, s.x, s.wr, s.b, s.w13, s.w2, y, s.ws[: moe.few_workspace_bytes(s.cfg) - 16].clone())
    assert e.value.status == -3
