"""Products with 4-bit weights against their formulas in 64 bits. The bounds come
from the stated roundings: a sum of C products in fp32 is off by at most
C 2^-23 of the sum of their magnitudes (and the group sums scaled and added by
as much again), a rounding to bf16 by 2^-8, the activation by 2^-18."""
import math

import pytest
import torch

import mixture_experts_routing_gb300 as moe

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F64 = torch.float64


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def normal(g, *shape, std=1.0):
    return (torch.randn(shape, device=DEV, generator=g) * std).to(torch.bfloat16)


def codes(g, *shape):
    return torch.randint(0, 256, shape, dtype=torch.uint8, device=DEV, generator=g)


def weights(q, scale):
    """The 64-bit matrix that codes and scales stand for (last two dimensions)."""
    v = torch.stack([q & 15, q >> 4], -1).flatten(-2).to(F64) - 8
    return v * scale.to(F64).repeat_interleave(v.shape[-1] // scale.shape[-1], -1)


def act64(g, act):
    return g * torch.sigmoid(g) if act == moe.ACT_SWIGLU else g * 0.5 * (1 + torch.erf(g / math.sqrt(2)))


def ok():
    torch.cuda.synchronize()
    assert moe.device_error() == 0


def within(got, ref, bound, what):
    d = (got.to(F64) - ref).abs()
    worst = (d - bound).max().item() if d.numel() else 0.0
    assert torch.isfinite(d).all() and worst <= 0, "%s: %.3g over its bound" % (what, worst)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("rows,cols", [(1, 128), (8, 256), (5, 384), (40, 128), (192, 512), (24, 4096)])
def test_quantize(rows, cols, group):
    m = normal(gen(rows + cols + group), rows, cols, std=0.02)
    m[0, :group] = 0
    q = torch.empty((rows, cols // 2), dtype=torch.uint8, device=DEV)
    s = torch.empty((rows, cols // group), dtype=torch.bfloat16, device=DEV)
    moe.w4_quantize(m, group, q, s)
    ok()
    b = m.to(F64).view(rows, -1, group)
    top = (b.abs().amax(2).float() / 7).to(torch.bfloat16)
    want = torch.where(top > 0, top, torch.ones_like(top))
    assert torch.equal(s, want)
    r = b / want.to(F64).unsqueeze(2)
    v = (torch.stack([q & 15, q >> 4], -1).flatten(-2).to(F64) - 8).view(b.shape)
    # nearest (a tie in the fp32 quotient may go either way), within -8..7
    assert ((v - r.clamp(-8, 7)).abs() <= 0.5 + 2.0 ** -20).all()


MATVEC = [(n, rows, cols, group) for n, rows, cols, group in [
    (1, 1, 128, 128), (1, 7, 32, 32), (1, 16, 64, 64), (1, 4104, 4096, 128), (1, 640, 7168, 128), (2, 33, 160, 32), (3, 17, 96, 32),
    (4, 100, 1408, 128), (5, 50, 192, 64), (7, 64, 2048, 64), (8, 136, 768, 128), (9, 128, 256, 32), (16, 72, 1056, 32), (17, 31, 640, 128),
    (31, 200, 448, 64), (32, 1000, 512, 128), (33, 48, 384, 128), (64, 65, 320, 64), (100, 24, 128, 32), (257, 40, 256, 128), (1024, 16, 64, 32),
]]


@pytest.mark.parametrize("n,rows,cols,group", MATVEC)
def test_matvec(n, rows, cols, group):
    g = gen(n + rows + cols)
    x, q, s = normal(g, n, cols), codes(g, rows, cols // 2), normal(g, rows, cols // group, std=0.02)
    full = torch.full((n * rows + 512,), 77, dtype=torch.bfloat16, device=DEV)
    y = full[: n * rows].view(n, rows)
    moe.w4_matvec(x, q, s, y)
    ok()
    assert (full[n * rows:] == 77).all()
    w = weights(q, s)
    ref = x.to(F64) @ w.t()
    # the codes may enter the sum as code + 128 with the offset taken off afterwards: up to 136 a term
    mag = x.to(F64).abs() @ (136 * s.to(F64).abs().repeat_interleave(group, 1)).t()
    within(y, ref, 2.0 ** -8 * ref.abs() + 2 * cols * 2.0 ** -23 * mag, "y")
    rel = ((y.to(F64) - ref).norm() / ref.norm()).item()
    assert rel <= 5e-3
    again = torch.empty_like(y)
    moe.w4_matvec(x, q, s, again)
    ok()
    assert torch.equal(again, y)


class Batch:
    def __init__(self, n, h, e, k, i, group, act=0, add=True, seed=0):
        g = gen(n + h + e + i + seed)
        self.cfg = moe.W4Config(n, h, e, k, i, group, activation=act)
        self.n, self.h, self.e, self.k, self.i, self.act = n, h, e, k, i, act
        self.x = normal(g, n, h)
        top = torch.randn((n, e), device=DEV, generator=g).topk(k)
        self.ids, self.p = top.indices.to(torch.int32).contiguous(), torch.softmax(top.values, 1).contiguous()
        self.q13, self.s13 = codes(g, e, 2 * i, h // 2), normal(g, e, 2 * i, h // group, std=0.2 * h ** -0.5)
        self.q2, self.s2 = codes(g, e, h, i // 2), normal(g, e, h, i // group, std=0.2 * i ** -0.5)
        self.add = normal(g, n, h) if add else None
        self.y = torch.empty((n, h), dtype=torch.bfloat16, device=DEV)
        self.ws = moe.alloc_w4_workspace(self.cfg, DEV)

    def run(self, stream=None, add=None):
        moe.w4_ffn_forward(self.cfg, self.ids, self.p, self.x, self.q13, self.s13, self.q2, self.s2, self.y, self.ws,
                           add=self.add if add is None else add, stream=stream)

    def reference(self):
        y = self.add.to(F64) if self.add is not None else torch.zeros((self.n, self.h), dtype=F64, device=DEV)
        bound = torch.zeros_like(y)
        for e in range(self.e):
            t, k = (self.ids == e).nonzero(as_tuple=True)
            if not len(t):
                continue
            x = self.x[t].to(F64)
            w13, w2 = weights(self.q13[e], self.s13[e]), weights(self.q2[e], self.s2[e])
            pre, c = x @ w13.t(), self.h // self.s13.shape[-1]
            epre = 2 * self.h * 2.0 ** -23 * (x.abs() @ (136 * self.s13[e].to(F64).abs().repeat_interleave(c, 1)).t())
            g, u = pre.split(self.i, 1)
            eg, eu = epre.split(self.i, 1)
            a = act64(g, self.act)
            hid = a * u
            eh = (2.0 ** -8 + 2.0 ** -18) * hid.abs() + 1.15 * eg * u.abs() + a.abs() * eu + 1.15 * eg * eu
            p = self.p[t, k].to(F64).unsqueeze(1)
            c = self.i // self.s2.shape[-1]
            big = 136 * self.s2[e].to(F64).abs().repeat_interleave(c, 1)
            y.index_add_(0, t, p * (hid @ w2.t()))
            bound.index_add_(0, t, p * (1.01 * eh @ w2.abs().t() + 2 * self.i * 2.0 ** -23 * (hid.abs() @ big.t())))
        return y, bound + 2.0 ** -8 * y.abs()

    def check(self):
        ok()
        y, bound = self.reference()
        within(self.y, y, bound, "y")
        assert ((self.y.to(F64) - y).norm() <= 5e-3 * y.norm()).item()


@pytest.mark.parametrize("act", [moe.ACT_SWIGLU, moe.ACT_GEGLU])
@pytest.mark.parametrize("n,h,e,k,i,group", [
    (1, 128, 1, 1, 128, 128), (1, 32, 3, 2, 64, 32), (1, 1024, 16, 8, 512, 128), (2, 96, 4, 2, 160, 32), (3, 640, 5, 5, 192, 64), (5, 2048, 128, 8, 768, 64),
    (8, 256, 8, 4, 384, 128), (9, 128, 2, 1, 256, 32), (16, 512, 256, 16, 128, 64), (33, 384, 4, 3, 128, 128), (64, 256, 64, 16, 128, 32),
    (100, 128, 1, 1, 96, 32), (128, 256, 16, 8, 192, 64), (1024, 64, 8, 1, 64, 64), (1, 7168, 8, 8, 2048, 128), (40, 4096, 3, 2, 1408, 128),
])
def test_experts(n, h, e, k, i, group, act):
    b = Batch(n, h, e, k, i, group, act, add=n % 2 == 1)
    b.run()
    b.check()


@pytest.mark.parametrize("idle", [0, 3])
@pytest.mark.parametrize("n,h,e,k,i,group", [
    (24, 2080, 40, 4, 1056, 32), (32, 1056, 20, 8, 2080, 32), (32, 1088, 24, 8, 1088, 64), (25, 2112, 70, 3, 1088, 64), (32, 1152, 60, 4, 1280, 128),
])
def test_blocks_that_take_rows_of_several_experts(n, h, e, k, i, group, idle):
    """More items than blocks: runs that begin and end inside an expert's rows,
    last items with fewer tiles than warps, and experts without a route."""
    b = Batch(n, h, e, k, i, group, moe.ACT_SWIGLU, add=True)
    b.ids[n - idle:] = -1
    b.run()
    b.check()


def test_routes_without_an_expert_contribute_nothing():
    for add in (True, False):
        b = Batch(21, 256, 8, 3, 128, 64, add=add)
        b.ids[4] = -1
        b.ids[7, 1] = -1
        b.ids[20] = -1
        b.ids[9, 0] = 8  # past the last expert
        b.p[4] = math.nan
        b.p[7, 1] = math.inf
        b.run()
        b.check()
        want = b.add if add else torch.zeros_like(b.y)
        assert torch.equal(b.y[4], want[4]) and torch.equal(b.y[20], want[20])
        b.ids.fill_(-1)
        b.run()
        ok()
        assert torch.equal(b.y, want)


def test_one_expert_twice_for_a_token_and_one_for_all():
    b = Batch(12, 128, 4, 4, 128, 32)
    b.ids.fill_(2)
    b.ids[5] = torch.tensor([1, 3, 1, 0], dtype=torch.int32, device=DEV)
    b.run()
    b.check()
    b = Batch(64, 128, 4, 4, 128, 32)
    b.ids.fill_(3)
    b.run()
    b.check()


@pytest.mark.parametrize("n", [3, 7, 40])
def test_routes_of_all_kinds_in_one_batch(n):
    """Tokens with an expert twice or three times, an id out of range (and a
    probability that must not count), no expert at all, and all the same one."""
    b = Batch(n, 256, 6, 4, 192, 64)
    b.ids[0] = torch.tensor([2, 5, 2, 2], dtype=torch.int32, device=DEV)
    b.ids[1] = torch.tensor([-1, 3, 6, 3], dtype=torch.int32, device=DEV)
    b.p[1, 0], b.p[1, 2] = math.nan, math.inf
    b.ids[2] = -1
    b.ids[4:] = torch.tensor([5, 5, 0, 1], dtype=torch.int32, device=DEV)
    b.run()
    b.check()
    assert torch.equal(b.y[2], b.add[2])


@pytest.mark.parametrize("n", [1, 6, 50])
def test_same_result_every_time_on_another_stream_and_in_place(n):
    b = Batch(n, 512, 16, 4, 256, 64)
    b.run()
    ok()
    first = b.y.clone()
    s = torch.cuda.Stream()
    for _ in range(3):
        b.y.zero_()
        torch.cuda.synchronize()
        b.run(stream=s)
        ok()
        assert torch.equal(b.y, first)
    b.y.copy_(b.add)
    b.run(add=b.y)
    ok()
    assert torch.equal(b.y, first)


def test_nothing_is_written_past_the_outputs_and_rows_stay_apart():
    b = Batch(19, 96, 5, 3, 160, 32, add=False)
    full = torch.full((19 * 96 + 256,), 77, dtype=torch.bfloat16, device=DEV)
    used = moe.w4_workspace_bytes(b.cfg)
    ws = torch.full((used + 256,), 77, dtype=torch.uint8, device=DEV)
    b.y, b.ws = full[: 19 * 96].view(19, 96), ws[:used]
    b.run()
    b.check()
    assert (full[19 * 96:] == 77).all() and (ws[used:] == 77).all()
    first = b.y.clone()
    b.x[6, 3] = math.nan
    b.run()
    ok()
    keep = torch.arange(19, device=DEV) != 6
    assert torch.equal(b.y[keep], first[keep]) and torch.isnan(b.y[6]).all()


def test_weights_past_32_bits_of_bytes():
    """An expert whose weights lie beyond 2^32 bytes."""
    n, h, e, k, i = 2, 4096, 256, 2, 4224
    b = Batch(n, h, e, k, i, 128)
    assert b.q13.numel() > 2 ** 32
    b.ids.copy_(torch.tensor([[255, 0], [254, 255]], dtype=torch.int32))
    b.run()
    b.check()


def test_a_whole_decode_step():
    """Routes of route_align, weights quantised by the library: the experts in 4
    bits plus the shared expert, against the bf16 experts to within what 4 bits lose."""
    n, h, e, k, i, group = 24, 256, 8, 2, 128, 32
    g = gen(3)
    cfg = moe.Config(n, h, e, k, i, cap_num=e, cap_den=1, block_m=16)
    x, wr = normal(g, n, h), torch.randn((h, e), device=DEV, generator=g) * 0.1
    w13, w2 = normal(g, e, 2 * i, h, std=h ** -0.5), normal(g, e, h, i, std=i ** -0.5)
    routes, ws = moe.alloc_routes(cfg, DEV), moe.alloc_workspace(cfg, DEV)
    hid, o, want = moe.alloc_buffers(cfg, DEV)
    moe.forward(cfg, x, wr, None, w13, w2, routes, ws, hid, o, want)
    wq = moe.W4Weights(w13, w2, group)
    c4 = moe.W4Config(n, h, e, k, i, group)
    y = torch.empty((n, h), dtype=torch.bfloat16, device=DEV)
    moe.w4_ffn_forward(c4, routes.topk_ids, routes.topk_p, x, wq.w13q, wq.w13_scale, wq.w2q, wq.w2_scale, y,
                       moe.alloc_w4_workspace(c4, DEV))
    ok()
    # a code is within half a step of amax/7 (~0.17 deviations for a group of 32 normal values): about
    # 0.1 of each weight in the mean square, in three factors
    rel = ((y.double() - want.double()).norm() / want.double().norm()).item()
    assert rel < 0.3
    shared = moe.SharedConfig(n, h, i)
    sw13, sw2 = normal(g, 2 * i, h, std=h ** -0.5), normal(g, h, i, std=i ** -0.5)
    sh, sy = moe.alloc_shared_buffers(shared, DEV)
    moe.shared_forward(shared, x, sw13, sw2, sh, sy)
    routed = y.clone()
    moe.shared_forward(shared, x, sw13, sw2, sh, y, add=y)
    ok()
    assert ((y.double() - routed.double() - sy.double()).norm() <= 1e-2 * y.double().norm()).item()


def test_refusals():
    b = Batch(2, 128, 4, 2, 128, 64)
    with pytest.raises(ValueError):
        moe.w4_matvec(b.x, b.q13[0][:, ::2], b.s13[0], b.y)
    with pytest.raises(ValueError):
        moe.w4_matvec(b.x.float(), b.q13[0], b.s13[0], b.y)
    with pytest.raises(ValueError):
        moe.w4_matvec(b.x.cpu(), b.q13[0], b.s13[0], b.y)
    y = torch.empty((2, 256), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(moe.MoEError) as e:  # one scale for 16 columns
        moe.w4_matvec(b.x, b.q13[0], torch.ones((256, 8), dtype=torch.bfloat16, device=DEV), y)
    assert e.value.status == -1
    b.ids = b.ids.long()
    with pytest.raises(ValueError):
        b.run()
    b.ids = b.ids.int()
    b.ws = b.ws[:16]
    with pytest.raises(moe.MoEError) as e:
        b.run()
    assert e.value.status == -3
    with pytest.raises(moe.MoEError) as e:
        moe.w4_workspace_bytes(moe.W4Config(600, 128, 4, 2, 128, 64))
    assert e.value.status == -2
    ok()
