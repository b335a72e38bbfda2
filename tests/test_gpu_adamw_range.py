"""AdamW where one step does not show it: 8-bit states of blocks whose values differ by many
orders of magnitude, both dithers of their codes, weight decay far below a weight's rounding;
tensors that overlap."""
import math

import numpy as np
import pytest
import torch

import mixture_experts_routing_gb300 as moe
from test_gpu_adamw import Set, check, decode
from test_gpu_w4 import DEV, F64, gen, ok

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("b2", [0.95, 0.999])
def test_8_bit_updates_stay_bounded_far_below_the_block_s_largest(b2):
    """In every block some values have the gradient 1 at every step, the others at most q / 2 with
    random signs and many zeros, q = 2^-9 / 448 being the smallest code's value next to the largest.
    The block's largest m is 1 - b1^t and its largest sqrt(v) is sqrt(1 - b2^t); by induction the
    others stay at codes up to 1, and at code 1 exactly for sqrt(v). So an update over lr is at most
    (b1 (1 - b1^(t-1)) q + (1 - b1) |g|) / (1 - b1^t) over the root of
    (b2 (1 - b2^(t-1)) q^2 + (1 - b2) g^2) / (1 - b2^t), which is no more than the sum of the two
    quotients. fp32 and eps are covered by one part in a hundred."""
    n, b1, q, g = 256 * 64, 0.9, 2.0 ** -9 / 448, gen(7)
    p, grad = torch.zeros(n, device=DEV), torch.zeros(n, device=DEV)
    opt = moe.AdamW([p], [grad], lr=1.0, betas=(b1, b2), weight_decay=0.0, state_bits=8)
    size = q / 2 * 10 ** (-4 * torch.rand(n, device=DEV, generator=g))
    for t in range(1, 301):
        grad.copy_(size * torch.sign(torch.rand(n, device=DEV, generator=g) - 0.5) * (torch.rand(n, device=DEV, generator=g) < 0.7))
        grad.view(-1, 256)[:, :8] = 1.0
        p.zero_()
        opt.step()
        c1, c2 = 1 - b1 ** t, 1 - b2 ** t
        bound = (1 - b1) / c1 * math.sqrt(c2 / (1 - b2))
        if t > 1:
            bound += b1 * (1 - b1 ** (t - 1)) / c1 * math.sqrt(c2 / (b2 * (1 - b2 ** (t - 1))))
        assert p.abs().max().item() <= 1.01 * bound, t
    ok()


def test_the_smallest_code_of_a_root():
    """sqrt(v) of a block that is not all zeros has code 1 at least; a block of zeros has code 0."""
    n = 256 * 30
    s = Set([n], True, True, 8)
    g = s.grads[0].view(-1, 256)
    g.mul_(torch.exp(4 * torch.randn(g.shape, device=DEV, generator=gen(1))))
    g[3] = 0
    g[4] *= 1e-36  # its squares are 0 in fp32
    for _ in range(5):
        s.opt.step()
    ok()
    v, m = s.opt.v.view(-1, 256), s.opt.m.view(-1, 256)
    rest = torch.ones(30, dtype=torch.bool, device=DEV)
    rest[3:5] = False
    assert (v[3:5] == 0).all() and (s.opt.v_scale[3:5] == 0).all() and (m[3] & 127 == 0).all()
    assert (v[rest] >= 1).all() and (v[rest] <= 126).all() and (v[rest] == 1).any()
    assert ((m[rest] & 127) == 0).any()  # m is rounded to 0 as to any other code


def test_the_dithers_of_both_states_are_those_of_the_hash():
    """Codes of a step from zero states, value by value: m = 0.1 g takes the lower 16 bits of the
    hash, sqrt(v) = 0.1 |g| the upper ones."""
    n = 70000
    s = Set([n], True, True, 8, betas=(0.9, 0.99), seed=77)
    g = s.grads[0].double().cpu().numpy()
    s.opt.step()
    ok()

    def mix(v):
        v = (v ^ (v >> np.uint32(16))) * np.uint32(0x7FEB352D)
        v = (v ^ (v >> np.uint32(15))) * np.uint32(0x846CA68B)
        return v ^ (v >> np.uint32(16))

    with np.errstate(over="ignore"):
        d = mix(np.arange(n, dtype=np.uint32) * np.uint32(0x9E3779B1) + mix(np.array([0x9E3779B1 + 77], dtype=np.uint32)))
    for codes, value, bits, least in ((s.opt.m, 0.1 * g, d & np.uint32(0xFFFF), 0.0), (s.opt.v, 0.1 * np.abs(g), d >> np.uint32(16), 2.0 ** -9)):
        b, frac = (np.zeros(-(-n // 256) * 256) for _ in range(2))
        b[:n], frac[:n] = value, (bits.astype(np.float64) + 0.5) / 65536
        b, frac = b.reshape(-1, 256), frac.reshape(-1, 256)
        a = np.abs(b) / (np.abs(b).max(1, keepdims=True) / 448)
        step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(a, 2.0 ** -30))), -6) - 3)
        want = np.where(b < 0, -1, 1) * np.clip(np.floor(a / step + frac) * step, least, 448)
        got = codes.view(torch.float8_e4m3fn).double().cpu().numpy().reshape(-1, 256)
        # fp32 puts a value on the other side of its dither with a probability of 2^-20 or so
        assert (got != want).ravel()[:n].mean() < 1e-4


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("lr,decay", [(2.5e-6, 0.01), (1e-5, 0.01), (1e-6, 0.1)])
def test_small_decays_add_up(lr, decay, bits):
    """lr decay is 2.5e-8 to 1e-7, below half a step of an fp32 value next to 1. The shrinkage, as the
    projection on the start of what is left of p once the updates are taken out, against 64 bits. A
    weight (about 0.05, a step of 3.7e-9) is rounded once a step, after an update of some lr, so the
    roundings are independent: 2^-24 of it each at most, over T steps and n values 2^-24 sqrt(T / n) of
    the projection, 6e-9 for T = 2000 and n = 2^18, of which six are 4e-8. T lr decay is 5e-5 at
    least, and 2 % of it 1e-6. The updates' own errors, 2^-19 of lr in sum with random signs, are
    smaller still. 8 bits: the updates follow from the states that were stored."""
    n, T, g = 1 << 18, 2000, gen(3)
    p = torch.randn(n, device=DEV, generator=g) * 0.05
    start, grad = p.to(F64), torch.empty(n, device=DEV)
    opt = moe.AdamW([p], [grad], lr=lr, betas=(0.9, 0.95), weight_decay=decay, state_bits=bits)
    want = start.clone()
    b1, b2 = 0.9, 0.95
    for t in range(1, T + 1):
        grad.normal_(generator=g)
        m = opt.m.to(F64) if bits == 32 else decode(opt.m, opt.m_scale)
        v = opt.v.to(F64) if bits == 32 else decode(opt.v, opt.v_scale).square()
        m, v = b1 * m + (1 - b1) * grad.to(F64), b2 * v + (1 - b2) * grad.to(F64).square()
        want -= lr * (m / (1 - b1 ** t) / (torch.sqrt(v / (1 - b2 ** t)) + 1e-8) + decay * want)
        opt.step()
    ok()
    off = ((p.to(F64) - want) @ start / (start @ start)).item()
    assert abs(off) <= 0.02 * T * lr * decay


def test_gradients_that_overlap_weights_are_refused():
    room = torch.zeros(4096, device=DEV)
    p = room[1024:2048]
    for g in (p, room[512:1536], room[1536:2560], room[1020:2044]):
        with pytest.raises(ValueError, match="overlap"):
            moe.AdamW([p], [g], lr=1e-3)
    q = room[2048:3072]
    with pytest.raises(ValueError, match="overlap"):  # another tensor's weights
        moe.AdamW([p, q], [room[3072:], p], lr=1e-3)
    with pytest.raises(ValueError, match="overlap"):
        moe.AdamW([p], [room.view(torch.bfloat16)[2048:3072]], lr=1e-3)
    # next to each other, and one gradient for two weights
    moe.AdamW([p, q, room[:0]], [room[:1024], room[:1024], room[1100:1100]], lr=1e-3).step()
    ok()


@pytest.mark.parametrize("sizes", [[0] * 300 + [5] + [0] * 300, [9] * 240 + [0] * 3, [9] * 241 + [0] * 240, [0] * 481], ids=lambda s: "%d" % len(s))
def test_empty_tensors_anywhere_in_a_long_list(sizes):
    s = Set(sizes, True, True, 32)
    for t in (1, 2):
        before = s.state()
        s.opt.step()
        ok()
        check(s, before, t)
