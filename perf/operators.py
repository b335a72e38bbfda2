"""Cases of the shared expert (a gated feed-forward block that every token passes), of its training
step from 8-bit activation checkpoints, and of the products with 4-bit weights that serve a few
tokens, with the plain form of each and its definition in 64 bits.

Layouts, as in the framework's header: x, y, add, dy, dx [N, H] bf16; w13 [2I, H] bf16, gate rows
then up rows; w2 [H, I] bf16. A checkpoint holds the pre-activations [g | u] of a row as E4M3 codes
[N, 2I] and one E8M0 byte per 32 of them [N, 2I/32]: value = code * 2^(byte - 127). A 4-bit matrix
[R, C] holds two values a byte, column 2j in the low half of byte j, as value + 8, and one bf16
scale per `group` columns: weight = scale * value.
"""
import math

import torch

own = False

SWIGLU, GEGLU = 0, 1


def listed():
    return [
        # one token of a decode step through the shared expert of the largest layer (latency, weights read once)
        dict(name="forward_1", op="forward", n=1, h=7168, i=2048, act=SWIGLU, add=True),
        # a small ragged decode batch on the small layer, the exact GELU form
        dict(name="forward_37_geglu", op="forward", n=37, h=2048, i=768, act=GEGLU, add=True),
        # a chunk of prompt tokens, its length no multiple of a tile
        dict(name="forward_500", op="forward", n=500, h=4096, i=1408, act=SWIGLU, add=False),
        # prefill of a whole batch on the largest layer
        dict(name="forward_4096", op="forward", n=4096, h=7168, i=2048, act=SWIGLU, add=True),
        # a training step (forward that keeps its 8-bit checkpoint, then backward) on a ragged short batch
        dict(name="step_1000_geglu", op="step", n=1000, h=4096, i=1408, act=GEGLU, add=True),
        # a training step on a long batch of the small layer
        dict(name="step_8192", op="step", n=8192, h=2048, i=768, act=SWIGLU, add=True),
        # the backward alone on a tiny layer with odd sizes (tails in every dimension)
        dict(name="backward_77", op="backward", n=77, h=520, i=160, act=SWIGLU, add=False),
        # the backward alone on the largest layer: most work of all cases
        dict(name="backward_4096", op="backward", n=4096, h=7168, i=2048, act=SWIGLU, add=True),
        # one token's eight routed experts out of 256, 4-bit weights (the latency of a decode step)
        dict(name="experts_1", op="experts", n=1, h=7168, i=2048, e=256, k=8, group=128, act=SWIGLU, add=True, idle=0),
        # a decode batch that hits most experts, several tokens sharing one, with two idle rows
        dict(name="experts_33", op="experts", n=33, h=2048, i=768, e=128, k=8, group=64, act=SWIGLU, add=False, idle=2),
        # one token through one 4-bit projection
        dict(name="matvec_1", op="matvec", n=1, rows=7168, cols=7168, group=128),
        # a few tokens through a 4-bit projection with the finest groups, rows no multiple of a tile
        dict(name="matvec_13", op="matvec", n=13, rows=4104, cols=4096, group=32),
    ]


def _log(rng, low, high, unit=1):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high))) / unit)) * unit))


def draw(rng):
    op = rng.choice(["forward", "step", "backward", "experts", "matvec"])
    act, add = rng.choice([SWIGLU, GEGLU]), rng.random() < 0.5
    if op == "matvec":
        group = rng.choice([32, 64, 128])
        rows, cols = _log(rng, 64, 8192, 8), _log(rng, 128, 7168, group)
        return dict(op=op, n=_log(rng, 1, 32), rows=rows + 8 * (rows == 3072), cols=cols + group * (cols == 3072), group=group)
    if op == "experts":
        group, e = rng.choice([32, 64, 128]), _log(rng, 1, 64)
        h, i = _log(rng, 128, 4096, group), _log(rng, 128, 1408, group)
        h += group * (h == 3072)
        n = _log(rng, 1, 32)
        return dict(op=op, n=n, h=h, i=i, e=e, k=rng.randint(1, min(8, e)), group=group, act=act, add=add, idle=rng.choice([0, n // 8]))
    h, i = _log(rng, 128, 7168, 8), _log(rng, 64, 2048, 32)
    return dict(op=op, n=_log(rng, 1, 4096), h=h + 8 * (h == 3072), i=i + 32 * (i == 1536), act=act, add=add)


def work(case):
    op, n = case["op"], case["n"]
    if op == "matvec":
        rows, cols = case["rows"], case["cols"]
        return {"bytes": rows * cols / 2 + rows * cols / case["group"] * 2 + 2 * n * (rows + cols), "flops": 2 * n * rows * cols}
    h, i = case["h"], case["i"]
    if op == "experts":
        live, e = n - case["idle"], case["e"]
        hit = e * (1 - (1 - case["k"] / e) ** live)  # experts that some token chose: its expected value
        return {"bytes": hit * 3 * h * i * (0.5 + 2 / case["group"]) + 2 * n * h * (2 + case["add"]) + 8 * n * case["k"],
                "flops": 6 * live * case["k"] * h * i}
    weights, rows, kept = 2 * 3 * h * i, 2 * n * h, 2 * n * i * (1 + 1 / 32)
    if op == "forward":
        return {"bytes": weights + rows * (2 + case["add"]), "flops": 6 * n * h * i}
    if op == "backward":  # x, dy, dx, the checkpoint; weights read, their gradients written
        return {"bytes": 2 * weights + rows * (3 + case["add"]) + kept, "flops": 12 * n * h * i}
    return {"bytes": 3 * weights + rows * (5 + 2 * case["add"]) + 2 * kept, "flops": 18 * n * h * i}


def _nibbles(rows, cols, gen):
    """4-bit codes of bell-shaped weights: each half of a byte is the sum of two uniform numbers of 3 bits, plus 1 (values -7 .. 7)."""
    a = torch.randint(0, 256, (rows, cols // 2), dtype=torch.uint8, device="cuda", generator=gen)
    b = torch.randint(0, 256, (rows, cols // 2), dtype=torch.uint8, device="cuda", generator=gen)
    return a.bitwise_and_(0x77).add_(b.bitwise_and_(0x77)).add_(0x11)


def _scales(rows, cols, group, std, gen):
    """Group scales of weights of the given deviation, each within a fifth of its mean."""
    u = torch.rand((rows, cols // group), device="cuda", generator=gen)
    return ((0.8 + 0.4 * u) * (std / 3.24)).to(torch.bfloat16)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    n, op = case["n"], case["op"]

    def normal(*shape, std=1.0):
        return (torch.randn(shape, device="cuda", generator=gen) * std).to(torch.bfloat16)

    s = {"op": op, "n": n}
    if op == "matvec":
        rows, cols, group = case["rows"], case["cols"], case["group"]
        s |= {"x": normal(n, cols), "q": _nibbles(rows, cols, gen), "scale": _scales(rows, cols, group, cols ** -0.5, gen), "group": group}
        s["y"] = torch.empty((n, rows), dtype=torch.bfloat16, device="cuda")
        return s
    h, i = case["h"], case["i"]
    s |= {"h": h, "i": i, "act": case["act"], "x": normal(n, h), "add": normal(n, h) if case["add"] else None}
    s["y"] = torch.empty((n, h), dtype=torch.bfloat16, device="cuda")
    if op == "experts":
        e, k, group = case["e"], case["k"], case["group"]
        s |= {"group": group, "e": e, "k": k}
        top = torch.randn((n, e), device="cuda", generator=gen).topk(k)
        p = torch.softmax(top.values, 1)
        ids = top.indices.to(torch.int32)
        if case["idle"]:  # rows past the live tokens of a batch hold no expert
            ids[-case["idle"]:] = -1
            p[-case["idle"]:] = 0
        s |= {"ids": ids.contiguous(), "p": p.contiguous()}
        s["q13"], s["s13"] = _nibbles(e * 2 * i, h, gen).view(e, 2 * i, h // 2), _scales(e * 2 * i, h, group, h ** -0.5, gen).view(e, 2 * i, h // group)
        s["q2"], s["s2"] = _nibbles(e * h, i, gen).view(e, h, i // 2), _scales(e * h, i, group, i ** -0.5, gen).view(e, h, i // group)
        if own:  # the plan and scratch that a serving program keeps
            import mixture_experts_routing_gb300 as moe
            s["cfg"] = moe.W4Config(n, h, e, k, i, group, activation=case["act"])
            s["ws"] = moe.alloc_w4_workspace(s["cfg"], "cuda")
        return s
    # weights that keep unit inputs near unit size, as trained ones do
    s |= {"w13": normal(2 * i, h, std=h ** -0.5), "w2": normal(h, i, std=i ** -0.5)}
    bf16 = dict(dtype=torch.bfloat16, device="cuda")
    if op != "backward":
        s["hid"] = torch.empty((n, i), **bf16)
    if op != "forward":
        s["dy"] = normal(n, h)
        s |= {"dx": torch.empty((n, h), **bf16), "dw13": torch.empty((2 * i, h), **bf16), "dw2": torch.empty((h, i), **bf16)}
        if op == "backward":  # what the forward kept: pre-activations of unit size in 8 bits
            s["ck"], s["sf"] = _keep(torch.randn((n, 2 * i), device="cuda", generator=gen))
        else:
            s["ck"], s["sf"] = torch.empty((n, 2 * i), dtype=torch.uint8, device="cuda"), torch.empty((n, 2 * i // 32), dtype=torch.uint8, device="cuda")
    if own:  # the shape, and the scratch that a program keeps
        import mixture_experts_routing_gb300 as moe
        s["cfg"] = moe.SharedConfig(n, h, i, activation=case["act"])
        if op != "forward":
            s["ws"] = moe.alloc_shared_backward_workspace(s["cfg"], "cuda")
    return s


# ------------------------------------------------------------------ plain form (32 bits)
def _keep(v):
    """E4M3 codes and E8M0 bytes of the rows of v, one scale 2^(floor(log2 max|v|) - 8) per 32 values."""
    b = v.float().view(v.shape[0], -1, 32)
    top = b.abs().amax(2)
    s = torch.where(top > 0, torch.frexp(top).exponent - 9, -127).clamp(-127, 127)
    scaled = torch.ldexp(b, -s.unsqueeze(2)).clamp(-448, 448)
    codes = scaled.to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.view(v.shape), (s + 127).to(torch.uint8)


def _kept(codes, sf):
    """The values that a checkpoint stands for."""
    b = codes.view(torch.float8_e4m3fn).float().view(codes.shape[0], -1, 32)
    return torch.ldexp(b, (sf.int() - 127).unsqueeze(2)).view(codes.shape)


def _core(g, act):
    """act(g) = g c(g): c is the logistic function or the normal distribution's."""
    return torch.sigmoid(g) if act == SWIGLU else 0.5 * (1 + torch.erf(g * math.sqrt(0.5)))


def _slope(g, c, act):
    return c * (1 + g * (1 - c)) if act == SWIGLU else c + g * torch.exp(-0.5 * g * g) * (1 / math.sqrt(2 * math.pi))


def _plain_forward(s):
    pre = s["x"].float() @ s["w13"].float().t()
    g, u = pre[:, : s["i"]], pre[:, s["i"]:]
    y = (g * _core(g, s["act"]) * u) @ s["w2"].float().t()
    return (y if s["add"] is None else y + s["add"].float()).to(torch.bfloat16), pre


def _plain_backward(s, ck, sf):
    pre = _kept(ck, sf)
    g, u = pre[:, : s["i"]], pre[:, s["i"]:]
    c = _core(g, s["act"])
    dy = s["dy"].float()
    da = dy @ s["w2"].float()
    d = torch.cat([da * u * _slope(g, c, s["act"]), da * g * c], 1)
    dx = d @ s["w13"].float()
    if s["add"] is not None:
        dx = dx + s["add"].float()
    dw13, dw2 = d.t() @ s["x"].float(), dy.t() @ (g * c * u)
    return {"dx": dx.to(torch.bfloat16), "dw13": dw13.to(torch.bfloat16), "dw2": dw2.to(torch.bfloat16)}


def _weights(q, scale, group):
    """A 4-bit matrix (the last two dimensions) in 32 bits."""
    v = torch.stack([q.bitwise_and(15), q.bitwise_right_shift(4)], -1).flatten(-2).float().sub_(8)
    return v.view(*scale.shape, group).mul_(scale.float().unsqueeze(-1)).flatten(-2)


def _plain_experts(s):
    n, k = s["ids"].shape
    live = (s["ids"] >= 0).flatten()
    at = s["ids"].flatten().clamp(min=0).long()
    x = s["x"].float().repeat_interleave(k, 0).unsqueeze(2)
    pre = torch.bmm(_weights(s["q13"][at], s["s13"][at], s["group"]), x).squeeze(2)
    g, u = pre[:, : s["i"]], pre[:, s["i"]:]
    o = torch.bmm(_weights(s["q2"][at], s["s2"][at], s["group"]), (g * _core(g, s["act"]) * u).unsqueeze(2)).squeeze(2)
    o = torch.where(live.unsqueeze(1), o * s["p"].flatten().unsqueeze(1), torch.zeros_like(o))
    y = o.view(n, k, -1).sum(1)
    return (y if s["add"] is None else y + s["add"].float()).to(torch.bfloat16)


def run(state):
    s = state
    op = s["op"]
    if own:
        import mixture_experts_routing_gb300 as moe
        if op == "matvec":
            moe.w4_matvec(s["x"], s["q"], s["scale"], s["y"])
            return {"y": s["y"]}
        if op == "experts":
            moe.w4_ffn_forward(s["cfg"], s["ids"], s["p"], s["x"], s["q13"], s["s13"], s["q2"], s["s2"], s["y"], s["ws"], add=s["add"])
            return {"y": s["y"]}
        if op == "forward":
            moe.shared_forward(s["cfg"], s["x"], s["w13"], s["w2"], s["hid"], s["y"], add=s["add"])
            return {"y": s["y"]}
        if op == "step":
            moe.shared_forward_train(s["cfg"], s["x"], s["w13"], s["w2"], s["hid"], s["y"], s["ck"], s["sf"], add=s["add"])
        moe.shared_backward(s["cfg"], s["x"], s["w13"], s["w2"], s["ck"], s["sf"], s["dy"], s["dx"], s["dw13"], s["dw2"], s["ws"], dx_add=s["add"])
        out = {"dx": s["dx"], "dw13": s["dw13"], "dw2": s["dw2"]}
        return out | {"y": s["y"]} if op == "step" else out
    if op == "matvec":
        return {"y": (s["x"].float() @ _weights(s["q"], s["scale"], s["group"]).t()).to(torch.bfloat16)}
    if op == "experts":
        return {"y": _plain_experts(s)}
    if op == "backward":
        return _plain_backward(s, s["ck"], s["sf"])
    y, pre = _plain_forward(s)
    return _plain_backward(s, *_keep(pre)) | {"y": y} if op == "step" else {"y": y}


# ------------------------------------------------------------------ the definition in 64 bits
def _act64(g, act):
    """act and its derivative."""
    if act == SWIGLU:
        e = torch.exp(-g)
        return g / (1 + e), (1 + e + g * e) / (1 + e) ** 2
    phi = torch.special.ndtr(g)
    return g * phi, phi + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)


def _e4m3_64(v):
    """The nearest E4M3 value (ties to the even code): 4 significant bits, steps of 2^-9 at least, at most 448."""
    step = torch.exp2(torch.clamp(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -60))), min=-6) - 3)
    return torch.clamp(torch.round(v / step) * step, -448, 448)


def _kept64(v):
    out = torch.empty_like(v).view(-1, 32)
    b = v.reshape(-1, 32)
    top = b.abs().amax(1, keepdim=True)
    s = torch.where(top > 0, torch.floor(torch.log2(top)) - 8, torch.full_like(top, -127)).clamp(-127, 127)
    out.copy_(_e4m3_64(b / torch.exp2(s)) * torch.exp2(s))
    return out.view(v.shape)


def _open64(q, scale, group):
    w = torch.empty((q.shape[0], 2 * q.shape[1]), dtype=torch.float64, device=q.device)
    w[:, 0::2] = (q % 16).double() - 8
    w[:, 1::2] = (q // 16).double() - 8
    return w * scale.double().repeat_interleave(group, 1)


def exact(case, seed):
    s = prepare(case, seed)
    x = s["x"].double()
    if s["op"] == "matvec":
        return {"y": torch.einsum("nc,rc->nr", x, _open64(s["q"], s["scale"], s["group"]))}
    i, add = s["i"], s["add"].double() if s["add"] is not None else torch.zeros_like(x)
    if s["op"] == "experts":
        y = add.clone()
        for e in sorted(set(s["ids"].flatten().tolist()) - {-1}):
            t, k = (s["ids"] == e).nonzero(as_tuple=True)
            w13, w2 = _open64(s["q13"][e], s["s13"][e], s["group"]), _open64(s["q2"][e], s["s2"][e], s["group"])
            a, _ = _act64(x[t] @ w13[:i].t(), s["act"])
            y.index_add_(0, t, s["p"][t, k].double().unsqueeze(1) * ((a * (x[t] @ w13[i:].t())) @ w2.t()))
        return {"y": y}
    gate, up, w2 = s["w13"][:i].double(), s["w13"][i:].double(), s["w2"].double()
    out = {}
    if s["op"] == "backward":
        b = s["ck"].view(torch.float8_e4m3fn).double().view(-1, 32) * torch.exp2(s["sf"].double().view(-1, 1) - 127)
        g, u = b.view(s["n"], 2 * i).split(i, 1)
    else:
        g, u = x @ gate.t(), x @ up.t()
        a, _ = _act64(g, s["act"])
        out["y"] = (a * u) @ w2.t() + add
        g, u = _kept64(g.contiguous()), _kept64(u.contiguous())
    if s["op"] != "forward":
        dy = s["dy"].double()
        a, da = _act64(g, s["act"])
        dh = dy @ w2
        dg, du = dh * u * da, dh * a
        out["dx"] = dg @ gate + du @ up + add
        out["dw13"], out["dw2"] = torch.cat([dg.t() @ x, du.t() @ x]), dy.t() @ (a * u)
    return out
