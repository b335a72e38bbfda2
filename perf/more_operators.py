"""Cases of the whole layer for a few tokens, of layer norm with its backward, and of the AdamW step over
many tensors, with the plain form of each and its definition in 64 bits.

Layouts, as in the framework's header. Layer: x, y, add [N, H] bf16; w_router [H, E] f32, bias [E] f32;
w13 [E, 2I, H] bf16 (gate rows, then up rows), w2 [E, H, I] bf16. Norm: rows [N, H] bf16, weight and bias
[H] f32. AdamW: the tensors' values lie in flat buffers, each tensor from a multiple of 256 on; 8-bit
states are E4M3 codes with one f32 scale per 256 values (m = code * scale, sqrt(v) = code * scale).
"""
import math

import torch

own = False

SWIGLU, GEGLU = 0, 1
LAYER, RMS = 0, 1
BLOCK = 256  # values that share a scale of an 8-bit state


def listed():
    return [
        # one token of a decode step through the largest layer: eight experts' weights read once
        dict(name="few_1", op="few", n=1, h=7168, i=2048, e=256, k=8, act=SWIGLU, renorm=1, bias=False, add=True, idle=0),
        # a handful of tokens on the dropless layer, the exact GELU form, a router bias, probabilities kept as they are
        dict(name="few_7_geglu", op="few", n=7, h=4096, i=1408, e=64, k=6, act=GEGLU, renorm=0, bias=True, add=False, idle=0),
        # a ragged decode batch on the small layer that hits most experts, captured for 33 tokens and holding 31
        dict(name="few_33", op="few", n=33, h=2048, i=768, e=128, k=8, act=SWIGLU, renorm=1, bias=True, add=True, idle=2),
        # many tokens for each of few experts, tiny weights
        dict(name="few_64", op="few", n=64, h=512, i=1024, e=8, k=2, act=SWIGLU, renorm=1, bias=False, add=True, idle=0),
        # the norm in front of the layer in a decode step (latency)
        dict(name="norm_1", op="norm", n=1, h=7168, kind=RMS, add=True, bias=False),
        # prefill or training of a batch on the largest layer
        dict(name="norm_4096", op="norm", n=4096, h=7168, kind=LAYER, add=True, bias=True),
        # the backward on a short ragged batch and a width that is no multiple of a warp's reach
        dict(name="norm_grad_1001", op="norm_grad", n=1001, h=4104, kind=RMS, add=False, bias=False),
        # the backward of a long batch of narrow rows: the sum over rows is the longest
        dict(name="norm_grad_16384", op="norm_grad", n=16384, h=2048, kind=LAYER, add=True, bias=True),
        # the backward of a batch on the largest layer
        dict(name="norm_grad_4096", op="norm_grad", n=4096, h=7168, kind=LAYER, add=True, bias=True),
        # a router, its bias and two norms: fp32 weights and gradients, a few small tensors (latency)
        dict(name="adamw_small", op="adamw", sizes="262144,128,2048,2048,2047", bits=32, wide=True, grad32=True),
        # a shared expert: three large bf16 matrices with fp32 masters and bf16 gradients
        dict(name="adamw_shared", op="adamw", sizes="29360128,14680064,7168", bits=32, wide=False, grad32=False),
        # the experts of a layer one tensor each, with router, bias and norms: fp32 gradients, 8-bit states
        dict(name="adamw_8bit", op="adamw", sizes="16*11534336,16*5767168,65536,16,4096,4096,999", bits=8, wide=False, grad32=True),
    ]


def _log(rng, low, high, unit=1):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high))) / unit)) * unit))


def draw(rng):
    op = rng.choice(["few", "few", "norm", "norm_grad", "adamw"])
    add, bias = rng.random() < 0.5, rng.random() < 0.5
    if op == "few":
        h, i, e = _log(rng, 128, 4096, 64), _log(rng, 64, 1408, 64), _log(rng, 1, 128)
        k = rng.randint(1, min(8, e))
        n = max(1, min(_log(rng, 1, 64), int(1e9 / (3 * h * i * k))))
        return dict(op=op, n=n, h=h, i=i, e=e, k=k, act=rng.choice([SWIGLU, GEGLU]), renorm=rng.choice([0, 1]), bias=bias, add=add, idle=rng.choice([0, n // 8]))
    if op == "adamw":
        sizes = [_log(rng, 100, 10_000_000) for _ in range(rng.randint(1, 12))]
        return dict(op=op, sizes=",".join(map(str, sizes)), bits=rng.choice([8, 32]), wide=rng.random() < 0.5, grad32=rng.random() < 0.5)
    h = _log(rng, 64, 8192, 8)
    return dict(op=op, n=max(1, min(_log(rng, 1, 16384), 29_000_000 // h)), h=h, kind=rng.choice([LAYER, RMS]), add=add, bias=bias)


def _sizes(case):
    """The tensors' lengths: "a,3*b" is a, b, b, b."""
    out = []
    for s in case["sizes"].split(","):
        times, _, size = s.rpartition("*")
        out += [int(size)] * int(times or 1)
    return out


def work(case):
    op = case["op"]
    if op == "adamw":
        n, state = sum(_sizes(case)), 8 if case["bits"] == 32 else 2 + 8 / BLOCK
        weight = 8 if case["wide"] else 8 + 2  # f32, or an f32 master and the bf16 weight made from it
        return {"bytes": n * ((4 if case["grad32"] else 2) + weight + 2 * state), "flops": 16 * n}
    n, h = case["n"], case["h"]
    if op == "few":
        live, e, k = n - case["idle"], case["e"], case["k"]
        hit = e * (1 - (1 - k / e) ** live)  # experts that some token chose: its expected value
        return {"bytes": hit * 6 * h * case["i"] + 4 * h * e + 2 * live * h * (2 + case["add"]), "flops": live * (6 * k * h * case["i"] + 2 * h * e)}
    if op == "norm":  # x, y, and with a residual the addend and the sum
        return {"bytes": 2 * n * h * (2 + 2 * case["add"]) + 4 * h * (1 + case["bias"]) + 4 * n * (2 - case["kind"]), "flops": 8 * n * h}
    return {"bytes": 2 * n * h * (3 + case["add"]) + 4 * h * (2 + case["bias"]) + 4 * n * (2 - case["kind"]), "flops": 14 * n * h}


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    bf16, f32 = dict(dtype=torch.bfloat16, device="cuda"), dict(dtype=torch.float32, device="cuda")

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return torch.empty(shape, dtype=dtype, device="cuda").normal_(std=std, generator=gen)

    s = dict(case)
    if case["op"] == "few":
        n, h, i, e, k = (case[q] for q in "nhiek")
        s |= {"x": normal(n, h), "rows": normal(n, h) if case["add"] else None, "y": torch.zeros((n, h), **bf16)}
        # logits of unit size, biases as a load balancer leaves them, weights that keep unit inputs near unit size
        s |= {"wr": normal(h, e, std=h ** -0.5, dtype=torch.float32), "b": normal(e, std=0.3, dtype=torch.float32) if case["bias"] else None}
        s |= {"w13": normal(e, 2 * i, h, std=h ** -0.5), "w2": normal(e, h, i, std=i ** -0.5)}
        s["live"] = torch.tensor([n - case["idle"]], dtype=torch.int32, device="cuda") if case["idle"] else None
        if own:  # the shape and scratch that a serving program keeps
            import mixture_experts_routing_gb300 as moe
            s["cfg"] = moe.FewConfig(n, h, e, k, i, renorm=case["renorm"], activation=case["act"])
            s["ws"] = moe.alloc_few_workspace(s["cfg"], "cuda")
        return s
    if case["op"] in ("norm", "norm_grad"):
        n, h = case["n"], case["h"]
        # rows of a residual stream: unlike sizes, and a mean that is not zero
        size = torch.exp(0.5 * torch.randn((n, 1), generator=gen, **f32))
        x = (torch.randn((n, h), generator=gen, **f32) * size + 0.1 * size).to(torch.bfloat16)
        s |= {"x": x, "rows": normal(n, h) if case["add"] else None, "w": 1 + normal(h, std=0.2, dtype=torch.float32)}
        s |= {"b": normal(h, std=0.2, dtype=torch.float32) if case["bias"] else None, "eps": 1e-5}
        if case["op"] == "norm":
            s |= {"y": torch.empty((n, h), **bf16), "sum": torch.empty((n, h), **bf16) if case["add"] else None}
            s |= {"mean": torch.empty(n, **f32) if case["kind"] == LAYER else None, "rstd": torch.empty(n, **f32)}
        else:
            c = x.float()
            s["mean"] = c.mean(1) if case["kind"] == LAYER else None  # what the forward kept
            c = c if s["mean"] is None else c - s["mean"].unsqueeze(1)
            s["rstd"] = (c.square().mean(1) + s["eps"]).rsqrt()
            s |= {"dy": normal(n, h), "dx": torch.empty((n, h), **bf16), "dw": torch.empty(h, **f32), "db": torch.empty(h, **f32) if case["bias"] else None}
        if own:
            import mixture_experts_routing_gb300 as moe
            s["cfg"] = moe.NormConfig(n, h, kind=case["kind"], eps=s["eps"])
            if case["op"] == "norm_grad":
                s["ws"] = moe.alloc_norm_backward_workspace(s["cfg"], "cuda")
        return s
    sizes = _sizes(case)
    at = [0]
    for n in sizes:
        at.append(at[-1] + -(-n // BLOCK) * BLOCK)
    total = at[-1]
    live = torch.zeros(total, dtype=torch.bool, device="cuda")  # not the gaps between tensors
    decay = torch.empty(total // BLOCK, **f32)
    for a, z, n in zip(at, at[1:], sizes):
        live[a: a + n] = True
        decay[a // BLOCK: z // BLOCK] = 0.1 if n > 10_000 else 0.0  # biases and norms do not decay
    # gradients of unlike sizes from block to block, states as earlier steps left them
    size = torch.exp(torch.randn((total // BLOCK, 1), generator=gen, **f32)) * 1e-3

    def scaled(factor):
        v = torch.empty((total // BLOCK, BLOCK), **f32).normal_(generator=gen)
        return v.mul_(size).mul_(factor).view(-1).mul_(live)

    master = torch.empty(total, **f32).normal_(std=0.02, generator=gen).mul_(live)
    s |= {"grad": scaled(1.0).to(torch.float32 if case["grad32"] else torch.bfloat16), "decay": decay, "seed": 1234}
    s |= {"lr": 3e-4, "beta1": 0.9, "beta2": 0.95, "eps": 1e-8, "scale": torch.tensor([0.25], **f32)}
    s |= {"master": master, "weight": None if case["wide"] else master.to(torch.bfloat16), "steps": torch.tensor([99, 0], dtype=torch.int32, device="cuda")}
    m, v = scaled(0.1), scaled(0.25).square_()
    if case["bits"] == 32:
        s |= {"m": m, "v": v}
    else:  # codes and scales that stand for them
        s["m"], s["m_scale"] = _codes(m, None)
        s["v"], s["v_scale"] = _codes(v.sqrt_(), None)
    if own:  # the optimizer that a training program keeps
        import mixture_experts_routing_gb300 as moe
        views = lambda t: [t[a: a + n] for a, n in zip(at, sizes)]  # noqa: E731
        s["opt"] = moe.AdamW(views(master if case["wide"] else s["weight"]), views(s["grad"]), lr=s["lr"], betas=(0.9, 0.95), eps=1e-8,
                             weight_decay=[0.1 if n > 10_000 else 0.0 for n in sizes], state_bits=case["bits"], seed=s["seed"])
        o = s["opt"]
        for name in ("m", "v") + (("m_scale", "v_scale") if case["bits"] == 8 else ()) + (() if case["wide"] else ("master",)):
            getattr(o, name).copy_(s[name])
            s[name] = getattr(o, name)
        o.steps.copy_(s["steps"])
        s["steps"] = o.steps
    return s


# ------------------------------------------------------------------ plain form (32 bits)
def _act(g, act):
    return g * torch.sigmoid(g) if act == SWIGLU else 0.5 * g * (1 + torch.erf(g * math.sqrt(0.5)))


def _plain_few(s):
    live, i, k = s["n"] - s["idle"], s["i"], s["k"]
    logits = s["x"][:live].double() @ s["wr"].double()  # in 64 bits: which logit is larger decides
    if s["b"] is not None:
        logits = logits + s["b"].double()
    p, ids = torch.sort(torch.softmax(logits, 1), dim=1, descending=True, stable=True)
    p, ids = p[:, :k], ids[:, :k]
    p = (p / p.sum(1, keepdim=True) if s["renorm"] else p).float()
    at = ids.flatten()
    x = s["x"][:live].float().repeat_interleave(k, 0).unsqueeze(2)
    pre = torch.bmm(s["w13"][at].float(), x).squeeze(2)
    hid = _act(pre[:, :i], s["act"]) * pre[:, i:]
    y = (torch.bmm(s["w2"][at].float(), hid.unsqueeze(2)).view(live, k, -1) * p.unsqueeze(2)).sum(1)
    s["y"][:live] = (y if s["rows"] is None else y + s["rows"][:live].float()).to(torch.bfloat16)
    return {"y": s["y"]}


def _plain_norm(s):
    x = s["x"]
    out = {}
    if s["rows"] is not None:
        x = out["sum"] = (x.float() + s["rows"].float()).to(torch.bfloat16)
    c = x.float()
    if s["kind"] == LAYER:
        out["mean"] = c.mean(1)
        c = c - out["mean"].unsqueeze(1)
    out["rstd"] = 1 / torch.sqrt(c.square().mean(1) + s["eps"])
    y = c * out["rstd"].unsqueeze(1) * s["w"]
    out["y"] = (y if s["b"] is None else y + s["b"]).to(torch.bfloat16)
    return out


def _plain_norm_grad(s):
    x, dy, r = s["x"].float(), s["dy"].float(), s["rstd"].unsqueeze(1)
    z = (x if s["kind"] == RMS else x - s["mean"].unsqueeze(1)) * r
    g = dy * s["w"]
    d = g - z * (g * z).mean(1, keepdim=True)
    if s["kind"] == LAYER:
        d = d - g.mean(1, keepdim=True)
    dx = d * r if s["rows"] is None else d * r + s["rows"].float()
    out = {"dx": dx.to(torch.bfloat16), "dw": (dy * z).sum(0)}
    if s["b"] is not None:
        out["db"] = dy.sum(0)
    return out


def _dither(count, seed, step, device):
    """32 even bits for each index below count, of this seed and step: xor-shifts and odd multiplications mod 2^32."""
    low = 0xFFFFFFFF

    def mix(v):
        v = ((v ^ (v >> 16)) * 0x7FEB352D) & low
        v = ((v ^ (v >> 15)) * 0x846CA68B) & low
        return v ^ (v >> 16)

    key = mix((step * 0x9E3779B1 + seed) & low)
    index = torch.arange(count, dtype=torch.int64, device=device)
    return mix((index * 0x9E3779B1 + (index >> 32) * 0x85EBCA77 + key) & low)


def _codes(v, dither):
    """E4M3 codes of blocks of v, scaled so that the largest is 448, and the scales. dither: 16 bits a value decide which of the two nearest codes; None: the nearest."""
    b = v.view(-1, BLOCK)
    top = b.abs().amax(1, keepdim=True)
    some = top >= 2.0 ** -100
    inv = torch.where(some, 448 / top, torch.zeros_like(top))
    # as a float whose exponent field is the code's, the code is the upper bits, and the lower 20 what is rounded
    bits = (b.abs() * inv * 2.0 ** -120).view(torch.int32)
    code = (bits + (2 ** 19 if dither is None else (dither.view(-1, BLOCK) * 16 + 8).to(torch.int32))) >> 20
    code = code.clamp(max=126) + 128 * (b < 0)
    return code.to(torch.uint8).view(-1), torch.where(some, top / 448, torch.zeros_like(top)).view(-1)


def _values(codes, scale):
    return (codes.view(torch.float8_e4m3fn).float().view(-1, BLOCK) * scale.unsqueeze(1)).view(-1)


def _plain_adamw(s):
    s["steps"][0] += 1
    t = s["steps"][0]
    g = s["grad"].float() * s["scale"]
    b1, b2 = s["beta1"], s["beta2"]
    small = s["bits"] == 8
    m, v = (_values(s["m"], s["m_scale"]), _values(s["v"], s["v_scale"]).square()) if small else (s["m"], s["v"])
    m = m * b1 + g * (1 - b1)
    v = v * b2 + g * g * (1 - b2)
    c1, c2 = (1 - b1 ** t.double()).float(), (1 - b2 ** t.double()).float()
    step = (m / c1) / (torch.sqrt(v / c2) + s["eps"])
    p = s["master"].view(-1, BLOCK)
    p.copy_(p - s["lr"] * (step.view(-1, BLOCK) + s["decay"].unsqueeze(1) * p))
    if s["weight"] is not None:
        s["weight"].copy_(s["master"])
    if small:
        d = _dither(m.numel(), s["seed"], t.long(), m.device)
        for name, value, bits in (("m", m, d & 0xFFFF), ("v", torch.sqrt(v), d >> 16)):
            codes, scale = _codes(value, bits)
            s[name].copy_(codes)
            s[name + "_scale"].copy_(scale)
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)
    return _updated(s)


def _updated(s):
    """What a step leaves: weights, states (8-bit ones as the numbers that they are, next to their scales) and the count of steps."""
    names = ["master", "weight", "m", "v"] + (["m_scale", "v_scale"] if s["bits"] == 8 else [])
    out = {n: s[n].view(torch.float8_e4m3fn) if s[n].dtype is torch.uint8 else s[n] for n in names if s[n] is not None}
    return out | {"steps": s["steps"]}


def run(state):
    s = state
    if own:
        import mixture_experts_routing_gb300 as moe
        if s["op"] == "few":
            moe.few_forward(s["cfg"], s["x"], s["wr"], s["b"], s["w13"], s["w2"], s["y"], s["ws"], add=s["rows"], n_valid=s["live"])
            return {"y": s["y"]}
        if s["op"] == "norm":
            moe.norm_forward(s["cfg"], s["x"], s["w"], s["y"], bias=s["b"], add=s["rows"], sum=s["sum"], mean=s["mean"], rstd=s["rstd"])
            return {n: s[n] for n in ("y", "sum", "mean", "rstd") if s[n] is not None}
        if s["op"] == "norm_grad":
            moe.norm_backward(s["cfg"], s["x"], s["w"], s["mean"], s["rstd"], s["dy"], s["dx"], s["dw"], s["ws"], dbias=s["db"], dx_add=s["rows"])
            return {n: s[n] for n in ("dx", "dw", "db") if s[n] is not None}
        s["opt"].step(grad_scale=s["scale"])
        return _updated(s)
    return {"few": _plain_few, "norm": _plain_norm, "norm_grad": _plain_norm_grad, "adamw": _plain_adamw}[s["op"]](s)


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_few(s):
    live, i = s["n"] - s["idle"], s["i"]
    x = s["x"][:live].double()
    logits = torch.einsum("nh,he->ne", x, s["wr"].double())
    if s["b"] is not None:
        logits += s["b"].double()
    w = torch.exp(logits - logits.max(1, keepdim=True).values)
    w /= w.sum(1, keepdim=True)
    left, chosen = w.clone(), torch.zeros_like(w)
    for _ in range(s["k"]):  # the largest that is left, the lower expert of equal ones
        at = (left == left.max(1, keepdim=True).values).double().argmax(1, keepdim=True)
        chosen.scatter_(1, at, w.gather(1, at))
        left.scatter_(1, at, -1.0)
    if s["renorm"]:
        chosen /= chosen.sum(1, keepdim=True)
    y = torch.zeros_like(s["y"], dtype=torch.float64)
    if s["rows"] is not None:
        y[:live] = s["rows"][:live].double()
    for e in (chosen > 0).any(0).nonzero().flatten().tolist():
        t = (chosen[:, e] > 0).nonzero().flatten()
        g, u = x[t] @ s["w13"][e, :i].double().t(), x[t] @ s["w13"][e, i:].double().t()
        a = g / (1 + torch.exp(-g)) if s["act"] == SWIGLU else g * torch.special.ndtr(g)
        y[t] += chosen[t, e].unsqueeze(1) * ((a * u) @ s["w2"][e].double().t())
    return {"y": y}


def _bf16_64(v):
    """The nearest bf16 value, ties to even."""
    f, e = torch.frexp(v)
    return torch.ldexp(torch.round(f * 256), e - 8)


def _exact_norm(s):
    c = s["x"].double()
    out = {}
    if s["rows"] is not None:
        c = out["sum"] = _bf16_64(c + s["rows"].double())
    if s["kind"] == LAYER:
        out["mean"] = c.sum(1) / s["h"]
        c = c - out["mean"][:, None]
    out["rstd"] = ((c * c).sum(1) / s["h"] + s["eps"]) ** -0.5
    out["y"] = c * out["rstd"][:, None] * s["w"].double() + (0 if s["b"] is None else s["b"].double())
    return out


def _exact_norm_grad(s):
    x, dy, r = s["x"].double(), s["dy"].double(), s["rstd"].double()[:, None]
    z = (x - (0 if s["mean"] is None else s["mean"].double()[:, None])) * r
    g = dy * s["w"].double()
    d = g - z * ((g * z).sum(1, keepdim=True) / s["h"])
    if s["kind"] == LAYER:
        d -= g.sum(1, keepdim=True) / s["h"]
    out = {"dx": d * r + (0 if s["rows"] is None else s["rows"].double()), "dw": torch.einsum("nh,nh->h", dy, z)}
    return out if s["b"] is None else out | {"db": dy.sum(0)}


def _noise64(count, seed, step, device):
    """The dither from products of 16-bit halves."""
    def times(v, c):
        return ((v & 65535) * c + (((v >> 16) * (c & 65535)) % 65536 << 16)) % 2 ** 32

    def mix(v):
        v = times(v ^ (v >> 16), 0x7FEB352D)
        v = times(v ^ (v >> 15), 0x846CA68B)
        return v ^ (v >> 16)

    key = int(mix(torch.tensor((step * 0x9E3779B1 + seed) % 2 ** 32)))
    return mix((times(torch.arange(count, device=device), 0x9E3779B1) + key) % 2 ** 32)  # fewer than 2^32 values


def _e4m3_64(v, noise):
    """Blocks of v on the grid of E4M3 times a scale that brings the largest to 448; a value between two steps goes up where its part of a step plus the noise reaches 1."""
    b = v.view(-1, BLOCK)
    scale = b.abs().amax(1, keepdim=True) / 448
    a = torch.where(scale > 0, b.abs() / scale.clamp(min=1e-300), 0.0)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -40))).clamp(min=-6) - 3)
    a = torch.floor(a / step + (noise.view(-1, BLOCK).double() + 0.5) / 65536) * step
    return (torch.sign(b) * a.clamp(max=448)).view(-1), scale.view(-1)


def _exact_adamw(s):
    t = int(s["steps"][0]) + 1
    g = s["grad"].double() * s["scale"].double()
    old = {}
    for n in ("m", "v"):
        old[n] = s[n].double() if s["bits"] == 32 else s[n].view(torch.float8_e4m3fn).double() * s[n + "_scale"].double().repeat_interleave(BLOCK)
    m = s["beta1"] * old["m"] + (1 - s["beta1"]) * g
    v = s["beta2"] * (old["v"] if s["bits"] == 32 else old["v"] ** 2) + (1 - s["beta2"]) * g ** 2
    del g, old
    u = m / (1 - s["beta1"] ** t) / ((v / (1 - s["beta2"] ** t)) ** 0.5 + s["eps"])
    p = s["master"].double()
    p = p * (1 - s["lr"] * s["decay"].double().repeat_interleave(BLOCK)) - s["lr"] * u
    del u
    out = {"master": p, "m": m, "v": v}
    if s["weight"] is not None:
        out["weight"] = p
    if s["bits"] == 8:
        noise = _noise64(m.numel(), s["seed"], t, m.device)
        out["m"], out["m_scale"] = _e4m3_64(m, noise % 65536)
        out["v"], out["v_scale"] = _e4m3_64(v ** 0.5, noise // 65536)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"few": _exact_few, "norm": _exact_norm, "norm_grad": _exact_norm_grad, "adamw": _exact_adamw}[s["op"]](s)
