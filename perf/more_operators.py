"""Further operators of a training step and their measured cases.

A pointwise (1 x 1) layer between deformable layers as matrix products of 8-bit
floating-point codes with a power-of-two scale for each block of 128 (forward,
and backward for input and weight), and the steps of an optimiser for matrices:
orthogonalising them by Newton-Schulz products, and the whole Muon step over
many weights.

``run`` computes them in their plain form (elementary torch operations in
float32) or, where ``own`` is true, by the framework's entry points.
"""
import math
import random

import torch

own = False

BLOCK = 128                               # values that share a scale
NS = (3.4445, -4.7750, 2.0315)            # the Newton-Schulz polynomial a x + b x^3 + c x^5
STEPS, EPS = 5, 1e-7
LR, MOMENTUM, DECAY, RMS = 1e-3, 0.95, 0.01, 0.2

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
# code type, exponent of its largest value 1.75 * 2^top, mantissa bits, lowest exponent of a normal code
FORMATS = {"e4m3": (torch.float8_e4m3fn, 8, 3, -6), "e5m2": (torch.float8_e5m2, 15, 2, -14)}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one small image: the calls' latency counts
        dict(name="pointwise fwd tiny", op="fwd", n=1, ci=64, co=64, h=32, w=32, dtype="bf16", layout="nchw"),
        # between two layers of the training stack, in the layout that the layer takes
        dict(name="pointwise fwd stack", op="fwd", n=8, ci=256, co=256, h=56, w=56, dtype="bf16", layout="nchw"),
        # a detector's resolution at a large batch, channels last: bound by memory
        dict(name="pointwise fwd detector", op="fwd", n=16, ci=256, co=256, h=100, w=168, dtype="bf16", layout="nhwc"),
        # the widest layers of a residual network at detector resolution: bound by the products
        dict(name="pointwise fwd wide", op="fwd", n=8, ci=2048, co=2048, h=50, w=84, dtype="bf16", layout="nhwc"),
        # the stack's backward: the deformable layer above hands down a float32 gradient
        dict(name="pointwise bwd stack", op="bwd", n=8, ci=256, co=256, h=56, w=56, dtype="bf16", layout="nchw", grad="f32", fmt="e4m3"),
        # a bottleneck's widening layer, channels last, gradients in the wide-range code
        dict(name="pointwise bwd widening", op="bwd", n=4, ci=512, co=2048, h=50, w=84, dtype="bf16", layout="nhwc", grad="bf16", fmt="e5m2"),
        # channels and pixels that fill no block of 128, float32
        dict(name="pointwise bwd odd", op="bwd", n=3, ci=200, co=328, h=29, w=43, dtype="f32", layout="nchw", grad="f32", fmt="e4m3"),
        # the stack's offset weights alone: short rows, where latency counts
        dict(name="orthogonalise offsets", op="ortho", count=1, mix=-2, dtype="bf16", out="bf16", precision=16),
        # the stack's main and offset weights, to float32
        dict(name="orthogonalise stack", op="ortho", count=8, mix=-1, dtype="f32", out="f32", precision=32),
        # four of a residual network's widest weights: bound by the products
        dict(name="orthogonalise wide", op="ortho", count=4, mix=-3, dtype="bf16", out="bf16", precision=16),
        # an optimiser step over the stack's weights: bf16 with float32 masters
        dict(name="muon stack", op="muon", count=8, mix=-1, param="master", grad="f32", precision=32),
        # a whole network's weights of every shape, bf16
        dict(name="muon network", op="muon", count=24, mix=7, param="bf16", grad="bf16", precision=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "bwd", "ortho", "ortho", "muon", "muon"])
    if op in ("fwd", "bwd"):
        while True:
            case = dict(op=op, n=_log(rng, 1, 16), ci=_log(rng, 8, 2048), co=_log(rng, 8, 2048), h=_log(rng, 4, 128),
                        w=_log(rng, 4, 128), dtype=rng.choice(["bf16", "bf16", "f32"]), layout=rng.choice(["nchw", "nhwc"]))
            if rng.random() < 0.5:  # whole vectors, as most networks have
                case["ci"], case["co"] = -(-case["ci"] // 16) * 16, -(-case["co"] // 16) * 16
            values = case["n"] * case["h"] * case["w"] * (case["ci"] + case["co"])
            if 16384 <= values <= 100_000_000 and work(dict(case, grad="f32"))["flops"] <= 2.5e11:
                break
        if op == "bwd":
            case.update(grad=rng.choice([case["dtype"], "f32"]), fmt=rng.choice(["e4m3", "e5m2"]))
        return case
    while True:
        case = dict(op=op, count=_log(rng, 1, 40), mix=rng.randrange(1 << 30))
        if sum(m * n for m, n in _shapes(case)) <= 16_000_000:
            break
    if op == "ortho":
        kind = rng.choice(["bf16", "f32"])
        return dict(case, dtype=rng.choice(["bf16", "f32"]), out=kind, precision=16 if kind == "bf16" else 32)
    param = rng.choice(["f32", "master", "bf16"])
    return dict(case, param=param, grad=rng.choice(["bf16", "f32"]), precision=16 if param == "bf16" else 32)


def _shapes(case):
    """Rows and columns of each matrix: the stack's main and offset weights
    (mix -1), its offset weights (-2), square ones (-3), else of every shape."""
    if case["mix"] == -1:
        return [(256, 2304), (18, 2304)] * (case["count"] // 2)
    if case["mix"] < 0:
        return [(18, 2304) if case["mix"] == -2 else (2048, 2048)] * case["count"]
    r, got = random.Random(case["mix"]), []
    for _ in range(case["count"]):
        m, n = (_log(r, 4, 2048) for _ in range(2))
        if r.random() < 0.7:
            m, n = -(-m // 32) * 32, -(-n // 32) * 32
        got.append((m, n))
    return got


def _views(case, flat):
    got, at = [], 0
    for m, n in _shapes(case):
        got.append(flat[at:at + m * n].view(m, n))
        at += -(-m * n // 64) * 64
    return got


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    if case["op"] in ("fwd", "bwd"):
        n, ci, co, h, w = (case[k] for k in ("n", "ci", "co", "h", "w"))
        dt, last = DTYPES[case["dtype"]], case["layout"] == "nhwc"

        def maps(c):
            return (n, h, w, c) if last else (n, c, h, w)
        # an activation's output: each channel with a spread of its own, most values small or below zero
        spread = (0.5 + randn(ci).abs()).view((ci,) if last else (ci, 1, 1))
        x = randn(*maps(ci)) * spread
        x = (x / (1.0 + torch.exp(-x))).to(dt)
        s = dict(case=case, x=x, w=(randn(co, ci) * (2.0 / ci) ** 0.5).to(dt), y=torch.empty(maps(co), dtype=dt, device="cuda"))
        if case["op"] == "bwd":
            # a loss's gradient: small, and each image with a size of its own
            size = torch.exp(randn(n)).view(n, 1, 1, 1) * 1e-4
            s["gy"] = (randn(*maps(co)) * size).to(DTYPES[case["grad"]])
            s.update(gx=torch.empty_like(x), gw=torch.empty(co, ci, device="cuda"))
        if own:
            from deformable_convolution_gb300 import binding as B, fp8
            code = {"f32": B.DC_F32, "bf16": B.DC_BF16}
            s["layer"] = fp8.Pointwise(n, ci, co, h, w, dtype=code[case["dtype"]], layout=B.DC_NHWC if last else B.DC_NCHW,
                                       training=case["op"] == "bwd", grad_dtype=code[case.get("grad", case["dtype"])],
                                       grad_format={"e4m3": B.DC_E4M3, "e5m2": B.DC_E5M2}[case.get("fmt", "e4m3")])
            s["layer"].load(s["w"])
            if case["op"] == "bwd":  # the forward before it keeps x's codes
                s["layer"].forward(x, s["y"])
        else:
            # the weight's codes, made once, and for the backward x's
            s["wq"] = _square(s["w"])
            if case["op"] == "bwd":
                s["xq"] = _runs(_rows(case, x).transpose(1, 2) if last else _rows(case, x), "e4m3")
        return s

    shapes = _shapes(case)
    total = sum(-(-m * n // 64) * 64 for m, n in shapes)

    def gradients():
        """A few directions that the whole batch shares, and noise."""
        flat = torch.zeros(total, device="cuda")
        for v in _views(case, flat):
            m, n = v.shape
            r = min(m, n, 12)
            fall = torch.exp(-0.3 * torch.arange(r, device="cuda"))
            v.copy_(((randn(m, r) * fall) @ randn(r, n) * 3.0 + randn(m, n)) * 1e-3)
        return flat

    s = dict(case=case)
    if case["op"] == "ortho":
        s["x"] = gradients().to(DTYPES[case["dtype"]])
        s["y"] = torch.zeros(total, dtype=DTYPES[case["out"]], device="cuda")
        if own:
            from deformable_convolution_gb300 import optim
            s["call"] = optim.Orthogonalize(_views(case, s["x"]), _views(case, s["y"]), precision=case["precision"])
        return s
    s["grad"] = gradients().to(DTYPES[case["grad"]])
    s["m"] = gradients()
    kept = torch.zeros(total, device="cuda")
    for v in _views(case, kept):
        v.copy_(randn(*v.shape) * 0.02)
    s["param"] = kept if case["param"] == "f32" else kept.to(torch.bfloat16)
    if case["param"] == "master":
        s["master"] = kept
    s["scale"] = torch.full((1,), 0.75, device="cuda")
    if own:
        from deformable_convolution_gb300 import optim
        parts = {k: _views(case, s[k]) for k in ("param", "grad", "m", "master") if k in s}
        params = [{k: v[i] for k, v in parts.items()} for i in range(len(shapes))]
        s["opt"] = optim.Muon(params, lr=LR, momentum=MOMENTUM, weight_decay=DECAY, precision=case["precision"])
    return s


# ---------------------------------------------------------------- plain forms

def _power(e):
    """2^e of whole numbers e in [-126, 127], exactly."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _coded(t, top, fmt):
    """The values that t's codes stand for: top, of t's shape or spread over it,
    is the largest magnitude of each value's block; its scale is the smallest
    power of two that brings it into the codes' range."""
    code, high = FORMATS[fmt][:2]
    part, e = torch.frexp(top)                  # top = part * 2^e, part in [0.5, 1)
    e = (e - (high + 1) + (part > 0.875)).clamp(min=-126)
    return (t * _power(-e)).to(code).float() * _power(e)


def _runs(t, fmt):
    """t [batch, rows, columns] with a scale for each run of 128 columns."""
    t = t.float()
    b, r, c = t.shape
    k = -(-c // BLOCK)
    p = torch.zeros(b, r, k * BLOCK, device=t.device)
    p[..., :c] = t
    p = p.view(b, r, k, BLOCK)
    return _coded(p, p.abs().amax(3, keepdim=True), fmt).view(b, r, -1)[..., :c]


def _square(w):
    """A weight with a scale for each 128 x 128 block."""
    w = w.float()
    r, c = w.shape
    i, k = -(-r // BLOCK), -(-c // BLOCK)
    p = torch.zeros(i * BLOCK, k * BLOCK, device=w.device)
    p[:r, :c] = w
    p = p.view(i, BLOCK, k, BLOCK)
    return _coded(p, p.abs().amax((1, 3), keepdim=True), "e4m3").view(i * BLOCK, -1)[:r, :c]


def _rows(case, t):
    """Channels last: [1, pixels of all images, channels]; else [images, channels, pixels]."""
    return t.reshape(1, -1, t.shape[3]) if case["layout"] == "nhwc" else t.flatten(2)


def _plain_fwd(s):
    case, x = s["case"], _rows(s["case"], s["x"])
    if case["layout"] == "nhwc":
        y = _runs(x, "e4m3")[0] @ s["wq"].t()
    else:
        y = s["wq"] @ _runs(x.transpose(1, 2), "e4m3").transpose(1, 2)
    return dict(y=y.to(s["y"].dtype).view(s["y"].shape))


def _plain_bwd(s):
    case, gy = s["case"], _rows(s["case"], s["gy"])
    if case["layout"] == "nhwc":
        gx = _runs(gy, case["fmt"])[0] @ s["wq"]
        gy = gy.transpose(1, 2)
    else:
        gx = s["wq"].t() @ _runs(gy.transpose(1, 2), case["fmt"]).transpose(1, 2)
    gw = (_runs(gy, case["fmt"]) @ s["xq"].transpose(1, 2)).sum(0)
    return dict(gx=gx.to(s["gx"].dtype).view(s["gx"].shape), gw=gw)


def _plain_orthogonal(g):
    a, b, c = NS
    x = g.float()
    x = x / (torch.sqrt((x * x).sum()) + EPS)
    tall = x.shape[0] > x.shape[1]
    x = x.t() if tall else x
    for _ in range(STEPS):
        p = x @ x.t()
        x = a * x + (b * p + c * (p @ p)) @ x
    return x.t() if tall else x


def _plain_ortho(s):
    for x, y in zip(_views(s["case"], s["x"]), _views(s["case"], s["y"])):
        y.copy_(_plain_orthogonal(x))
    return dict(y=s["y"])


def _plain_muon(s):
    case = s["case"]
    g = s["grad"].float() * s["scale"]
    s["m"].copy_(s["m"] * MOMENTUM + g * (1.0 - MOMENTUM))
    u = g * (1.0 - MOMENTUM) + s["m"] * MOMENTUM
    kept = s["master"] if case["param"] == "master" else s["param"]
    for p, v in zip(_views(case, kept), _views(case, u)):
        rate = LR * RMS * math.sqrt(max(v.shape))
        p.copy_(p.float() * (1.0 - LR * DECAY) - _plain_orthogonal(v) * rate)
    if case["param"] == "master":
        s["param"].copy_(kept)
    return _muon_outputs(s)


def _muon_outputs(s):
    return {k: s[k] for k in ("param", "m", "master") if k in s}


def run(state):
    op = state["case"]["op"]
    if not own:
        return {"fwd": _plain_fwd, "bwd": _plain_bwd, "ortho": _plain_ortho, "muon": _plain_muon}[op](state)
    s = state
    if op == "fwd":
        s["layer"].forward(s["x"], s["y"])
        return dict(y=s["y"])
    if op == "bwd":
        s["layer"].backward(s["gy"], s["gx"], s["gw"])
        return dict(gx=s["gx"], gw=s["gw"])
    if op == "ortho":
        s["call"]()
        return dict(y=s["y"])
    s["opt"].step(grad_scale=s["scale"])
    return _muon_outputs(s)


def work(case):
    if case["op"] in ("fwd", "bwd"):
        pixels = case["n"] * case["h"] * case["w"]
        size = 2 if case["dtype"] == "bf16" else 4
        product = 2 * pixels * case["ci"] * case["co"]
        weight = case["ci"] * case["co"]
        if case["op"] == "fwd":
            return {"bytes": size * pixels * (case["ci"] + case["co"]) + weight, "flops": product}
        grad = 2 if case["grad"] == "bf16" else 4
        return {"bytes": pixels * (grad * case["co"] + (1 + size) * case["ci"]) + 5 * weight, "flops": 2 * product}
    shapes = _shapes(case)
    values = sum(m * n for m, n in shapes)
    # a step's products: a symmetric one over the long side, its square, and the one with the matrix
    flops = sum(STEPS * (3 * min(s) ** 2 * max(s) + min(s) ** 3) for s in shapes)
    size = {"f32": 4, "bf16": 2}
    if case["op"] == "ortho":
        return {"bytes": values * (size[case["dtype"]] + size[case["out"]]), "flops": flops}
    param = {"f32": 8, "master": 10, "bf16": 4}[case["param"]]
    return {"bytes": values * (param + 8 + size[case["grad"]]), "flops": flops}


# ---------------------------------------------------------------- in 64 bits

def _exact_coded(t, dims, fmt):
    """t with its blocks along `dims` as the values its codes stand for."""
    _, high, mantissa, low = FORMATS[fmt]
    top = t.abs().amax(dims, keepdim=True)
    e = torch.ceil(torch.log2(top.clamp_min(2.0 ** -140) / (1.75 * 2.0 ** high)) - 1e-13).clamp_min(-126.0)
    v = t / torch.exp2(e)
    quantum = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -200))).clamp_min(low) - mantissa)
    return torch.round(v / quantum) * quantum * torch.exp2(e)


def _exact_runs(t, fmt):
    """Runs of 128 along the last dimension."""
    t = t.double()
    pad = -t.shape[-1] % BLOCK
    v = torch.nn.functional.pad(t, (0, pad)).unflatten(-1, (-1, BLOCK))
    return _exact_coded(v, -1, fmt).flatten(-2)[..., :t.shape[-1]]


def _exact_weight(w):
    r, c = w.shape
    v = torch.nn.functional.pad(w.double(), (0, -c % BLOCK, 0, -r % BLOCK))
    v = v.unflatten(1, (-1, BLOCK)).unflatten(0, (-1, BLOCK))
    return _exact_coded(v, (1, 3), "e4m3").flatten(2).flatten(0, 1)[:r, :c]


def _exact_pointwise(case, s):
    last, w = case["layout"] == "nhwc", _exact_weight(s["w"])
    # channels along the last dimension, [images, pixels, channels], and pixels: all of them in one row, or each image's
    by_channel = (lambda t: t.flatten(1, 2)) if last else (lambda t: t.flatten(2).mT)  # noqa: E731
    by_pixel = (lambda t: t.flatten(0, 2).t()[None]) if last else (lambda t: t.flatten(2))  # noqa: E731

    def back(t, like):
        return (t if last else t.mT).reshape(like.shape)
    if case["op"] == "fwd":
        return dict(y=back(torch.einsum("bpi,oi->bpo", _exact_runs(by_channel(s["x"]), "e4m3"), w), s["y"]))
    gx = torch.einsum("bpo,oi->bpi", _exact_runs(by_channel(s["gy"]), case["fmt"]), w)
    gw = torch.einsum("bop,bip->oi", _exact_runs(by_pixel(s["gy"]), case["fmt"]), _exact_runs(by_pixel(s["x"]), "e4m3"))
    return dict(gx=back(gx, s["gx"]), gw=gw)


def _exact_orthogonal(g):
    a, b, c = NS
    x = g.double()
    x = x / (torch.linalg.matrix_norm(x) + EPS)
    for _ in range(STEPS):
        if x.shape[0] <= x.shape[1]:
            p = x.mm(x.mT)
            x = torch.addmm(x, torch.addmm(p, p, p, beta=b, alpha=c), x, beta=a)
        else:
            p = x.mT.mm(x)
            x = torch.addmm(x, x, torch.addmm(p, p, p, beta=b, alpha=c), beta=a)
    return x


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("fwd", "bwd"):
        return _exact_pointwise(case, s)
    if case["op"] == "ortho":
        y = torch.zeros_like(s["y"], dtype=torch.float64)
        for u, v in zip(_views(case, s["x"]), _views(case, y)):
            v.copy_(_exact_orthogonal(u))
        return dict(y=y)
    g = s["grad"].double() * s["scale"].double()
    m = torch.lerp(g, s["m"].double(), MOMENTUM)
    u = torch.lerp(g, m, MOMENTUM)
    p = (s["master"] if case["param"] == "master" else s["param"]).double()
    for q, v in zip(_views(case, p), _views(case, u)):
        q.mul_(1 - LR * DECAY).sub_(_exact_orthogonal(v), alpha=LR * RMS * max(v.shape) ** 0.5)
    out = dict(param=p, m=m)
    if case["param"] == "master":
        out["master"] = p
    return out
