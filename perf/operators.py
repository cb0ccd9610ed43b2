"""The training-step operators and their measured cases.

Three operators that finish a training step around the deformable layers:
group norm with an activation (forward and backward, channels first and
channels last), AdamW over many tensors at once (states in 32 or in 8 bits),
and the global gradient norm with its clip factor.

``run`` computes them in their plain form (elementary torch operations in
float32) or, where ``own`` is true, by the framework's entry points.
"""
import math
import random

import torch

own = False

BLOCK = 256          # elements of an 8-bit state that share a scale
EPS = 1e-5           # group norm
LR, BETA1, BETA2, ADAM_EPS, DECAY = 1e-3, 0.9, 0.999, 1e-8, 0.01
CLIP_EPS = 1e-6
TINY = 2.0 ** -126   # a block's scale below this counts as zero

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # the 1 x 16 x 32 x 32 float32 layer: one image, where the call's latency counts
        dict(name="norm fwd tiny", op="fwd", n=1, c=16, h=32, w=32, groups=4, dtype="f32", layout="nchw", act="relu"),
        # between two layers of the training stack, in the layout the layer takes
        dict(name="norm fwd stack", op="fwd", n=8, c=256, h=56, w=56, groups=32, dtype="bf16", layout="nchw", act="relu"),
        # a detector's resolution at a large batch, channels last: bound by memory
        dict(name="norm fwd detector", op="fwd", n=16, c=256, h=100, w=168, groups=32, dtype="bf16", layout="nhwc", act="silu"),
        # res4 at detector resolution, two images, channels last
        dict(name="norm bwd res4", op="bwd", n=2, c=256, h=50, w=84, groups=32, dtype="bf16", layout="nhwc", act="silu", grad="bf16"),
        # the stack's backward: the layer above hands down a float32 gradient
        dict(name="norm bwd stack", op="bwd", n=8, c=256, h=56, w=56, groups=32, dtype="bf16", layout="nchw", act="relu", grad="f32"),
        # odd rows (nothing after the first starts on a 16-byte boundary), five channels a group
        dict(name="norm bwd odd", op="bwd", n=6, c=60, h=101, w=67, groups=12, dtype="f32", layout="nchw", act="gelu", grad="f32"),
        # the stack's main and offset weights: bf16 with float32 masters, eight tensors
        dict(name="adamw stack", op="adamw", tensors=8, total=2525184, mix=-1, pack=True, param="master", grad="f32", bits=32),
        # a whole network in float32, tensors of every size packed end to end
        dict(name="adamw network", op="adamw", tensors=160, total=60000000, mix=7, pack=True, param="f32", grad="f32", bits=32),
        # the stack's weights again with the states in 8 bits
        dict(name="adamw8 stack", op="adamw", tensors=8, total=2525184, mix=-1, pack=True, param="master", grad="f32", bits=8),
        # a whole network, bf16 weights and gradients, masters, 8-bit states
        dict(name="adamw8 network", op="adamw", tensors=160, total=64000000, mix=8, pack=False, param="master", grad="bf16", bits=8),
        # clipping the stack's gradients
        dict(name="grad norm stack", op="gnorm", tensors=8, total=2525184, mix=-1, pack=True, grad="f32"),
        # clipping a whole network's
        dict(name="grad norm network", op="gnorm", tensors=160, total=60000000, mix=9, pack=True, grad="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "bwd", "adamw", "adamw", "gnorm"])
    if op in ("fwd", "bwd"):
        while True:
            groups = rng.choice([1, 2, 4, 8, 12, 16, 32, 32, 32])
            c = groups * rng.choice([1, 2, 3, 4, 5, 8, 8, 10, 16, 20])
            case = dict(op=op, n=_log(rng, 1, 32), c=c, h=_log(rng, 4, 200), w=_log(rng, 4, 200), groups=groups,
                        dtype=rng.choice(["bf16", "bf16", "f32"]), layout=rng.choice(["nchw", "nhwc"]),
                        act=rng.choice(["none", "relu", "silu", "gelu"]))
            if 4096 <= case["n"] * c * case["h"] * case["w"] <= 34_000_000:
                break
        if op == "bwd":
            case["grad"] = rng.choice([case["dtype"], "f32"])
        return case
    total = _log(rng, 20_000, 60_000_000)
    case = dict(op=op, tensors=_log(rng, 1, min(400, total // 2000)), total=total, mix=rng.randrange(1 << 30),
                pack=rng.random() < 0.5, grad=rng.choice(["f32", "bf16"]))
    if op == "adamw":
        case.update(param=rng.choice(["f32", "master", "bf16"]), bits=rng.choice([32, 8]))
    return case


def _sizes(case):
    """Elements of each tensor: the stack's own (mix -1), else a spread over a
    factor of some thousands, as biases and weights of a network have."""
    if case["mix"] == -1:
        return [41472, 589824] * (case["tensors"] // 2)
    r = random.Random(case["mix"])
    weights = [math.exp(r.uniform(0.0, 10.0)) for _ in range(case["tensors"])]
    scale = case["total"] / sum(weights)
    return [max(1, int(v * scale)) for v in weights]


def _layout(case):
    """(sizes, start of each tensor in its flat buffer, the buffer's length):
    end to end, or each on a boundary of 256 elements."""
    sizes, starts, at = _sizes(case), [], 0
    for s in sizes:
        starts.append(at)
        at += s if case["pack"] else -(-s // BLOCK) * BLOCK
    return sizes, starts, at


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    if case["op"] in ("fwd", "bwd"):
        n, c, h, w, g = case["n"], case["c"], case["h"], case["w"], case["groups"]
        dt, last = DTYPES[case["dtype"]], case["layout"] == "nhwc"
        shape = (n, h, w, c) if last else (n, c, h, w)
        per_channel = (c,) if last else (c, 1, 1)
        # a convolution's output: each channel with a mean and a spread of its own
        x = (randn(*shape) * (0.5 + randn(c).abs()).view(per_channel) + 0.5 * randn(c).view(per_channel)).to(dt)
        s = dict(case=case, x=x, gamma=1.0 + 0.1 * randn(c), beta=0.1 * randn(c), y=torch.empty_like(x),
                 mean=torch.empty(n, g, device="cuda"), rstd=torch.empty(n, g, device="cuda"))
        if case["op"] == "bwd":
            gdt = DTYPES[case["grad"]]
            s["gy"] = randn(*shape).to(gdt)
            mean, rstd = _plain_stats(case, x)[1:]
            s["mean"].copy_(mean)
            s["rstd"].copy_(rstd)
            s.update(gx=torch.empty_like(x), ggamma=torch.empty(c, device="cuda"), gbeta=torch.empty(c, device="cuda"))
        if own:
            from deformable_convolution_gb300 import binding as B
            s["p"] = B.NormProblem(n, c, h, w, g, B.DC_BF16 if case["dtype"] == "bf16" else B.DC_F32,
                                   B.DC_NHWC if last else B.DC_NCHW,
                                   {"none": B.DC_ACT_NONE, "relu": B.DC_ACT_RELU, "silu": B.DC_ACT_SILU,
                                    "gelu": B.DC_ACT_GELU}[case["act"]], EPS,
                                   B.DC_BF16 if case.get("grad", case["dtype"]) == "bf16" else B.DC_F32)
            s["ws"] = B.norm_workspace(s["p"], case["op"] == "bwd")
        return s

    sizes, starts, length = _layout(case)
    gdt = DTYPES[case["grad"]]
    s = dict(case=case)
    grad = (randn(length) * 1e-2).to(gdt)
    # the padding between tensors holds zeros and stays so
    size_t = torch.tensor(sizes, device="cuda")
    start_t = torch.tensor(starts, device="cuda")
    room = torch.diff(torch.tensor(starts + [length], device="cuda"))
    tensor_of = torch.repeat_interleave(torch.arange(len(sizes), device="cuda"), room, output_size=length)
    within = torch.arange(length, device="cuda") - start_t[tensor_of]
    inside = within < size_t[tensor_of]
    grad = torch.where(inside, grad, torch.zeros_like(grad))
    s["grad"] = grad
    if case["op"] == "gnorm":
        s.update(norm=torch.empty(1, device="cuda"), scale=torch.empty(1, device="cuda"))
        if own:
            from deformable_convolution_gb300 import optim
            s["opt"] = optim.GradNorm([grad[a:a + k] for a, k in zip(starts, sizes)])
        return s

    master = torch.where(inside, randn(length) * 0.02, torch.zeros((), device="cuda"))
    m = torch.where(inside, randn(length) * 2e-3, torch.zeros((), device="cuda"))
    v = torch.where(inside, (randn(length) * 1e-2).square() * 0.5 + 1e-6, torch.zeros((), device="cuda"))
    kind = case["param"]
    s["param"] = master.clone() if kind == "f32" else master.to(torch.bfloat16)
    if kind == "master":
        s["master"] = master
    # weights decay, tensors of under 2048 elements (biases, norms) do not
    decays = [DECAY if k >= 2048 else 0.0 for k in sizes]
    s["decay"] = torch.tensor(decays, device="cuda")[tensor_of]
    s["step"], s["scale"] = 1000, torch.full((1,), 0.75, device="cuda")
    if case["bits"] == 8:
        blocks = -(-size_t // BLOCK)
        first = torch.cumsum(blocks, 0) - blocks
        count = int(blocks.sum())
        # where each tensor starts on a block, the flat buffer's blocks are the tensors'; else the block of each element
        if all(a % BLOCK == 0 for a in starts + [length]):
            s["block"] = None
        else:
            s["block"] = first[tensor_of] + torch.where(inside, within // BLOCK, blocks[tensor_of] - 1)
        s["m8"], s["m_scale"] = _encode_m(m, s["block"], count)
        s["v8"], s["v_scale"] = _encode_v(v, s["block"], count)
        s["firsts"] = first.tolist() + [count]
        s["m"], s["v"] = torch.empty(length, device="cuda"), torch.empty(length, device="cuda")
    else:
        s["m"], s["v"] = m, v
    del tensor_of, within, inside
    if own:
        from deformable_convolution_gb300 import optim
        params = []
        for i, (a, k) in enumerate(zip(starts, sizes)):
            q = dict(param=s["param"][a:a + k], grad=grad[a:a + k], weight_decay=decays[i])
            if kind == "master":
                q["master"] = master[a:a + k]
            if case["bits"] == 8:
                f, e = s["firsts"][i], s["firsts"][i + 1]
                q.update(m=s["m8"][a:a + k], v=s["v8"][a:a + k], m_scale=s["m_scale"][f:e], v_scale=s["v_scale"][f:e])
            else:
                q.update(m=m[a:a + k], v=v[a:a + k])
            params.append(q)
        s["opt"] = optim.AdamW(params, lr=LR, betas=(BETA1, BETA2), eps=ADAM_EPS, state_bits=case["bits"], step=s["step"])
        if case["bits"] == 8:
            s["m"].zero_()
            s["v"].zero_()
            s["values"] = optim.StateValues(s["opt"], [(s["m"][a:a + k], s["v"][a:a + k]) for a, k in zip(starts, sizes)])
    return s


# ---------------------------------------------------------------- plain forms

def _grouped(case, t):
    """t in float32 as [n, pixels, groups, channels of a group]."""
    n, g = case["n"], case["groups"]
    if case["layout"] == "nhwc":
        return t.float().reshape(n, -1, g, case["c"] // g)
    return t.float().reshape(n, g, case["c"] // g, -1).permute(0, 3, 1, 2)


def _back(case, t):
    """[n, pixels, groups, channels] back to the case's layout."""
    n, c, h, w = case["n"], case["c"], case["h"], case["w"]
    if case["layout"] == "nhwc":
        return t.reshape(n, h, w, c)
    return t.permute(0, 2, 3, 1).reshape(n, c, h, w)


def _plain_stats(case, x):
    xg = _grouped(case, x)
    mean = xg.mean((1, 3))
    d = xg - mean[:, None, :, None]
    rstd = 1.0 / torch.sqrt((d * d).mean((1, 3)) + EPS)
    return d, mean, rstd


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).float()
    if act == "silu":
        sg = 1.0 / (1.0 + torch.exp(-z))
        return sg * (1.0 + z * (1.0 - sg))
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    return torch.ones_like(z)


def _plain_fwd(s):
    case, g = s["case"], s["case"]["groups"]
    d, mean, rstd = _plain_stats(case, s["x"])
    z = d * rstd[:, None, :, None] * s["gamma"].view(g, -1) + s["beta"].view(g, -1)
    return dict(y=_back(case, _act(z, case["act"])).to(s["x"].dtype), mean=mean, rstd=rstd)


def _plain_bwd(s):
    case, g = s["case"], s["case"]["groups"]
    gamma, beta = s["gamma"].view(g, -1), s["beta"].view(g, -1)
    rstd = s["rstd"][:, None, :, None]
    xh = (_grouped(case, s["x"]) - s["mean"][:, None, :, None]) * rstd
    dz = _grouped(case, s["gy"]) * _act_slope(xh * gamma + beta, case["act"])
    a, b = dz.sum(1), (dz * xh).sum(1)
    m = case["h"] * case["w"] * (case["c"] // g)
    s1 = ((a * gamma).sum(2) / m)[:, None, :, None]
    s2 = ((b * gamma).sum(2) / m)[:, None, :, None]
    gx = rstd * (gamma * dz - s1 - xh * s2)
    return dict(gx=_back(case, gx).to(s["x"].dtype), ggamma=b.sum(0).reshape(-1), gbeta=a.sum(0).reshape(-1))


def _spread(scale, block):
    """A block's number at each of its elements."""
    return scale[:, None].expand(-1, BLOCK).reshape(-1) if block is None else scale[block]


def _block_max(t, block, count):
    if block is None:
        top = t.view(count, BLOCK).amax(1)
    else:
        top = torch.zeros(count, device=t.device).scatter_reduce_(0, block, t, "amax")
    top = torch.where(top < TINY, torch.zeros_like(top), top)
    return top, _spread(torch.where(top > 0, 1.0 / top, torch.zeros_like(top)), block)


def _encode_m(m, block, count):
    top, inv = _block_max(m.abs(), block, count)
    q = torch.round(torch.sqrt(m.abs() * inv) * 127.0)
    return torch.where(m < 0, -q, q).to(torch.int8), top


def _encode_v(v, block, count):
    root = torch.sqrt(v)
    top, inv = _block_max(root, block, count)
    q = torch.round(torch.sqrt(root * inv) * 255.0)
    q = torch.where((v > 0) & (q < 1) & (inv > 0), torch.ones_like(q), q)
    return q.to(torch.uint8), top


def _decode_m(q, top, block):
    t = q.float() * (1.0 / 127.0)
    return t * t.abs() * _spread(top, block)


def _decode_v(q, top, block):
    t = q.float() * (1.0 / 255.0)
    root = t * t * _spread(top, block)
    return root * root


def _plain_adamw(s):
    case = s["case"]
    eight = case["bits"] == 8
    s["step"] += 1
    bias1, bias2 = 1.0 - BETA1 ** s["step"], 1.0 - BETA2 ** s["step"]
    g = s["grad"].float() * s["scale"]
    m = _decode_m(s["m8"], s["m_scale"], s["block"]) if eight else s["m"]
    v = _decode_v(s["v8"], s["v_scale"], s["block"]) if eight else s["v"]
    m = m * BETA1 + g * (1.0 - BETA1)
    v = v * BETA2 + g * g * (1.0 - BETA2)
    kept = s["master"] if case["param"] == "master" else s["param"]
    p = kept.float() * (1.0 - LR * s["decay"])
    p = p - (m / (torch.sqrt(v) * (1.0 / math.sqrt(bias2)) + ADAM_EPS)) * (LR / bias1)
    kept.copy_(p)
    if case["param"] == "master":
        s["param"].copy_(p)
    if eight:
        count = s["m_scale"].numel()
        m8, m_scale = _encode_m(m, s["block"], count)
        v8, v_scale = _encode_v(v, s["block"], count)
        s["m8"].copy_(m8), s["m_scale"].copy_(m_scale), s["v8"].copy_(v8), s["v_scale"].copy_(v_scale)
        s["m"].copy_(_decode_m(m8, m_scale, s["block"]))
        s["v"].copy_(_decode_v(v8, v_scale, s["block"]))
    else:
        s["m"].copy_(m), s["v"].copy_(v)
    return _adamw_outputs(s)


def _adamw_outputs(s):
    out = dict(param=s["param"], m=s["m"], v=s["v"])
    if s["case"]["param"] == "master":
        out["master"] = s["master"]
    return out


def _plain_gnorm(s):
    g = s["grad"].float()
    norm = torch.sqrt((g * g).sum())
    return dict(norm=norm.reshape(1), scale=torch.clamp(0.5 / (norm + CLIP_EPS), max=1.0).reshape(1))


def run(state):
    op = state["case"]["op"]
    if not own:
        return {"fwd": _plain_fwd, "bwd": _plain_bwd, "adamw": _plain_adamw, "gnorm": _plain_gnorm}[op](state)
    s = state
    if op == "gnorm":
        s["opt"](0.5, s["norm"], s["scale"])
        return dict(norm=s["norm"], scale=s["scale"])
    if op == "adamw":
        s["opt"].step(grad_scale=s["scale"])
        if s["case"]["bits"] == 8:  # the states as the numbers they stand for
            s["values"]()
        return _adamw_outputs(s)
    from deformable_convolution_gb300 import binding as B
    if op == "fwd":
        B.dc_group_norm_fwd(s["p"], s["x"], s["gamma"], s["beta"], s["y"], s["mean"], s["rstd"], s["ws"])
        return dict(y=s["y"], mean=s["mean"], rstd=s["rstd"])
    B.dc_group_norm_bwd(s["p"], s["x"], s["gamma"], s["beta"], s["mean"], s["rstd"], s["gy"], s["gx"], s["ggamma"],
                        s["gbeta"], s["ws"])
    return dict(gx=s["gx"], ggamma=s["ggamma"], gbeta=s["gbeta"])


def work(case):
    if case["op"] in ("fwd", "bwd"):
        elements = case["n"] * case["c"] * case["h"] * case["w"]
        size = 2 if case["dtype"] == "bf16" else 4
        small = 4 * (2 * case["c"] + 2 * case["n"] * case["groups"])
        if case["op"] == "fwd":
            return {"bytes": 2 * size * elements + small, "flops": 12 * elements}
        grad = 2 if case["grad"] == "bf16" else 4
        return {"bytes": (2 * size + grad) * elements + small + 8 * case["c"], "flops": 24 * elements}
    elements = sum(_sizes(case))
    grad = 2 if case["grad"] == "bf16" else 4
    if case["op"] == "gnorm":
        return {"bytes": grad * elements + 8, "flops": 2 * elements}
    param = {"f32": 8, "master": 10, "bf16": 4}[case["param"]]
    # 8-bit states: read and written with their scales, then written out as float32
    states = 16 if case["bits"] == 32 else 4 + 16 / BLOCK + 8
    return {"bytes": int((param + grad + states) * elements), "flops": 16 * elements}


# ---------------------------------------------------------------- in 64 bits

def _exact_norm(case, s):
    n, c, h, w, g = case["n"], case["c"], case["h"], case["w"], case["groups"]
    last = case["layout"] == "nhwc"
    to_first = (lambda t: t.double().movedim(3, 1)) if last else (lambda t: t.double())  # noqa: E731
    out_of = (lambda t: t.movedim(1, 3).contiguous()) if last else (lambda t: t)  # noqa: E731
    x = to_first(s["x"]).reshape(n, g, -1)
    gamma, beta = (s[k].double().view(1, c, 1, 1) for k in ("gamma", "beta"))
    if case["op"] == "fwd":
        var, mean = torch.var_mean(x, dim=2, correction=0)
        rstd = (var + EPS).rsqrt()
    else:
        mean, rstd = s["mean"].double(), s["rstd"].double()
    xh = ((x - mean[..., None]) * rstd[..., None]).view(n, c, h, w)
    z = (xh * gamma + beta).requires_grad_(case["op"] == "bwd")
    act = {"none": lambda t: t * 1.0, "relu": torch.relu, "silu": lambda t: t * torch.sigmoid(t),
           "gelu": lambda t: t * torch.special.ndtr(t)}[case["act"]]
    y = act(z)
    if case["op"] == "fwd":
        return dict(y=out_of(y), mean=mean, rstd=rstd)
    dz, = torch.autograd.grad(y, z, to_first(s["gy"]))
    with torch.no_grad():
        dxh = (dz * gamma).reshape(n, g, -1)
        flat = xh.reshape(n, g, -1)
        gx = rstd[..., None] * (dxh - dxh.mean(2, keepdim=True) - flat * (dxh * flat).mean(2, keepdim=True))
        return dict(gx=out_of(gx.view(n, c, h, w)), ggamma=(dz * xh).sum((0, 2, 3)), gbeta=dz.sum((0, 2, 3)))


def _exact_adamw(case, s):
    t = s["step"] + 1
    g = s["grad"].double() * s["scale"].double()
    if case["bits"] == 8:
        block = torch.arange(s["m8"].numel(), device="cuda") // BLOCK if s["block"] is None else s["block"]
        per = lambda k: s[k].double()[block]  # noqa: E731
        q = s["m8"].double()
        m = per("m_scale") * q.sign() * (q / 127).square()
        v = (per("v_scale") * (s["v8"].double() / 255).square()).square()
    else:
        m, v = s["m"].double(), s["v"].double()
    m = torch.lerp(g, m, BETA1)
    v = torch.lerp(g.square(), v, BETA2)
    m_hat, v_hat = m / (1 - BETA1 ** t), v / (1 - BETA2 ** t)
    p = (s["master"] if case["param"] == "master" else s["param"]).double()
    p = p - LR * s["decay"].double() * p - LR * m_hat / (v_hat.sqrt() + ADAM_EPS)
    if case["bits"] == 8:
        def scale_of(a):
            return torch.zeros(s["m_scale"].numel(), dtype=torch.float64, device=a.device).index_reduce_(
                0, block, a, "amax", include_self=True)[block]
        top = scale_of(m.abs())
        m = m.sign() * top * (torch.round(127 * (m.abs() / top.clamp_min(TINY)).sqrt()) / 127).square()
        root = v.sqrt()
        top = scale_of(root)
        q = torch.round(255 * (root / top.clamp_min(TINY)).sqrt())
        q = torch.where(root > 0, q.clamp_min(1), q)
        v = (top * (q / 255).square()).square()
    out = dict(param=p, m=m, v=v)
    if case["param"] == "master":
        out["master"] = p
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("fwd", "bwd"):
        return _exact_norm(case, s)
    if case["op"] == "adamw":
        return _exact_adamw(case, s)
    norm = torch.linalg.vector_norm(s["grad"].double())
    return dict(norm=norm.reshape(1), scale=torch.minimum(torch.ones_like(norm), 0.5 / (norm + CLIP_EPS)).reshape(1))
