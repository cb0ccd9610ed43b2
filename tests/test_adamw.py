"""AdamW over many tensors, its 8-bit states and the gradient norm: refusals
(CPU) and the kernels against a plain form in 64 bits (GPU)."""
import ctypes
import math

import pytest
import torch

from deformable_convolution_gb300 import binding as B
from deformable_convolution_gb300 import optim

gpu = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


def on_gpu(f):
    for m in gpu:
        f = m(f)
    return f


U = 2.0 ** -24
LR, B1, B2, EPS = 3e-3, 0.9, 0.999, 1e-8
F32, BF16 = torch.float32, torch.bfloat16


# ---------------------------------------------------------------- refusals

def entry(**kw):
    # made-up, aligned addresses
    t = B.DcAdamwTensor(0x1000, None, 0x2000, 0x3000, 0x4000, 0x5000, 0x6000, 100, B.DC_F32, B.DC_F32, B.DC_STATE_F32, 0.01)
    for k, v in kw.items():
        setattr(t, k, v)
    return (B.DcAdamwTensor * 1)(t)


def step(tensors, count=1, scale=None, schedule=None, **kw):
    h = B.DcAdamwHyper(*[kw.get(k, d) for k, d in (("lr", LR), ("beta1", B1), ("beta2", B2), ("eps", EPS), ("step", 1))])
    return B.lib().dc_adamw_step(tensors, count, ctypes.byref(h), scale, schedule, None)


@pytest.mark.parametrize("kw", [dict(lr=-1.0), dict(lr=math.nan), dict(lr=math.inf), dict(beta1=1.0), dict(beta1=-0.1),
                                dict(beta2=1.0), dict(beta2=math.nan), dict(eps=-1e-8), dict(eps=math.inf), dict(step=0),
                                dict(count=-1)])
def test_hyper_parameters_are_checked(kw):
    assert step(entry(), **kw) == B.DC_ERR_INVALID_ARG


@pytest.mark.parametrize("kw,status", [
    (dict(count=-1), B.DC_ERR_INVALID_ARG), (dict(param=None), B.DC_ERR_INVALID_ARG),
    (dict(grad=None), B.DC_ERR_INVALID_ARG), (dict(m=None), B.DC_ERR_INVALID_ARG), (dict(v=None), B.DC_ERR_INVALID_ARG),
    (dict(state=B.DC_STATE_Q8, m_scale=None), B.DC_ERR_INVALID_ARG),
    (dict(state=B.DC_STATE_Q8, v_scale=None), B.DC_ERR_INVALID_ARG),
    (dict(master=0x7000), B.DC_ERR_INVALID_ARG),  # a master of a float32 parameter
    (dict(param_dtype=2), B.DC_ERR_INVALID_ARG), (dict(grad_dtype=-1), B.DC_ERR_INVALID_ARG),
    (dict(state=2), B.DC_ERR_INVALID_ARG), (dict(weight_decay=-0.1), B.DC_ERR_INVALID_ARG),
    (dict(weight_decay=math.nan), B.DC_ERR_INVALID_ARG),
    (dict(param=0x1002), B.DC_ERR_UNSUPPORTED), (dict(grad=0x2001), B.DC_ERR_UNSUPPORTED),
    (dict(m=0x3002), B.DC_ERR_UNSUPPORTED), (dict(v=0x4001), B.DC_ERR_UNSUPPORTED),
    (dict(param_dtype=B.DC_BF16, master=0x7002), B.DC_ERR_UNSUPPORTED),
    (dict(state=B.DC_STATE_Q8, v_scale=0x6002), B.DC_ERR_UNSUPPORTED),
])
def test_tensors_are_checked(kw, status):
    assert step(entry(**kw)) == status


def test_other_arguments_are_checked():
    L, vp = B.lib(), ctypes.c_void_p
    assert step(None) == B.DC_ERR_INVALID_ARG
    assert L.dc_adamw_step(entry(), 1, None, None, None, None) == B.DC_ERR_INVALID_ARG
    assert step(entry(), scale=vp(0x8002)) == B.DC_ERR_UNSUPPORTED
    assert step(entry(), schedule=vp(0x8002)) == B.DC_ERR_UNSUPPORTED
    assert step(None, count=0) == B.DC_OK
    assert step(entry(count=0, param=None, grad=None, m=None, v=None)) == B.DC_OK
    outs = (vp * 1)(0x9002)
    assert L.dc_adamw_state_values(entry(), 1, outs, None, None) == B.DC_ERR_UNSUPPORTED
    assert L.dc_adamw_state_values(entry(m=None), 1, None, None, None) == B.DC_ERR_INVALID_ARG
    assert L.dc_adamw_state_values(None, 1, None, None, None) == B.DC_ERR_INVALID_ARG
    need = B.dc_grad_norm_workspace_size(1)

    def norm(tensors=entry(), count=1, most=1.0, out=vp(0x1000), scale=vp(0x1100), ws=vp(0x2000), nbytes=need):
        return L.dc_grad_norm(tensors, count, most, out, scale, ws, nbytes, None)
    assert norm(count=-1) == norm(tensors=None) == norm(most=0.0) == norm(most=math.nan) == B.DC_ERR_INVALID_ARG
    assert norm(entry(grad=None)) == norm(entry(count=-1)) == norm(entry(grad_dtype=5)) == B.DC_ERR_INVALID_ARG
    assert norm(ws=None) == norm(nbytes=need - 1) == B.DC_ERR_WORKSPACE
    assert norm(ws=vp(0x2008)) == norm(out=vp(0x1002)) == norm(entry(grad=0x2002)) == B.DC_ERR_UNSUPPORTED
    out = ctypes.c_size_t(0)
    assert L.dc_grad_norm_workspace_size(-1, ctypes.byref(out)) == B.DC_ERR_INVALID_ARG
    assert L.dc_grad_norm_workspace_size(1, None) == B.DC_ERR_INVALID_ARG


@on_gpu
def test_the_optimiser_checks_its_tensors():
    p, g = torch.zeros(8, 3, device="cuda"), torch.zeros(8, 3, device="cuda")
    for bad in (dict(param=p, grad=g[:4]), dict(param=p.double(), grad=g), dict(param=p.cpu(), grad=g),
                dict(param=p.t(), grad=g.t()), dict(param=p, grad=g, m=torch.zeros(8, 3, device="cuda"), v=g[:4])):
        with pytest.raises(ValueError):
            optim.AdamW([bad])
    with pytest.raises(ValueError):
        optim.AdamW([dict(param=p, grad=g)], state_bits=16)
    opt = optim.AdamW([dict(param=p, grad=g)])
    with pytest.raises(ValueError):
        opt.step(grad_scale=torch.ones(2, device="cuda"))
    with pytest.raises(ValueError):
        opt.step(schedule=torch.ones(3))
    assert opt.step_count == 0


# ---------------------------------------------------------------- plain form

def blocks_of(t):
    """[blocks, 256] with zeros behind the last element."""
    n = t.numel()
    out = torch.zeros(-(-n // 256) * 256, dtype=t.dtype)
    out[:n] = t.reshape(-1)
    return out.view(-1, 256)


def decode(q):
    """float64 (m, v) of an entry's state."""
    if q["m"].dtype != torch.int8:
        return q["m"].double().cpu(), q["v"].double().cpu()
    n = q["m"].numel()
    m, v = blocks_of(q["m"].cpu()).double() / 127, blocks_of(q["v"].cpu()).double() / 255
    m = q["m_scale"].double().cpu()[:, None] * m * m.abs()
    v = (q["v_scale"].double().cpu()[:, None] * v * v) ** 2
    return m.view(-1)[:n], v.view(-1)[:n]


def plain_step(q, m, v, t, scale, wd):
    """float64 p, m, v after step t, and bounds on float32's error in them."""
    g = q["grad"].double().cpu() * scale
    kept = q["master"] if q.get("master") is not None else q["param"]
    p = kept.double().cpu()
    # a decoded state: q / top is off by 2 U (the reciprocal, the product), its
    # square by 5, times the scale by 6: m; squared once more by 13: v.  Then
    # a product by a constant (rounded too) and a sum: 3 more, and for g^2 one.
    # Below the normal numbers each rounding is 2^-150 instead
    d_m = 9 * U * (B1 * m.abs() + (1 - B1) * g.abs()) + 8 * 2.0 ** -150
    d_v = 16 * U * (B2 * v + (1 - B2) * g * g) + 8 * 2.0 ** -150
    m = B1 * m + (1 - B1) * g
    v = B2 * v + (1 - B2) * g * g
    c1, c2 = 1 - B1 ** t, 1 - B2 ** t
    denom = torch.sqrt(v / c2) + EPS
    u = LR / c1 * m / denom
    d_u = u.abs() * (8 * U + torch.minimum(d_v / (2 * v).clamp_min(1e-300), torch.sqrt(d_v / c2) / denom)) + LR / c1 * (d_m + m.abs() * 6 * U) / denom
    d_p = 4 * U * p.abs() + d_u + U * u.abs() + 8 * 2.0 ** -150
    p = p * (1 - LR * wd) - u
    return p, m, v, d_p, d_m, d_v


def near(got, want, bound, what):
    err = (got.double().cpu() - want).abs()
    bad = ~(err <= bound + 1e-44)
    assert not bad.any(), f"{what}: {int(bad.sum())} beyond the bound, worst {float((err / (bound + 1e-44)).max()):.3g} of it"


def check_codes(q, m, v, d_m, d_v):
    """The codes are the nearest: their value, in steps of the code, within half
    a step of the exact one (and 2^-12 for float32's rounding of up to 255)."""
    n = m.numel()
    for x, d, code, scale, top, low in ((m, d_m, q["m"], q["m_scale"], 127, 0), (v.sqrt(), None, q["v"], q["v_scale"], 255, 1)):
        xb = blocks_of(x)
        s = xb.abs().amax(1)
        tiny = s < 2.0 ** -126
        near(scale, torch.where(tiny, torch.zeros_like(s), s), 8 * U * s, "scale")
        k = top * torch.sqrt(xb.abs() / s.clamp_min(1e-300)[:, None])
        k = torch.where(tiny[:, None], torch.zeros_like(k), k)
        want = torch.where((k > 0) & ~tiny[:, None], k.clamp_min(low), k) * torch.sign(xb)
        got = blocks_of(code.cpu()).double()
        half = 0.5 + 2.0 ** -12
        # (a v that float32's underflow may have taken to 0 may have the code 0)
        lost = blocks_of(v <= d_v) & (got == 0) & (k < 0.5) if low else torch.zeros_like(got, dtype=torch.bool)
        assert (((got - want).abs() <= half) | lost).view(-1)[:n].all()
        if low:
            assert ((got >= 1) | (k == 0) | lost).view(-1)[:n].all()


def make(sizes, param=F32, master=False, grad=F32, bits=32, shift=0, seed=0, step=5):
    """An optimiser over tensors cut from flat buffers, `shift` elements off
    their starts, with states as after some steps."""
    gen = torch.Generator().manual_seed(seed)
    params = []
    for k, n in enumerate(sizes):
        def cut(t, dt):
            buf = torch.zeros(n + shift, dtype=dt, device="cuda")
            buf[shift:] = t.to(dt).cuda()
            return buf[shift:]
        p0 = torch.randn(n, generator=gen) * 0.1
        q = dict(param=cut(p0, param), grad=cut(torch.randn(n, generator=gen) * torch.exp(torch.randn(n, generator=gen)) * 1e-2, grad),
                 weight_decay=0.05 * (k % 2))
        if master:
            q["master"] = cut(p0, F32)
        m, v = torch.randn(n, generator=gen) * 1e-3, (torch.randn(n, generator=gen) * 1e-2) ** 2
        if bits == 8:
            blocks = -(-n // 256)
            sm = blocks_of(m).abs().amax(1) if n else torch.zeros(0)
            sv = blocks_of(v).sqrt().amax(1) if n else torch.zeros(0)
            code_m = torch.round(127 * torch.sqrt(blocks_of(m).abs() / sm[:, None])) * torch.sign(blocks_of(m))
            code_v = torch.round(255 * torch.sqrt(blocks_of(v).sqrt() / sv[:, None])).clamp_min(1)
            q.update(m=cut(code_m.view(-1)[:n], torch.int8), v=cut(code_v.view(-1)[:n], torch.uint8),
                     m_scale=sm.cuda(), v_scale=sv.cuda())
            assert q["m_scale"].numel() == blocks
        else:
            q.update(m=cut(m, F32), v=cut(v, F32))
        params.append(q)
    return optim.AdamW(params, lr=LR, betas=(B1, B2), eps=EPS, step=step)


def run_and_check(opt, scale=None):
    before = [(decode(q), {k: (q[k].clone() if isinstance(q.get(k), torch.Tensor) else q.get(k)) for k in q}) for q in opt.params]
    s = None if scale is None else torch.tensor([scale], device="cuda")
    opt.step(grad_scale=s)
    t = opt.step_count
    for q, ((m, v), old) in zip(opt.params, before):
        p, m, v, d_p, d_m, d_v = plain_step(old, m, v, t, 1.0 if scale is None else scale, q["weight_decay"])
        if q.get("master") is not None:
            near(q["master"], p, d_p, "master")
        half = 2.0 ** -8 * (p.abs() + d_p) * 1.01 if q["param"].dtype == BF16 else 0
        near(q["param"], p, d_p + half, "param")
        if q["m"].dtype == torch.int8:
            check_codes(q, m, v, d_m, d_v)
        else:
            near(q["m"], m, d_m, "m")
            near(q["v"], v, d_v, "v")
    got = opt.state_values()
    for q, (m, v) in zip(opt.params, got):
        wm, wv = decode(q)
        near(m, wm, 6 * U * wm.abs(), "m value")
        near(v, wv, 13 * U * wv, "v value")
    assert all(torch.equal(q["grad"], old["grad"]) for q, (_, old) in zip(opt.params, before))


SIZES = [1, 0, 2, 255, 256, 257, 2047, 2048, 2049, 5000, 100003]
MODES = [(F32, False, F32), (F32, False, BF16), (BF16, True, F32), (BF16, True, BF16), (BF16, False, F32), (BF16, False, BF16)]


@on_gpu
@pytest.mark.parametrize("bits", (32, 8))
@pytest.mark.parametrize("shift", (0, 1, 4, 8))
@pytest.mark.parametrize("param,master,grad", MODES)
def test_step_matches_the_plain_form(param, master, grad, shift, bits):
    opt = make(SIZES, param, master, grad, bits, shift, seed=shift + bits)
    run_and_check(opt, None)
    run_and_check(opt, 0.37)


@on_gpu
@pytest.mark.parametrize("bits", (32, 8))
def test_first_step_from_zero_states(bits):
    gen = torch.Generator().manual_seed(1)
    params = [dict(param=torch.randn(n, generator=gen).cuda(), grad=torch.randn(n, generator=gen).cuda()) for n in (7, 300, 4096)]
    opt = optim.AdamW(params, lr=LR, betas=(B1, B2), eps=EPS, weight_decay=0.0, state_bits=bits)
    old = [q["param"].clone() for q in opt.params]
    run_and_check(opt)
    for q, p in zip(opt.params, old):  # the first step moves every element by lr against its gradient's sign
        near(q["param"], (p - LR * torch.sign(q["grad"])).double().cpu(), 1e-5 * LR + 4 * U * p.abs().double().cpu(), "first step")


@on_gpu
def test_more_tensors_than_one_launch_takes_and_mixed_kinds():
    gen = torch.Generator().manual_seed(2)
    sizes = [int(v) for v in torch.randint(0, 3000, (1001,), generator=gen)]
    parts = [make(sizes[k::4], *MODES[k], 32 if k % 2 else 8, k, seed=k).params for k in range(4)]
    params = [parts[i % 4][i // 4] for i in range(len(sizes))]
    opt = optim.AdamW(params, lr=LR, betas=(B1, B2), eps=EPS, step=9)
    n0 = B.launch_count()
    opt.step()
    assert B.launch_count() - n0 == 3
    run_and_check(opt, 0.5)


@on_gpu
@pytest.mark.parametrize("bits", (32, 8))
@pytest.mark.parametrize("scale", (float("nan"), float("inf")))
def test_a_scale_that_is_not_finite_skips_the_step(scale, bits):
    opt = make([5, 3000], BF16, True, F32, bits)
    old = [{k: t.clone() for k, t in q.items() if isinstance(t, torch.Tensor)} for q in opt.params]
    opt.step(grad_scale=torch.tensor([scale], device="cuda"))
    for q, o in zip(opt.params, old):
        assert all(torch.equal(q[k], o[k]) for k in o)


@on_gpu
@pytest.mark.parametrize("value", (float("nan"), float("inf")))
def test_a_gradient_that_is_not_finite_stays_in_its_element_or_block(value):
    for bits in (32, 8):
        opt, ref = (make([1000], bits=bits, seed=3) for _ in range(2))
        opt.params[0]["grad"][300] = value
        opt.step()
        ref.step()
        a, b = opt.params[0], ref.params[0]
        other = torch.arange(1000, device="cuda") != 300
        assert torch.equal(a["param"][other], b["param"][other]) and not torch.isfinite(a["param"][300])
        m, v = opt.state_values()[0]
        rm, rv = ref.state_values()[0]
        hit = ~other if bits == 32 else (torch.arange(1000, device="cuda") // 256 == 1)
        assert torch.equal(m[~hit], rm[~hit]) and torch.equal(v[~hit], rv[~hit])
        assert not torch.isfinite(m[hit]).any() and not torch.isfinite(v[hit]).any()


@on_gpu
def test_blocks_of_zeros_of_tiny_and_of_far_apart_values():
    n = 5 * 256
    g = torch.zeros(n)
    g[256:512] = torch.linspace(-1, 1, 256) * 1e-38      # states below the smallest normal number
    g[512:768] = torch.logspace(-30, 0, 256)             # ratios far beyond the code's range
    g[768] = 1e18                                        # one huge value among zeros
    g[1024:] = 1e-3
    q = dict(param=torch.zeros(n, device="cuda"), grad=g.cuda())
    opt = optim.AdamW([q], lr=LR, betas=(B1, B2), eps=EPS, weight_decay=0.0, state_bits=8)
    q = opt.params[0]
    for _ in range(3):
        run_and_check(opt)
    assert torch.isfinite(q["param"]).all()
    assert not q["m"][:256].any() and not q["v"][:256].any()
    assert (q["v"][768 + 1:1024] == 0).all()
    # a small element beside large ones keeps a second moment above zero
    live = (opt.state_values()[0][1][512:768] > 0)
    assert torch.equal(live, (g[512:768] * g[512:768] * torch.tensor(1 - B2)).cuda() > 0)


@on_gpu
def test_a_captured_step_follows_its_schedule():
    a, b = (make([700, 4097], BF16, True, F32, 8, seed=4) for _ in range(2))
    sched = torch.zeros(3, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            a.step(schedule=sched)
    torch.cuda.synchronize()
    for t in range(6, 9):
        lr = LR * (10 - t) / 4
        sched.copy_(a.schedule(t, lr))
        graph.replay()
        b.lr = lr
        b.step()
        torch.cuda.synchronize()
        for q, r in zip(a.params, b.params):
            # the schedule's numbers are rounded before they are divided
            near(q["master"], r["master"].double().cpu(), 4 * U * r["master"].abs().double().cpu() + 2e-6 * lr, "master")
            assert torch.equal(q["m"], r["m"]) and torch.equal(q["v"], r["v"])


@on_gpu
def test_state_dict_resumes_bit_for_bit():
    a, b = make([513, 9000], F32, False, F32, 8, seed=6), make([513, 9000], F32, False, F32, 8, seed=7)
    a.step()
    b.load_state_dict(a.state_dict())
    for q, r in zip(a.params, b.params):
        r["param"].copy_(q["param"]), r["grad"].copy_(q["grad"])
    a.step(), b.step()
    for q, r in zip(a.params, b.params):
        assert all(torch.equal(q[k], r[k]) for k in ("param", "m", "v", "m_scale", "v_scale"))
    with pytest.raises(ValueError):
        make([513, 9000], bits=32).load_state_dict(a.state_dict())


@on_gpu
@pytest.mark.parametrize("bits", (32, 8))
def test_state_dict_carries_the_masters(bits):
    a, b = (make([513, 9000], BF16, True, F32, bits, seed=k) for k in (6, 7))
    a.step()
    saved = a.state_dict()
    b.load_state_dict(saved)
    for q, r in zip(a.params, b.params):
        assert torch.equal(q["master"], r["master"]) and torch.equal(q["param"], r["param"])
        r["grad"].copy_(q["grad"])
    a.step(), b.step()
    for q, r in zip(a.params, b.params):
        assert all(torch.equal(q[k], r[k]) for k in ("param", "master", "m", "v"))
    # a state of another kind changes nothing
    short = dict(saved, state=[saved["state"][0], dict(saved["state"][1], master=saved["state"][1]["master"][1:])])
    old = [r["master"].clone() for r in b.params]
    with pytest.raises(ValueError):
        b.load_state_dict(short)
    assert all(torch.equal(r["master"], o) for r, o in zip(b.params, old))
    with pytest.raises(ValueError):
        make([513, 9000], F32, False, F32, bits).load_state_dict(saved)
    # one saved without masters leaves them as they are
    b.load_state_dict(dict(saved, state=[{k: v for k, v in s.items() if k != "master"} for s in saved["state"]]))
    assert all(torch.equal(r["master"], o) for r, o in zip(b.params, old))


@on_gpu
def test_side_stream():
    opt, ref = (make([3000, 70001], BF16, True, BF16, 8, seed=8) for _ in range(2))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        _, scale = opt.grad_norm(0.1)
        opt.step(scale)
    s.synchronize()
    _, scale = ref.grad_norm(0.1)
    ref.step(scale)
    for q, r in zip(opt.params, ref.params):
        assert all(torch.equal(q[k], r[k]) for k in ("param", "master", "m", "v", "m_scale", "v_scale"))


@on_gpu
def test_offsets_beyond_32_bits():
    n = 2 ** 31 + 1003
    gen = torch.Generator(device="cuda").manual_seed(5)
    q = dict(param=torch.empty(n, dtype=BF16, device="cuda").normal_(generator=gen),
             grad=torch.empty(n, dtype=BF16, device="cuda").normal_(generator=gen))
    opt = optim.AdamW([q], lr=LR, betas=(B1, B2), eps=EPS, weight_decay=0.0, state_bits=8)
    q = opt.params[0]
    # the last whole blocks and the short one at the end, in an optimiser of their own
    k = 256 * 8 + n % 256
    small = optim.AdamW([dict(param=q["param"][-k:].clone(), grad=q["grad"][-k:].clone())], lr=LR, betas=(B1, B2),
                        eps=EPS, weight_decay=0.0, state_bits=8)
    norm, _ = opt.grad_norm(1.0)
    opt.step()
    small.step()
    r = small.params[0]
    for key in ("param", "m", "v"):
        assert torch.equal(q[key][-k:], r[key])
    # (N(0, 1) rounded to bf16: the squares' mean is 1 within a few parts in 10^4)
    assert abs(float(norm) / math.sqrt(n) - 1) < 1e-3


# ---------------------------------------------------------------- gradient norm

def exact_norm(grads):
    return math.sqrt(sum(float(g.double().square().sum()) for g in grads))


@on_gpu
@pytest.mark.parametrize("dtype", (F32, BF16))
@pytest.mark.parametrize("shift", (0, 1, 3))
def test_norm_matches_the_plain_form(dtype, shift):
    gen = torch.Generator().manual_seed(shift)
    for sizes in ([1], [0], [3, 0, 2049], SIZES, [1000000], [17] * 900):
        grads = [(torch.randn(n + shift, generator=gen) * 3).to(dtype).cuda()[shift:] for n in sizes]
        norm, scale = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
        optim.GradNorm(grads)(2.0, norm, scale)
        want = exact_norm(grads)
        # non-negative terms: at most 2^11 roundings of a running sum in a row, halved by the root
        assert abs(float(norm) - want) <= 2 ** 10 * U * want
        assert abs(float(scale) - min(1.0, 2.0 / (want + 1e-6))) <= (2 ** 10 + 8) * U
        again = torch.empty(1, device="cuda")
        optim.GradNorm(grads)(2.0, again, None)
        assert torch.equal(again, norm)


@on_gpu
def test_norm_of_nothing_of_no_limit_and_of_what_is_not_finite():
    norm, scale = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
    optim.GradNorm([])(1.0, norm, scale)
    assert float(norm) == 0.0 and float(scale) == 1.0
    g = torch.randn(5000, device="cuda")
    optim.GradNorm([g])(math.inf, None, scale)
    assert float(scale) == 1.0
    for value in (math.nan, math.inf, 1e30):
        h = g.clone()
        h[4321] = value
        optim.GradNorm([g, h])(1.0, norm, scale)
        assert not math.isfinite(float(norm)) and math.isnan(float(scale))


@on_gpu
def test_gradients_are_renewed_by_set_grads_alone():
    opt, ref = (make([5, 3000, 4097], BF16, True, F32, 8, seed=9) for _ in range(2))
    # the table holds addresses: a tensor put into the optimiser's dicts would not be read
    with pytest.raises(TypeError):
        opt.params[1]["grad"] = torch.ones_like(opt.params[1]["grad"])
    with pytest.raises(TypeError):
        opt.params[1] = dict(opt.params[1])
    opt.grad_norm(1.0)
    gen = torch.Generator().manual_seed(10)
    for dtype in (F32, BF16):
        fresh = [torch.randn(q["grad"].shape, generator=gen).to(dtype).cuda() for q in ref.params]
        opt.set_grads(fresh)
        assert all(q["grad"] is g for q, g in zip(opt.params, fresh))
        norm, scale = opt.grad_norm(0.5)
        assert abs(float(norm) - exact_norm(fresh)) <= 2 ** 10 * U * exact_norm(fresh)
        opt.step(scale)
        want = optim.AdamW([dict(q, grad=g) for q, g in zip(ref.params, fresh)], lr=LR, betas=(B1, B2), eps=EPS, step=ref.step_count)
        want.step(scale)
        ref._hyper.step = want.step_count
        for q, r in zip(opt.params, ref.params):
            assert all(torch.equal(q[k], r[k]) for k in ("param", "master", "m", "v", "m_scale", "v_scale"))
    # refusals leave the gradients that were there
    for bad in (fresh[:2], [g[:-1] for g in fresh], [g.double() for g in fresh], [g.cpu() for g in fresh], [None] + fresh[1:]):
        with pytest.raises(ValueError):
            opt.set_grads(bad)
    assert all(q["grad"] is g for q, g in zip(opt.params, fresh))
    # the norm's own list
    n = optim.GradNorm(fresh)
    with pytest.raises(TypeError):
        n.grads[0] = fresh[0]
    with pytest.raises(ValueError):
        n.set_grads(fresh[1:])
    other = [2 * g for g in fresh]
    n.set_grads(other)
    out = torch.empty(1, device="cuda")
    n(1.0, out, None)
    assert abs(float(out) - exact_norm(other)) <= 2 ** 10 * U * exact_norm(other)
