"""Group norm with an activation: the 64-bit plain form against differences
(CPU), the refusals (CPU), and the kernels against the plain form (GPU)."""
import ctypes
import dataclasses

import pytest
import torch

import norm_plain as P
from deformable_convolution_gb300 import binding as B

gpu = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


def on_gpu(f):
    for m in gpu:
        f = m(f)
    return f


ACTS = (B.DC_ACT_NONE, B.DC_ACT_RELU, B.DC_ACT_SILU, B.DC_ACT_GELU)


# ---------------------------------------------------------------- the plain form

@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("layout", (B.DC_NCHW, B.DC_NHWC))
def test_plain_gradients_match_differences(act, layout):
    p = B.NormProblem(2, 6, 3, 4, 3, B.DC_F32, layout, act, 1e-5)
    gen = torch.Generator().manual_seed(3)
    x, gy, dx = (torch.randn(p.shape, generator=gen, dtype=torch.float64) for _ in range(3))
    gamma, beta, dg, db = (torch.randn(p.c, generator=gen, dtype=torch.float64) for _ in range(4))

    def loss(t):
        return float((P.forward(p, x + t * dx, gamma + t * dg, beta + t * db)["y"] * gy).sum())

    f = P.forward(p, x, gamma, beta)
    g = P.backward(p, x, gamma, beta, f["mean"], f["rstd"], gy)
    want = (g["grad_x"] * dx).sum() + (g["grad_gamma"] * dg).sum() + (g["grad_beta"] * db).sum()
    # central differences: error h^2 times the third derivative, and rounding / h
    h = 1e-6
    assert abs((loss(h) - loss(-h)) / (2 * h) - float(want)) < 1e-6 * (1 + abs(float(want)))


# ---------------------------------------------------------------- refusals

def ws_status(p):
    out = ctypes.c_size_t(0)
    st = p.c_struct()
    return B.lib().dc_group_norm_workspace_size(ctypes.byref(st), 0, ctypes.byref(out))


GOOD = B.NormProblem(2, 8, 5, 6, 4, B.DC_BF16, B.DC_NHWC, B.DC_ACT_SILU, 1e-5, B.DC_BF16)


@pytest.mark.parametrize("kw,status", [
    (dict(), B.DC_OK), (dict(n=0), B.DC_OK), (dict(eps=0.0), B.DC_OK), (dict(grad_dtype=B.DC_F32), B.DC_OK),
    (dict(n=-1), B.DC_ERR_INVALID_ARG), (dict(c=0), B.DC_ERR_INVALID_ARG), (dict(h=0), B.DC_ERR_INVALID_ARG),
    (dict(w=-3), B.DC_ERR_INVALID_ARG), (dict(groups=0), B.DC_ERR_INVALID_ARG),
    (dict(groups=3), B.DC_ERR_INVALID_ARG), (dict(dtype=2), B.DC_ERR_INVALID_ARG),
    (dict(layout=2), B.DC_ERR_INVALID_ARG), (dict(act=4), B.DC_ERR_INVALID_ARG),
    (dict(act=-1), B.DC_ERR_INVALID_ARG), (dict(eps=-1e-5), B.DC_ERR_INVALID_ARG),
    (dict(eps=float("nan")), B.DC_ERR_INVALID_ARG), (dict(eps=float("inf")), B.DC_ERR_INVALID_ARG),
    (dict(dtype=B.DC_F32), B.DC_ERR_INVALID_ARG),  # a bf16 gradient of a float32 problem
    (dict(h=1 << 16, w=1 << 15), B.DC_ERR_UNSUPPORTED), (dict(c=1 << 21), B.DC_ERR_UNSUPPORTED),
    (dict(n=1 << 30), B.DC_ERR_UNSUPPORTED),
])
def test_problems_are_checked(kw, status):
    assert ws_status(dataclasses.replace(GOOD, **kw)) == status


def test_calls_check_their_arguments_before_any_launch():
    # made-up addresses: every check is on the host, ahead of the first launch
    st = GOOD.c_struct()
    vp = ctypes.c_void_p

    def fwd(ptrs, ws_bytes):
        return B.lib().dc_group_norm_fwd(ctypes.byref(st), *[vp(v) if v else None for v in ptrs], ws_bytes, None)

    def bwd(ptrs, ws_bytes):
        return B.lib().dc_group_norm_bwd(ctypes.byref(st), *[vp(v) if v else None for v in ptrs], ws_bytes, None)

    def swap(ptrs, k, v):
        return ptrs[:k] + [v] + ptrs[k + 1:]

    f = [0x10000 * (i + 1) for i in range(7)]   # x gamma beta y mean rstd ws
    b = [0x10000 * (i + 1) for i in range(10)]  # x gamma beta mean rstd gy gx ggamma gbeta ws
    big = 1 << 30
    for k in (0, 3):
        assert fwd(swap(f, k, 0), big) == B.DC_ERR_INVALID_ARG
    for k in range(7):
        assert fwd(swap(f, k, f[k] + 8), big) == B.DC_ERR_UNSUPPORTED
    for k in (0, 3, 4, 5, 6):
        assert bwd(swap(b, k, 0), big) == B.DC_ERR_INVALID_ARG
    for k in range(10):
        assert bwd(swap(b, k, b[k] + 4), big) == B.DC_ERR_UNSUPPORTED
    for call, ptrs, back in ((fwd, f, False), (bwd, b, True)):
        need = B.dc_group_norm_workspace_size(GOOD, back)
        if need:
            assert call(ptrs, need - 1) == B.DC_ERR_WORKSPACE
            assert call(swap(ptrs, len(ptrs) - 1, 0), need) == B.DC_ERR_WORKSPACE
    assert B.lib().dc_group_norm_fwd(None, *[vp(v) for v in f], big, None) == B.DC_ERR_INVALID_ARG


@on_gpu
def test_binding_checks_shapes_types_and_contiguity():
    p = GOOD
    x = torch.zeros(p.shape, dtype=torch.bfloat16, device="cuda")
    y, ws = torch.empty_like(x), B.norm_workspace(p, False)
    for bad in (x.float(), x[:, :, :, :4], x.cpu(), x.permute(0, 3, 1, 2)):
        with pytest.raises(ValueError):
            B.dc_group_norm_fwd(p, bad, None, None, y, ws=ws)
    strided = torch.zeros((*p.shape[:3], 2 * p.c), dtype=torch.bfloat16, device="cuda")[..., ::2]
    with pytest.raises(ValueError):
        B.dc_group_norm_fwd(p, strided, None, None, y, ws=ws)
    with pytest.raises(ValueError):
        B.dc_group_norm_fwd(p, x, torch.ones(p.c, device="cuda", dtype=torch.bfloat16), None, y, ws=ws)
    with pytest.raises(ValueError):
        B.dc_group_norm_fwd(p, x, None, torch.ones(p.c + 1, device="cuda"), y, ws=ws)


# ---------------------------------------------------------------- the kernels

def inputs(p, seed, offset=0.5, spread=1.0):
    gen = torch.Generator().manual_seed(seed)
    dt = p.torch_dtype
    x = (torch.randn(p.shape, generator=gen) * spread + offset).to(dt)
    gy = torch.randn(p.shape, generator=gen).to(torch.bfloat16 if p.grad_dtype == B.DC_BF16 else torch.float32)
    gamma = 1 + 0.2 * torch.randn(p.c, generator=gen)
    beta = 0.2 * torch.randn(p.c, generator=gen)
    return x, gamma, beta, gy


def cuda(t):
    return None if t is None else t.cuda()


def within(got, want, bound, what):
    err = (got.double().cpu() - want).abs()
    assert err.shape == want.shape
    bad = ~(err <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} beyond the bound, worst {float((err / bound).max()):.3g} of it"


def check(p, x, gamma, beta, gy):
    xd, gd, bd, gyd = map(cuda, (x, gamma, beta, gy))
    y, mean, rstd = B.group_norm(p, xd, gd, bd)
    f = P.forward(p, x, gamma, beta)
    for got, k in ((mean, "mean"), (rstd, "rstd"), (y, "y")):
        within(got, f[k], f["d_" + k], k)
    assert y.dtype == p.torch_dtype
    g = B.group_norm_backward(p, xd, gd, bd, mean, rstd, gyd)
    w = P.backward(p, x, gamma, beta, mean.cpu(), rstd.cpu(), gy)
    for k in ("grad_x", "grad_gamma", "grad_beta"):
        within(g[k], w[k], w["d_" + k], k)
    return y, mean, rstd, g


SHAPES = [  # n, c, h, w, groups
    (1, 1, 1, 1, 1), (1, 8, 1, 1, 8), (3, 8, 1, 1, 2), (2, 6, 5, 7, 3), (1, 16, 32, 32, 4), (3, 60, 13, 9, 12),
    (2, 40, 7, 7, 4), (5, 24, 3, 3, 8), (2, 320, 10, 10, 32), (2, 64, 17, 19, 1), (1, 256, 28, 28, 32),
    (1, 4, 120, 131, 2), (2, 2048, 4, 4, 1), (1, 36, 9, 1, 4), (300, 2, 1, 2, 1), (2, 33, 21, 5, 33),
    (1, 12, 64, 200, 1), (2, 128, 56, 56, 32),
]


@on_gpu
@pytest.mark.parametrize("layout", (B.DC_NCHW, B.DC_NHWC))
@pytest.mark.parametrize("dtype,grad", [(B.DC_F32, B.DC_F32), (B.DC_BF16, B.DC_BF16), (B.DC_BF16, B.DC_F32)])
@pytest.mark.parametrize("shape", SHAPES)
def test_kernels_match_the_plain_form(shape, dtype, grad, layout):
    n, c, h, w, groups = shape
    act = ACTS[(c + h + w + dtype + layout) % 4]
    p = B.NormProblem(n, c, h, w, groups, dtype, layout, act, 1e-5, grad)
    check(p, *inputs(p, 11 + c))


@on_gpu
@pytest.mark.parametrize("layout", (B.DC_NCHW, B.DC_NHWC))
@pytest.mark.parametrize("dtype", (B.DC_F32, B.DC_BF16))
@pytest.mark.parametrize("act", ACTS)
def test_every_activation(act, dtype, layout):
    p = B.NormProblem(2, 24, 11, 13, 4, dtype, layout, act, 1e-5, dtype)
    x, gamma, beta, gy = inputs(p, 5, spread=3.0)
    check(p, x, gamma, beta, gy)
    check(p, x, None, None, gy)
    check(p, x, 20 * gamma, 20 * beta, gy)  # both tails of the activations


@on_gpu
@pytest.mark.parametrize("layout", (B.DC_NCHW, B.DC_NHWC))
@pytest.mark.parametrize("shape", [(2, 16, 40, 40, 2), (1, 8, 150, 150, 1)])
def test_a_mean_far_above_the_spread_keeps_the_variance(shape, layout):
    n, c, h, w, groups = shape
    p = B.NormProblem(n, c, h, w, groups, B.DC_F32, layout, B.DC_ACT_NONE, 1e-5)
    x, gamma, beta, gy = inputs(p, 6, offset=4000.0)
    # the first pixels apart from the rest: no origin taken from them may cost digits
    x.view(-1)[:: x.numel() // (2 * n)] = 3900.0
    y, mean, rstd, _ = check(p, x, gamma, beta, gy)
    assert torch.isfinite(y).all()


@on_gpu
@pytest.mark.parametrize("layout", (B.DC_NCHW, B.DC_NHWC))
def test_constant_groups(layout):
    p = B.NormProblem(2, 8, 9, 9, 4, B.DC_F32, layout, B.DC_ACT_RELU, 1e-5)
    x = torch.full(p.shape, 3.0)
    gamma, beta = torch.ones(8), torch.linspace(-1, 1, 8)
    y, mean, rstd, g = check(p, x, gamma, beta, torch.randn(p.shape, generator=torch.Generator().manual_seed(1)))
    assert torch.equal(mean.cpu(), torch.full((2, 4), 3.0))
    # eps 0 over a constant group has no answer: not a number, and no fault
    q = dataclasses.replace(p, eps=0.0)
    y = B.group_norm(q, x.cuda(), cuda(gamma), cuda(beta))[0]
    assert torch.isnan(y).all()


@on_gpu
@pytest.mark.parametrize("layout", (B.DC_NCHW, B.DC_NHWC))
@pytest.mark.parametrize("value", (float("nan"), float("inf"), -float("inf")))
def test_a_value_that_is_not_finite_stays_in_its_group(value, layout):
    p = B.NormProblem(2, 16, 12, 11, 4, B.DC_BF16, layout, B.DC_ACT_SILU, 1e-5, B.DC_BF16)
    x, gamma, beta, gy = inputs(p, 8)
    clean = B.group_norm(p, x.cuda(), gamma.cuda(), beta.cuda())
    x2 = x.clone()
    if layout == B.DC_NHWC:
        x2[1, 3, 2, 5] = value
    else:
        x2[1, 5, 3, 2] = value
    y, mean, rstd = B.group_norm(p, x2.cuda(), gamma.cuda(), beta.cuda())
    hit = torch.zeros(p.n, p.groups, p.c // p.groups, p.h * p.w, dtype=torch.bool)
    hit[1, 1] = True
    hit = P.layout(p, hit).cuda()
    assert torch.isnan(y[hit]).all()
    assert torch.equal(y[~hit].view(torch.int16), clean[0][~hit].view(torch.int16))


@on_gpu
@pytest.mark.parametrize("layout", (B.DC_NCHW, B.DC_NHWC))
def test_in_place_side_stream_and_same_bits_twice(layout):
    p = B.NormProblem(4, 48, 31, 17, 6, B.DC_BF16, layout, B.DC_ACT_GELU, 1e-5, B.DC_BF16)
    x, gamma, beta, gy = (t.cuda() for t in inputs(p, 9))
    y, mean, rstd = B.group_norm(p, x, gamma, beta)
    g = B.group_norm_backward(p, x, gamma, beta, mean, rstd, gy)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        a = x.clone()
        m2, r2 = torch.empty_like(mean), torch.empty_like(rstd)
        B.dc_group_norm_fwd(p, a, gamma, beta, a, m2, r2, B.norm_workspace(p, False))
        b = gy.clone()
        gg, gb = torch.empty_like(gamma), torch.empty_like(beta)
        B.dc_group_norm_bwd(p, x, gamma, beta, m2, r2, b, b, gg, gb, B.norm_workspace(p, True))
    s.synchronize()
    for u, v in ((a, y), (m2, mean), (r2, rstd), (b, g["grad_x"]), (gg, g["grad_gamma"]), (gb, g["grad_beta"])):
        assert torch.equal(u, v)
    # mean and rstd are optional, as are the parameters' gradients
    y2 = torch.full_like(x, 7)
    B.dc_group_norm_fwd(p, x, gamma, beta, y2, ws=B.norm_workspace(p, False))
    gx2 = torch.full_like(x, 7)
    B.dc_group_norm_bwd(p, x, gamma, beta, mean, rstd, gy, gx2, ws=B.norm_workspace(p, True))
    assert torch.equal(y2, y) and torch.equal(gx2, g["grad_x"])


@on_gpu
def test_empty_batch():
    p = B.NormProblem(0, 8, 4, 4, 2, B.DC_F32, B.DC_NHWC, B.DC_ACT_RELU)
    x = torch.empty(p.shape, device="cuda")
    y, mean, rstd = B.group_norm(p, x)
    assert y.shape == p.shape and mean.shape == (0, 2)
    gg, gb = torch.full((8,), 5.0, device="cuda"), torch.full((8,), 5.0, device="cuda")
    B.dc_group_norm_bwd(p, x, None, None, mean, rstd, y, y, gg, gb)
    assert not gg.any() and not gb.any()


@on_gpu
@pytest.mark.parametrize("layout", (B.DC_NCHW, B.DC_NHWC))
def test_many_images(layout):
    p = B.NormProblem(70001, 2, 1, 3, 1, B.DC_F32, layout, B.DC_ACT_NONE)
    check(p, *inputs(p, 10))


@on_gpu
@pytest.mark.parametrize("layout", (B.DC_NCHW, B.DC_NHWC))
@pytest.mark.parametrize("shape", [(2, 64, 4200, 4000, 32), (130, 64, 512, 512, 8)])
def test_offsets_beyond_32_bits(shape, layout):
    n, c, h, w, groups = shape
    p = B.NormProblem(n, c, h, w, groups, B.DC_BF16, layout, B.DC_ACT_SILU, 1e-5, B.DC_BF16)
    assert n * c * h * w > 2 ** 31
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.empty(p.shape, dtype=torch.bfloat16, device="cuda").normal_(0.5, 1.0, generator=gen)
    gy = torch.empty_like(x).normal_(generator=gen)
    gamma, beta = 1 + 0.1 * torch.randn(c, device="cuda", generator=gen), 0.1 * torch.randn(c, device="cuda", generator=gen)
    y, mean, rstd = B.group_norm(p, x, gamma, beta)
    g = B.group_norm_backward(p, x, gamma, beta, mean, rstd, gy)
    # the last image's last group, in 64 bits on the GPU
    per = c // groups
    q = dataclasses.replace(p, n=1, c=per, groups=1)
    cut = (lambda t: t[-1:, :, :, -per:]) if layout == B.DC_NHWC else (lambda t: t[-1:, -per:])
    one = dict(x=cut(x), gy=cut(gy), gamma=gamma[-per:], beta=beta[-per:], mean=mean[-1:, -1:], rstd=rstd[-1:, -1:])
    f = P.forward(q, one["x"], one["gamma"], one["beta"])
    for got, k in ((one["mean"], "mean"), (one["rstd"], "rstd"), (cut(y), "y")):
        assert ((got.double() - f[k]).abs() <= f["d_" + k]).all(), k
    del f
    b = P.backward(q, one["x"], one["gamma"], one["beta"], one["mean"], one["rstd"], one["gy"])
    assert ((cut(g["grad_x"]).double() - b["grad_x"]).abs() <= b["d_grad_x"]).all()


@on_gpu
@pytest.mark.parametrize("layout", (B.DC_NCHW, B.DC_NHWC))
def test_gradients_match_differences_of_the_plain_forward(layout):
    p = B.NormProblem(2, 12, 6, 5, 3, B.DC_F32, layout, B.DC_ACT_GELU, 1e-5)
    x, gamma, beta, gy = inputs(p, 21)
    xd, gd, bd, gyd = map(cuda, (x, gamma, beta, gy))
    _, mean, rstd = B.group_norm(p, xd, gd, bd)
    g = B.group_norm_backward(p, xd, gd, bd, mean, rstd, gyd)
    gen = torch.Generator().manual_seed(4)
    dx = torch.randn(p.shape, generator=gen, dtype=torch.float64)
    dg, db = (torch.randn(p.c, generator=gen, dtype=torch.float64) for _ in range(2))

    def loss(t):
        return float((P.forward(p, x.double() + t * dx, gamma.double() + t * dg, beta.double() + t * db)["y"] * gy).sum())

    terms = [g["grad_x"].double().cpu() * dx, g["grad_gamma"].double().cpu() * dg, g["grad_beta"].double().cpu() * db]
    want = sum(float(t.sum()) for t in terms)
    scale = sum(float(t.abs().sum()) for t in terms)
    h = 1e-6
    # float32 gradients: 2^-18 of the terms' absolute sum; the differences add 1e-6
    assert abs((loss(h) - loss(-h)) / (2 * h) - want) < 2.0 ** -18 * scale + 1e-6 * (1 + abs(want))


@on_gpu
def test_a_group_of_more_than_2_to_the_31_vectors():
    c, size = 66, 16384
    p = B.NormProblem(1, c, size, size, 1, B.DC_BF16, B.DC_NCHW, B.DC_ACT_SILU, 1e-5, B.DC_BF16)
    gen = torch.Generator(device="cuda").manual_seed(7)
    plane = torch.empty(size, size, device="cuda").normal_(generator=gen)
    scale = 0.5 + torch.rand(c, generator=torch.Generator().manual_seed(8))
    shift = torch.linspace(-1, 1, c)

    def channel(k):
        return (plane * float(scale[k]) + float(shift[k])).to(torch.bfloat16)

    x = torch.empty(p.shape, dtype=torch.bfloat16, device="cuda")
    sums, top = torch.zeros(2, dtype=torch.float64, device="cuda"), 0.0
    for k in range(c):
        x[0, k] = channel(k)
        v = x[0, k].double()
        sums += torch.stack([v.sum(), v.square().sum()])
        top = max(top, float(v.abs().max()))
    m = c * size * size
    mean = float(sums[0]) / m
    var = float(sums[1]) / m - mean ** 2  # (64 bits: the mean is of the spread's order)
    rstd = (var + p.eps) ** -0.5
    gamma = 1 + 0.2 * torch.randn(c, generator=torch.Generator().manual_seed(9))
    beta = torch.linspace(-0.5, 0.5, c)
    got_mean, got_rstd = (torch.empty(1, 1, device="cuda") for _ in range(2))
    B.dc_group_norm_fwd(p, x, gamma.cuda(), beta.cuda(), x, got_mean, got_rstd, B.norm_workspace(p, False))  # in place
    # a thread merges at most 2^12 batches one after the other, each a rounding
    # of the mean and of the variance; then 64 as at every other size
    chain = (2 ** 12 + 64) * P.U
    d_mean = chain * top
    d_rstd = rstd * (chain + 0.5 * rstd ** 2 * d_mean ** 2)
    assert abs(float(got_mean) - mean) <= d_mean and abs(float(got_rstd) - rstd) <= d_rstd
    for k in range(c):
        z = (channel(k).double() - mean) * rstd * float(gamma[k]) + float(beta[k])
        want = z / (1 + torch.exp(-z))
        d_z = abs(float(gamma[k])) * rstd * d_mean + (z.abs() + 1) * d_rstd / rstd + 8 * P.U * (z.abs() + 1)
        bound = 1.2 * d_z + (want.abs() + 1.2 * d_z) * 2.0 ** -8 * 1.01
        assert ((x[0, k].double() - want).abs() <= bound).all(), k


NOT_FINITE_SHAPES = [  # n, c, h, w, groups: in one launch and in two, whole vectors and odd rows
    (2, 16, 12, 12, 4), (2, 12, 11, 13, 4), (2, 16, 400, 336, 2), (2, 20, 401, 333, 2),
]


@on_gpu
@pytest.mark.parametrize("layout", (B.DC_NCHW, B.DC_NHWC))
@pytest.mark.parametrize("dtype,grad", [(B.DC_F32, B.DC_F32), (B.DC_BF16, B.DC_BF16), (B.DC_BF16, B.DC_F32)])
@pytest.mark.parametrize("act", (B.DC_ACT_NONE, B.DC_ACT_RELU))
@pytest.mark.parametrize("shape", NOT_FINITE_SHAPES)
def test_slopes_where_a_group_is_not_a_number(shape, act, dtype, grad, layout):
    """act'(z) is 1 without an activation, whatever z is, and z > 0 for the
    ReLU: a group that holds a NaN passes all of grad_y on, or none of it."""
    n, c, h, w, groups = shape
    p = B.NormProblem(n, c, h, w, groups, dtype, layout, act, 1e-5, grad)
    x, gamma, beta, gy = (t.cuda() for t in inputs(p, 31))
    hit = torch.zeros(n, groups, c // groups, h * w, dtype=torch.bool)
    hit[1, 1] = True
    hit = P.layout(p, hit).cuda()
    x2 = x.clone()
    if layout == B.DC_NHWC:
        x2[1, 3, 2, c // groups] = float("nan")
    else:
        x2[1, c // groups, 3, 2] = float("nan")
    _, mean, rstd = B.group_norm(p, x2, gamma, beta)
    assert torch.isnan(mean[1, 1]) and torch.isfinite(mean).sum() == mean.numel() - 1
    clean = B.group_norm_backward(p, x, gamma, beta, *B.group_norm(p, x, gamma, beta)[1:], gy)
    g = B.group_norm_backward(p, x2, gamma, beta, mean, rstd, gy)
    assert torch.isnan(g["grad_x"][hit]).all()
    assert torch.equal(g["grad_x"][~hit], clean["grad_x"][~hit])
    per = c // groups
    assert torch.isnan(g["grad_gamma"][per:2 * per]).all()
    # grad_beta: sums of non-negative terms' worth of at most 96 roundings in a row
    over = (0, 1, 2) if layout == B.DC_NHWC else (0, 2, 3)
    dz = gy.double()
    if act == B.DC_ACT_RELU:
        shape4 = (1, 1, 1, c) if layout == B.DC_NHWC else (1, c, 1, 1)
        m4, r4 = (P.layout(p, t.double()[:, :, None, None].expand(n, groups, per, h * w)) for t in (mean, rstd))
        z = (x2.double() - m4) * r4 * gamma.double().view(shape4) + beta.double().view(shape4)
        near_kink = (z.abs() <= 8 * P.U * (1 + z.abs()))
        slack = (dz.abs() * near_kink).sum(over)
        dz = dz * (z > 0)
    else:
        slack = 0
    bound = 96 * P.U * dz.abs().sum(over) + slack + 1e-38
    assert ((g["grad_beta"].double() - dz.sum(over)).abs() <= bound).all()


@on_gpu
@pytest.mark.parametrize("layout", (B.DC_NCHW, B.DC_NHWC))
@pytest.mark.parametrize("shape", NOT_FINITE_SHAPES)
def test_a_channel_at_minus_infinity_passes_its_gradient_without_an_activation(shape, layout):
    n, c, h, w, groups = shape
    p = B.NormProblem(n, c, h, w, groups, B.DC_F32, layout, B.DC_ACT_NONE)
    x, gamma, beta, gy = (t.cuda() for t in inputs(p, 32))
    y, mean, rstd = B.group_norm(p, x, gamma, beta)
    want = B.group_norm_backward(p, x, gamma, beta, mean, rstd, gy)
    beta[1] = -float("inf")  # (no gradient depends on beta without an activation)
    y = B.group_norm(p, x, gamma, beta)[0]
    cut = y[..., 1] if layout == B.DC_NHWC else y[:, 1]
    assert (cut == -float("inf")).all()
    g = B.group_norm_backward(p, x, gamma, beta, mean, rstd, gy)
    assert all(torch.equal(g[k], want[k]) for k in want)


@on_gpu
@pytest.mark.parametrize("layout", (B.DC_NCHW, B.DC_NHWC))
@pytest.mark.parametrize("value", (float("nan"), float("inf"), -float("inf")))
@pytest.mark.parametrize("shape", NOT_FINITE_SHAPES)
def test_statistics_of_a_group_that_is_not_finite_are_nan(shape, value, layout):
    n, c, h, w, groups = shape
    p = B.NormProblem(n, c, h, w, groups, B.DC_F32, layout, B.DC_ACT_RELU)
    x = inputs(p, 33)[0].cuda()
    x.view(-1)[0] = value  # of the first image's first group
    y, mean, rstd = B.group_norm(p, x)
    bad = torch.zeros(n, groups, dtype=torch.bool, device="cuda")
    bad[0, 0] = True
    assert torch.equal(torch.isnan(mean), bad) and torch.equal(torch.isnan(rstd), bad)
    assert int(torch.isnan(y).sum()) == y.numel() // (n * groups)
