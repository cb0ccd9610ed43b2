"""Group norm's two-launch kernels (units that no cluster of blocks holds, and
backward passes whose blocks do not run at once) against the 64-bit plain form:
every type, layout, activation, whole-vector and odd rows, in place, several
turns of images (GPU)."""
import pytest
import torch

import norm_plain as P
from deformable_convolution_gb300 import binding as B

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

ACTS = (B.DC_ACT_NONE, B.DC_ACT_RELU, B.DC_ACT_SILU, B.DC_ACT_GELU)
TYPES = ((B.DC_F32, B.DC_F32), (B.DC_BF16, B.DC_BF16), (B.DC_BF16, B.DC_F32))
# The plain form's bounds allow 64 roundings in a row.  Here a lane adds up to
# 64 terms (16 vectors of 4 pairs), or a block's 85 rows of pixels one after
# the other, then 5 shuffles, 13 images' parts and 5 shuffles: 112 at most
CHAIN = 2.0


def inputs(p, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)
    gdt = torch.bfloat16 if p.grad_dtype == B.DC_BF16 else torch.float32
    return ((randn(*p.shape) + 0.5).to(p.torch_dtype), 1 + 0.2 * randn(p.c), 0.2 * randn(p.c), randn(*p.shape).to(gdt))


def within(got, want, bound, what):
    bad = ~((got.double() - want).abs() <= CHAIN * bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} beyond the bound"


def launches(call):
    """The call's kernels by name, and its result."""
    B.kernel_timing(True)
    try:
        result = call()
        return {name for name, _ in B.kernel_times()}, result
    finally:
        B.kernel_timing(False)


def check(p, seed, forward_two=True):
    x, gamma, beta, gy = inputs(p, seed)
    names, (y, mean, rstd) = launches(lambda: B.group_norm(p, x, gamma, beta))
    assert names == ({"norm_stats", "norm_apply"} if forward_two else {"norm_fwd"})
    f = P.forward(p, x, gamma, beta)
    for got, k in ((mean, "mean"), (rstd, "rstd"), (y, "y")):
        within(got, f[k], f["d_" + k], k)
    del f
    names, g = launches(lambda: B.group_norm_backward(p, x, gamma, beta, mean, rstd, gy))
    assert names == {"norm_sums", "norm_grads", "norm_params"}
    w = P.backward(p, x, gamma, beta, mean, rstd, gy)
    for k in ("grad_x", "grad_gamma", "grad_beta"):
        within(g[k], w[k], w["d_" + k], k)


@pytest.mark.parametrize("layout", (B.DC_NCHW, B.DC_NHWC))
@pytest.mark.parametrize("dtype,grad", TYPES)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("shape", [(1, 8, 401, 333, 1), (2, 16, 400, 336, 2)])
def test_every_activation_and_type(shape, act, dtype, grad, layout):
    n, c, h, w, groups = shape
    check(B.NormProblem(n, c, h, w, groups, dtype, layout, act, 1e-5, grad), 1 + act)


SHAPES = [  # n, c, h, w, groups, [n][c][h][w] forwards (bf16) in two launches
    (1, 4096, 20, 21, 1, True),     # many rows of some vectors, the last one short
    (1, 40000, 5, 5, 1, True),      # rows of three or four vectors, eight to a warp; slices that share a group
    (5, 16, 600, 600, 2, True),     # several turns of images
    (2, 320, 200, 201, 32, False),  # ten channels to a group: vectors of two groups, the last slice narrower
    (2, 12, 401, 333, 4, False),    # three channels to a group, 8-byte vectors
    (2, 20, 401, 333, 2, True),     # ten channels to a group, 8-byte vectors
    (1, 33, 301, 303, 3, True),     # one channel to a vector
]


@pytest.mark.parametrize("layout", (B.DC_NCHW, B.DC_NHWC))
@pytest.mark.parametrize("dtype,grad", TYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_shapes(shape, dtype, grad, layout):
    n, c, h, w, groups, two = shape
    act = ACTS[(c + h + dtype + grad + layout) % 4]
    check(B.NormProblem(n, c, h, w, groups, dtype, layout, act, 1e-5, grad), c,
          two or layout == B.DC_NHWC or dtype == B.DC_F32)


@pytest.mark.parametrize("layout", (B.DC_NCHW, B.DC_NHWC))
@pytest.mark.parametrize("act,grad", [(B.DC_ACT_SILU, B.DC_BF16), (B.DC_ACT_SILU, B.DC_F32), (B.DC_ACT_RELU, B.DC_F32)])
def test_backwards_whose_blocks_do_not_run_at_once(act, grad, layout):
    check(B.NormProblem(16, 256, 56, 56, 32, B.DC_BF16, layout, act, 1e-5, grad), 3, forward_two=False)


@pytest.mark.parametrize("layout", (B.DC_NCHW, B.DC_NHWC))
@pytest.mark.parametrize("dtype", (B.DC_F32, B.DC_BF16))
@pytest.mark.parametrize("shape", [(2, 16, 401, 333, 2), (2, 16, 400, 336, 2), (2, 20, 401, 333, 2), (1, 33, 301, 303, 3)])
def test_in_place_on_a_side_stream_and_the_same_bits_twice(shape, dtype, layout):
    n, c, h, w, groups = shape
    p = B.NormProblem(n, c, h, w, groups, dtype, layout, B.DC_ACT_SILU, 1e-5, dtype)
    x, gamma, beta, gy = inputs(p, 9)
    y, mean, rstd = B.group_norm(p, x, gamma, beta)
    g = B.group_norm_backward(p, x, gamma, beta, mean, rstd, gy)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        a, b = x.clone(), gy.clone()
        m2, r2, gg, gb = (torch.empty_like(t) for t in (mean, rstd, gamma, beta))
        B.dc_group_norm_fwd(p, a, gamma, beta, a, m2, r2, B.norm_workspace(p, False))
        B.dc_group_norm_bwd(p, x, gamma, beta, m2, r2, b, b, gg, gb, B.norm_workspace(p, True))
    s.synchronize()
    for u, v in ((a, y), (m2, mean), (r2, rstd), (b, g["grad_x"]), (gg, g["grad_gamma"]), (gb, g["grad_beta"])):
        assert torch.equal(u, v)


@pytest.mark.parametrize("layout", (B.DC_NCHW, B.DC_NHWC))
def test_a_mean_far_above_the_spread(layout):
    p = B.NormProblem(1, 8, 401, 333, 1, B.DC_F32, layout, B.DC_ACT_NONE)
    x, gamma, beta, gy = inputs(p, 6)
    x += 4000.0
    x.view(-1)[:: x.numel() // 2] = 3900.0
    y, mean, rstd = B.group_norm(p, x, gamma, beta)
    f = P.forward(p, x, gamma, beta)
    for got, k in ((mean, "mean"), (rstd, "rstd"), (y, "y")):
        within(got, f[k], f["d_" + k], k)


@pytest.mark.parametrize("layout", (B.DC_NCHW, B.DC_NHWC))
def test_what_lies_around_the_tensors_is_neither_read_nor_written(layout):
    """Odd rows hang over their ends in vectors: the tensors lie between NaNs."""
    p = B.NormProblem(1, 8, 401, 333, 1, B.DC_BF16, layout, B.DC_ACT_GELU, 1e-5, B.DC_BF16)
    x, gamma, beta, gy = inputs(p, 5)
    n, pad = x.numel(), 64

    def framed(t):
        buf = torch.full((n + 2 * pad,), float("nan"), dtype=t.dtype, device="cuda")
        buf[pad:pad + n] = t.reshape(-1)
        return buf, buf[pad:pad + n].view(p.shape)
    (bx, fx), (bg, fg) = framed(x), framed(gy)
    (by, fy), (bo, fo) = framed(torch.zeros_like(x)), framed(torch.zeros_like(x))
    mean, rstd = (torch.empty(p.stat_shape, device="cuda") for _ in range(2))
    gg, gb = torch.empty_like(gamma), torch.empty_like(beta)
    B.dc_group_norm_fwd(p, fx, gamma, beta, fy, mean, rstd, B.norm_workspace(p, False))
    B.dc_group_norm_bwd(p, fx, gamma, beta, mean, rstd, fg, fo, gg, gb, B.norm_workspace(p, True))
    y, m2, r2 = B.group_norm(p, x, gamma, beta)
    g = B.group_norm_backward(p, x, gamma, beta, m2, r2, gy)
    for u, v in ((fy, y), (mean, m2), (rstd, r2), (fo, g["grad_x"]), (gg, g["grad_gamma"]), (gb, g["grad_beta"])):
        assert torch.equal(u, v)
    for buf in (bx, bg, by, bo):
        assert torch.isnan(buf[:pad]).all() and torch.isnan(buf[pad + n:]).all()
