"""Matrices in 8 bits and their products: refusals (CPU), and the kernels
against plain forms in 64 bits (GPU)."""
import ctypes

import pytest
import torch

import matrix_plain as P
from deformable_convolution_gb300 import binding as B
from deformable_convolution_gb300 import fp8


def on_gpu(f):
    f = pytest.mark.gpu(f)
    return pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")(f)


F32, BF16 = torch.float32, torch.bfloat16
KIND = {B.DC_F32: F32, B.DC_BF16: BF16}
INVALID, UNSUPPORTED, WORKSPACE = B.DC_ERR_INVALID_ARG, B.DC_ERR_UNSUPPORTED, B.DC_ERR_WORKSPACE


# ---------------------------------------------------------------- refusals

def quantize_status(codes=0x1000, scales=0x2000, codes_t=0x3000, scales_t=0x4000, x=0x5000, **kw):
    d = dict(batch=1, rows=8, cols=8, dtype=B.DC_BF16, format=B.DC_E4M3, square=0)
    d.update(kw)
    return B.lib().dc_fp8_quantize(ctypes.byref(B.DcFp8Problem(**d)), x, codes, scales, codes_t, scales_t, None)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), INVALID), (dict(rows=0), INVALID), (dict(cols=-3), INVALID), (dict(dtype=2), INVALID),
    (dict(format=2), INVALID), (dict(square=2), INVALID), (dict(x=None), INVALID), (dict(scales=None), INVALID),
    (dict(codes_t=None), INVALID), (dict(codes=None, scales=None, codes_t=None, scales_t=None), INVALID),
    (dict(rows=(1 << 24) + 1), UNSUPPORTED), (dict(batch=65536), UNSUPPORTED),
    (dict(batch=1024, rows=1 << 24, cols=1 << 10), UNSUPPORTED), (dict(codes=0x1008), UNSUPPORTED),
    (dict(scales_t=0x4001), UNSUPPORTED), (dict(x=0x5001), UNSUPPORTED), (dict(dtype=B.DC_F32, x=0x5002), UNSUPPORTED),
    (dict(batch=0, x=None), B.DC_OK),
])
def test_quantize_checks_its_arguments(kw, status):
    assert quantize_status(**kw) == status


def test_other_calls_check_their_arguments():
    L, vp = B.lib(), ctypes.c_void_p
    p = B.Fp8Problem(1, 8, 8)
    assert L.dc_fp8_quantize(None, vp(0x1000), vp(0x1000), vp(0x1000), None, None, None) == INVALID
    assert L.dc_fp8_sizes(p, 0, None, None) == INVALID
    assert L.dc_fp8_values(p, 0, None, vp(0x1000), vp(0x2000), None) == INVALID
    assert L.dc_fp8_values(p, 0, vp(0x1000), vp(0x1000), vp(0x2002), None) == UNSUPPORTED
    assert L.dc_fp8_values(p, 0, vp(0x1008), vp(0x1000), vp(0x2000), None) == UNSUPPORTED
    with pytest.raises(ValueError):
        B.dc_fp8_quantize(p, torch.zeros(1, 8, 8))
    with pytest.raises(B.DcError):
        B.dc_fp8_sizes(B.Fp8Problem(1, 0, 8), False)


def test_sizes():
    assert B.dc_fp8_sizes(B.Fp8Problem(3, 130, 520), False) == (3 * 130 * 640, 3 * 2 * 2 * 512)
    assert B.dc_fp8_sizes(B.Fp8Problem(3, 130, 520), True) == (3 * 520 * 256, 3 * 5 * 1 * 512)
    assert B.dc_fp8_sizes(B.Fp8Problem(0, 1, 1), False) == (0, 0)


def product_status(a=0x1000, sa=0x2000, b=0x3000, sb=0x4000, d=0x5000, ws=None, nbytes=0, **kw):
    q = dict(batch=1, m=8, n=8, k=8, a_format=0, b_format=0, a_shared=0, b_shared=0, sum=0, out=B.DC_F32)
    q.update(kw)
    return B.lib().dc_fp8_matmul(ctypes.byref(B.DcFp8Product(**q)), a, sa, b, sb, d, ws, nbytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), INVALID), (dict(m=0), INVALID), (dict(n=0), INVALID), (dict(k=-1), INVALID),
    (dict(a_format=2), INVALID), (dict(b_format=-1), INVALID), (dict(a_shared=2), INVALID), (dict(sum=-1), INVALID),
    (dict(out=2), INVALID), (dict(a=None), INVALID), (dict(sb=None), INVALID), (dict(d=None), INVALID),
    (dict(m=(1 << 24) + 1), UNSUPPORTED), (dict(batch=65536), UNSUPPORTED), (dict(a=0x1008), UNSUPPORTED),
    (dict(m=1 << 20, k=1 << 19), UNSUPPORTED), (dict(n=1 << 24, k=1 << 15), UNSUPPORTED),
    (dict(m=1 << 20, n=1 << 18), UNSUPPORTED), (dict(batch=60000, m=1 << 18, n=8192), UNSUPPORTED),
    (dict(batch=60000, k=1 << 23, sum=1), UNSUPPORTED),
    (dict(sa=0x2004), UNSUPPORTED), (dict(d=0x5002), UNSUPPORTED), (dict(d=0x5001, out=B.DC_BF16), UNSUPPORTED),
    (dict(ws=0x6008), UNSUPPORTED), (dict(batch=0), B.DC_OK),
])
def test_matmul_checks_its_arguments(kw, status):
    assert product_status(**kw) == status


def test_matmul_beside_is_a_flag():
    for beside, status in ((2, INVALID), (-1, INVALID), (0, B.DC_OK), (1, B.DC_OK)):
        q, out = B.DcFp8Product(1, 64, 64, 128, 0, 0, 0, 0, 0, B.DC_F32, beside), ctypes.c_size_t(0)
        assert B.lib().dc_fp8_matmul_workspace_size(ctypes.byref(q), ctypes.byref(out)) == status


def test_matmul_checks_its_workspace():
    p = B.Fp8Product(64, 64, 64, 1 << 16, sum=1)
    need = B.dc_fp8_matmul_workspace_size(p)
    if need:
        kw = dict(batch=64, m=64, n=64, k=1 << 16, sum=1)
        assert product_status(ws=0x6000, nbytes=need - 1, **kw) == WORKSPACE
        assert product_status(**kw) == WORKSPACE


def pointwise_status(x=0x1000, w=0x2000, sw=0x3000, y=0x4000, **kw):
    d = dict(n=1, pixels=8, c_in=8, c_out=8, layout=B.DC_NCHW)
    d.update(kw)
    return B.lib().dc_fp8_pointwise(ctypes.byref(B.DcFp8Layer(**d)), x, w, sw, y, None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), INVALID), (dict(pixels=0), INVALID), (dict(c_in=0), INVALID), (dict(c_out=-1), INVALID),
    (dict(layout=2), INVALID), (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(sw=None), INVALID),
    (dict(y=None), INVALID), (dict(c_out=257), UNSUPPORTED), (dict(c_in=(1 << 20) + 1), UNSUPPORTED),
    (dict(n=1 << 20, pixels=2048), UNSUPPORTED), (dict(x=0x1001), UNSUPPORTED), (dict(w=0x2008), UNSUPPORTED),
    (dict(sw=0x3004), UNSUPPORTED), (dict(y=0x4001), UNSUPPORTED), (dict(n=0, x=None), B.DC_OK),
])
def test_pointwise_checks_its_arguments(kw, status):
    assert pointwise_status(**kw) == status
    assert B.lib().dc_fp8_pointwise(None, 0x1000, 0x2000, 0x3000, 0x4000, None) == INVALID


def test_layer_checks_its_arguments():
    with pytest.raises(B.DcError):
        fp8.Pointwise(1, 0, 4, 4, 4, device="cpu")
    layer = fp8.Pointwise(1, 8, 4, 4, 4, training=False, device="cpu")
    with pytest.raises(ValueError):
        layer.backward(torch.zeros(1, 4, 4, 4))
    with pytest.raises(ValueError):
        layer.forward(torch.zeros(1, 8, 4, 4))  # no weight yet
    layer = fp8.Pointwise(1, 8, 4, 4, 4, device="cpu")
    with pytest.raises(ValueError):
        layer.backward(torch.zeros(1, 4, 4, 4))  # no forward yet
    with pytest.raises(ValueError):
        layer.load(torch.zeros(8, 4))


# ---------------------------------------------------------------- codes

def values(shape, kind, seed, spread=3.0):
    """Rows and columns of very different sizes."""
    gen = torch.Generator().manual_seed(seed)
    t = torch.randn(shape, generator=gen)
    t = t * torch.exp(spread * torch.randn(shape[:2] + (1,), generator=gen))
    t = t * torch.exp(spread * torch.randn(shape[:1] + (1,) + shape[2:], generator=gen))
    return t.to(KIND[kind])


def scale_bytes(p, scales, transposed):
    """The scale byte of each element, by the documented layout."""
    r, c = (p.cols, p.rows) if transposed else (p.rows, p.cols)
    runs = -(-c // 128)
    i, row, col = torch.meshgrid(*(torch.arange(n) for n in (p.batch, r, c)), indexing="ij")
    k = col // 128
    at = ((i * -(-r // 128) + row // 128) * -(-runs // 4) + k // 4) * 512 + row % 32 * 16 + row % 128 // 32 * 4 + k % 4
    return scales.cpu()[at]


def check_codes(p, x):
    """Codes, scales and padding of both orientations of x."""
    q = fp8.Quantized(p, True, True)
    for t in (q.codes, q.codes_t):
        t.fill_(0xAA)
    q.load(x.cuda())
    for transposed in (False, True):
        v = x.transpose(1, 2) if transposed else x
        want, byte = P.quantize(v, p.format, p.square)
        got = q.values(transposed).cpu().double()
        # what a code stands for is a float32 number, but for 2^128, which the largest float32 values round to:
        # 1.99..9 * 2^127 has the scale 2^120 (2^113) and the code 256 (2^15)
        want = want.float().double()
        # every code and scale is determined: the values are equal, NaN in the same places
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(torch.nan_to_num(got, posinf=1e300), torch.nan_to_num(want, posinf=1e300))
        assert torch.equal(scale_bytes(p, q.scales_t if transposed else q.scales, transposed), byte)
        codes = (q.codes_t if transposed else q.codes).cpu()
        # the columns past the last are zero, but in a block of NaN
        assert not codes[..., v.shape[2]:][byte[..., -1] != 255].any()
    # one orientation alone gives the same
    for transposed in (False, True):
        one = fp8.Quantized(p, not transposed, transposed)
        one.load(x.cuda())
        a, b = (one.codes_t, q.codes_t) if transposed else (one.codes, q.codes)
        assert torch.equal(a, b)


@on_gpu
@pytest.mark.parametrize("square", (0, 1))
@pytest.mark.parametrize("fmt", (B.DC_E4M3, B.DC_E5M2))
@pytest.mark.parametrize("kind", (B.DC_F32, B.DC_BF16))
@pytest.mark.parametrize("shape", [(1, 1, 1), (2, 3, 257), (1, 128, 128), (3, 130, 72), (1, 257, 1000), (2, 64, 49)])
def test_codes_are_exact(shape, kind, fmt, square):
    check_codes(B.Fp8Problem(*shape, kind, fmt, square), values(shape, kind, sum(shape)))


@on_gpu
@pytest.mark.parametrize("fmt", (B.DC_E4M3, B.DC_E5M2))
def test_codes_at_the_edges(fmt):
    """Blocks whose largest magnitude sits at and beside a scale's border, ties
    half way between codes, zeros, the smallest and largest numbers, and what is
    not finite."""
    most = P.FORMATS[fmt][2]
    x = torch.zeros(1, 24, 256)
    gen = torch.Generator().manual_seed(0)
    x[0, :, :] = torch.randint(-2048, 2049, (24, 256), generator=gen).float() / 16  # many ties
    x[0, 0] = 0.0
    for r, top in enumerate((most, most * (1 + 2.0 ** -20), most * (1 - 2.0 ** -20), most * 2.0 ** -40, most * 2.0 ** 30,
                             1e-45, 3e-38, 2.0 ** -126, 3.4028234663852886e38, 2.0 ** 120 * most / 512)):
        x[0, r + 1] *= top / 256
        x[0, r + 1, 17] = top
    x[0, 12, 3] = float("inf")
    x[0, 13, 200] = float("nan")
    x[0, 14, 130] = -float("inf")
    x[0, 15] = -0.0
    check_codes(B.Fp8Problem(1, 24, 256, B.DC_F32, fmt, 0), x)
    check_codes(B.Fp8Problem(1, 24, 256, B.DC_F32, fmt, 1), x[:, :, :])
    check_codes(B.Fp8Problem(1, 8, 256, B.DC_F32, fmt, 1), x[:, :8].contiguous())


@on_gpu
def test_values_that_start_off_a_vector():
    """x needs only its element's alignment."""
    for kind, off in ((B.DC_BF16, 1), (B.DC_F32, 3)):
        flat = values((1, 1, 140 * 136 + 8), kind, 4).flatten()
        x = flat[off:off + 140 * 136].view(1, 140, 136)
        p = B.Fp8Problem(1, 140, 136, kind)
        q = fp8.Quantized(p, True, True)
        q.load(flat.cuda()[off:off + 140 * 136].view(1, 140, 136))
        assert torch.equal(q.values().cpu().double(), P.quantize(x, p.format, 0)[0])
        assert torch.equal(q.values(True).cpu().double(), P.quantize(x.transpose(1, 2), p.format, 0)[0])


# ---------------------------------------------------------------- products

def operands(p, seed):
    gen = torch.Generator().manual_seed(seed)
    got = []
    for shared, rows, fmt in ((p.a_shared, p.m, p.a_format), (p.b_shared, p.n, p.b_format)):
        shape = (1 if shared else p.batch, rows, p.k)
        x = torch.randn(shape, generator=gen) * torch.exp(torch.randn(shape[:2] + (1,), generator=gen))
        q = fp8.Quantized(B.Fp8Problem(*shape, B.DC_F32, fmt))
        q.load(x.cuda())
        got.append(q)
    return got


def check_product(p, seed=0):
    a, b = operands(p, seed)
    ws = torch.empty(max(1, B.dc_fp8_matmul_workspace_size(p)), dtype=torch.uint8, device="cuda")
    count = 1
    for n in p.shape:
        count *= n
    # guards on both sides of D
    room = torch.full((count + 64,), 7.0, dtype=p.torch_dtype, device="cuda")
    d = room[32:32 + count].view(p.shape)
    B.dc_fp8_matmul(p, a.codes, a.scales, b.codes, b.scales, d, ws)
    av, bv = a.values().double(), b.values().double()
    want, size = av @ bv.transpose(1, 2), av.abs() @ bv.abs().transpose(1, 2)
    depth = p.k
    if p.sum:
        rep = 1 if not (p.a_shared and p.b_shared) else p.batch
        want, size, depth = want.sum(0) * rep, size.sum(0) * rep, p.k * p.batch
    # products are exact; `depth` float32 additions of terms whose magnitudes sum to `size` are off by at most
    # half a step each (truncated ones by a whole one) of a partial sum no larger than `size`
    tol = size * (depth * 2.0 ** -23)
    if p.out == B.DC_BF16:
        tol = tol + want.abs() * 2.0 ** -8
    assert ((d.double() - want).abs() <= tol).all()
    # and in the middle: errors of that many random roundings, the root of the bound's sum, four times over
    rms = (size * depth ** 0.5 * 2.0 ** -23).square().mean().sqrt()
    if p.out == B.DC_BF16:
        rms = rms + want.square().mean().sqrt() * 2.0 ** -8
    assert (d.double() - want).square().mean().sqrt() <= 4 * rms
    assert (room[:32] == 7).all() and (room[32 + count:] == 7).all()
    again = torch.empty_like(d)
    B.dc_fp8_matmul(p, a.codes, a.scales, b.codes, b.scales, again, ws)
    assert torch.equal(d, again)
    return d


SIZES = [(1, 1, 1, 1), (1, 128, 128, 128), (2, 130, 70, 200), (1, 257, 129, 513), (3, 64, 1247, 200), (1, 300, 300, 1),
         (2, 1, 333, 1030), (2, 333, 1, 1030), (1, 512, 384, 2048), (5, 200, 49, 640),
         (40, 300, 500, 700), (90, 257, 129, 130), (3, 2500, 2100, 384)]  # enough tiles for wide ones, several to a pair


@on_gpu
@pytest.mark.parametrize("out", (B.DC_F32, B.DC_BF16))
@pytest.mark.parametrize("size", SIZES)
def test_products(size, out):
    check_product(B.Fp8Product(*size, out=out))


@on_gpu
@pytest.mark.parametrize("formats", [(0, 1), (1, 0), (1, 1)])
def test_products_of_both_formats(formats):
    check_product(B.Fp8Product(2, 200, 136, 300, *formats, out=B.DC_F32))


@on_gpu
@pytest.mark.parametrize("out", (B.DC_F32, B.DC_BF16))
@pytest.mark.parametrize("shared", [(1, 0), (0, 1), (1, 1)])
def test_products_with_a_shared_factor(shared, out):
    check_product(B.Fp8Product(3, 72, 200, 260, 0, 0, *shared, 0, out))
    check_product(B.Fp8Product(3, 72, 200, 260, 0, 0, *shared, 1, out))


@on_gpu
@pytest.mark.parametrize("size", [(1, 64, 64, 4000), (8, 256, 256, 3136), (7, 200, 328, 1247), (2, 130, 17, 30000),
                                  (300, 16, 24, 90), (1, 2048, 512, 129), (9, 640, 640, 128)])
def test_sums_over_matrices(size):
    check_product(B.Fp8Product(*size, sum=1, out=B.DC_F32))
    check_product(B.Fp8Product(*size, sum=1, out=B.DC_BF16))


@on_gpu
def test_empty_products():
    p = B.Fp8Product(2, 3, 5, 0, out=B.DC_F32)
    d = torch.ones(2, 3, 5, device="cuda")
    empty = torch.empty(0, dtype=torch.uint8, device="cuda")
    assert B.lib().dc_fp8_matmul(p, None, None, None, None, d.data_ptr(), None, 0,
                                 torch.cuda.current_stream().cuda_stream) == B.DC_OK
    assert not d.any()
    p = B.Fp8Product(0, 3, 5, 8, sum=1, out=B.DC_F32)
    d = torch.ones(3, 5, device="cuda")
    B.dc_fp8_matmul(p, torch.empty(0, 3, 128, dtype=torch.uint8, device="cuda"), empty,
                    torch.empty(0, 5, 128, dtype=torch.uint8, device="cuda"), empty, d)
    assert not d.any()


@on_gpu
def test_what_is_not_finite_stays_in_its_rows():
    p = B.Fp8Product(1, 200, 150, 300, out=B.DC_F32)
    x, y = torch.ones(1, 200, 300), torch.ones(1, 150, 300)
    x[0, 5, 130] = float("nan")
    x[0, 131, 0] = float("inf")
    y[0, 149, 299] = float("-inf")
    a, b = fp8.Quantized(B.Fp8Problem(1, 200, 300, B.DC_F32)), fp8.Quantized(B.Fp8Problem(1, 150, 300, B.DC_F32))
    a.load(x.cuda())
    b.load(y.cuda())
    d = torch.empty(p.shape, device="cuda")
    ws = torch.empty(max(1, B.dc_fp8_matmul_workspace_size(p)), dtype=torch.uint8, device="cuda")
    B.dc_fp8_matmul(p, a.codes, a.scales, b.codes, b.scales, d, ws)
    want = torch.full((200, 150), 300.0)
    want[5] = want[131] = float("nan")
    want[:, 149] = float("nan")
    assert torch.equal(torch.nan_to_num(d[0].cpu(), nan=-1.0), torch.nan_to_num(want, nan=-1.0))


# ---------------------------------------------------------------- the layer

def rows(t, last):
    return t.reshape(1, -1, t.shape[3]) if last else t.flatten(2)


def check_layer(n, ci, co, h, w, dtype, layout, grad_dtype, fmt, seed=0):
    last = layout == B.DC_NHWC
    gen = torch.Generator().manual_seed(seed)

    def maps(c, kind):
        t = torch.randn((n, h, w, c) if last else (n, c, h, w), generator=gen)
        return t.to(KIND[kind])
    x, gy = maps(ci, dtype), maps(co, grad_dtype)
    weight = (torch.randn(co, ci, generator=gen) * (2 / ci) ** 0.5).to(KIND[dtype])
    layer = fp8.Pointwise(n, ci, co, h, w, dtype, layout, True, grad_dtype, fmt)
    layer.load(weight.cuda())
    y = layer.forward(x.cuda())
    gx, gw = layer.backward(gy.cuda())
    plain = fp8.Pointwise(n, ci, co, h, w, dtype, layout, False)
    plain.load(weight.cuda())
    assert torch.equal(plain.forward(x.cuda()), y)
    wq = P.quantize(weight[None], 0, True)[0][0]
    mt = (lambda t: t) if last else (lambda t: t.transpose(1, 2))  # noqa: E731
    xc, gc = (P.quantize(mt(rows(t, last)), f, False)[0] for t, f in ((x, 0), (gy, fmt)))   # runs of channels
    tm = (lambda t: t.transpose(1, 2)) if last else (lambda t: t)  # noqa: E731
    xp, gp = (P.quantize(tm(rows(t, last)), f, False)[0] for t, f in ((x, 0), (gy, fmt)))   # runs of pixels

    def close(got, want, size, depth, half):
        tol = size * (depth * 2.0 ** -23) + want.abs() * half
        assert ((got.cpu().double() - want).abs() <= tol).all()
    half = 2.0 ** -8 if dtype == B.DC_BF16 else 0.0
    close(mt(rows(y, last)), xc @ wq.T, xc.abs() @ wq.abs().T, ci, half)
    close(mt(rows(gx, last)), gc @ wq, gc.abs() @ wq.abs(), co, half)
    depth = n * h * w
    close(gw, (gp @ xp.transpose(1, 2)).sum(0), (gp.abs() @ xp.abs().transpose(1, 2)).sum(0), depth, 0.0)


@on_gpu
@pytest.mark.parametrize("fmt", (B.DC_E4M3, B.DC_E5M2))
@pytest.mark.parametrize("layout", (B.DC_NCHW, B.DC_NHWC))
@pytest.mark.parametrize("kinds", [(B.DC_BF16, B.DC_F32), (B.DC_BF16, B.DC_BF16), (B.DC_F32, B.DC_F32)])
@pytest.mark.parametrize("size", [(1, 16, 16, 1, 1), (2, 200, 72, 5, 31), (3, 64, 256, 12, 12), (1, 130, 8, 40, 40)])
def test_layer(size, kinds, layout, fmt):
    check_layer(*size, kinds[0], layout, kinds[1], fmt)


@on_gpu
@pytest.mark.parametrize("layout", (B.DC_NCHW, B.DC_NHWC))
@pytest.mark.parametrize("size", [(1, 8, 1, 1), (3, 24, 24, 130), (2, 700, 200, 257), (1, 129, 193, 4000), (8, 256, 256, 3136),
                                  (40, 64, 256, 1000), (5, 72, 40, 1247), (2, 1024, 31, 128), (1, 300, 225, 40000)])
def test_one_launch_gives_what_two_give(size, layout):
    """The forward that quantises on the way against codes and product apart, bit
    for bit, with guards around y and a block that is not finite."""
    n, ci, co, pixels = size
    last = layout == B.DC_NHWC
    x = values((n, pixels, ci) if last else (n, ci, pixels), B.DC_BF16, 7, spread=1.0)
    if pixels > 100:
        x[0, 70 if last else 5, 5 if last else 70] = float("nan")
    x = x.cuda()
    gen = torch.Generator().manual_seed(2)
    w = fp8.Quantized(B.Fp8Problem(1, co, ci, B.DC_F32, B.DC_E4M3, 1))
    w.load((torch.randn(co, ci, generator=gen) * ci ** -0.5).cuda())
    q = fp8.Quantized(B.Fp8Problem(n, *x.shape[1:], B.DC_BF16), last, not last)
    q.load(x)
    if last:
        p = B.Fp8Product(n, pixels, co, ci, b_shared=1)
        args = q.codes, q.scales, w.codes, w.scales
    else:
        p = B.Fp8Product(n, co, pixels, ci, a_shared=1)
        args = w.codes, w.scales, q.codes_t, q.scales_t
    want = torch.empty(p.shape, dtype=BF16, device="cuda")
    ws = torch.empty(max(1, B.dc_fp8_matmul_workspace_size(p)), dtype=torch.uint8, device="cuda")
    B.dc_fp8_matmul(p, *args, want, ws)
    for skip in (16, 1):  # y on a vector's boundary, and off it
        room = torch.full((want.numel() + 64,), 7.0, dtype=BF16, device="cuda")
        y = room[skip:skip + want.numel()].view(p.shape)
        B.dc_fp8_pointwise(B.DcFp8Layer(n, pixels, ci, co, layout), x, w.codes, w.scales, y)
        assert torch.equal(torch.nan_to_num(y, nan=-1e30), torch.nan_to_num(want, nan=-1e30))
        assert torch.isnan(want).any() or pixels <= 100
        assert (room[:skip] == 7).all() and (room[skip + want.numel():] == 7).all()


@on_gpu
def test_one_launch_reads_x_off_a_vector():
    flat = values((1, 1, 72 * 131 + 8), B.DC_BF16, 4, spread=1.0).flatten().cuda()
    w = fp8.Quantized(B.Fp8Problem(1, 40, 72, B.DC_F32, B.DC_E4M3, 1))
    w.load(torch.ones(40, 72, device="cuda"))
    for layout in (B.DC_NCHW, B.DC_NHWC):
        shape = (1, 131, 72) if layout == B.DC_NHWC else (1, 72, 131)
        got = []
        for x in (flat[1:1 + 72 * 131].view(shape), flat[1:1 + 72 * 131].clone().view(shape)):
            y = torch.empty((1, 131, 40) if layout == B.DC_NHWC else (1, 40, 131), dtype=BF16, device="cuda")
            B.dc_fp8_pointwise(B.DcFp8Layer(1, 131, 72, 40, layout), x, w.codes, w.scales, y)
            got.append(y)
        assert torch.equal(*got)


@on_gpu
@pytest.mark.parametrize("layout", (B.DC_NCHW, B.DC_NHWC))
def test_gradients_against_differences(layout):
    """Whole numbers up to 7 are codes themselves: the layer is then linear to
    the last bit and its gradients are the differences of sum(y * gy)."""
    n, ci, co, h, w = 2, 20, 12, 3, 5
    last = layout == B.DC_NHWC
    gen = torch.Generator().manual_seed(3)

    def whole(*shape):
        return torch.randint(-4, 5, shape, generator=gen).float().cuda()
    x, gy = (whole(*((n, h, w, c) if last else (n, c, h, w))) for c in (ci, co))
    weight = whole(co, ci)
    layer = fp8.Pointwise(n, ci, co, h, w, B.DC_F32, layout)

    def value(x, weight):
        layer.load(weight)
        return float((layer.forward(x) * gy).sum(dtype=torch.float64))
    base = value(x, weight)
    gx, gw = layer.backward(gy)
    for t, g in ((x, gx), (weight, gw)):
        for i in torch.randint(0, t.numel(), (24,), generator=gen).tolist():
            moved = t.clone()
            moved.view(-1)[i] += 1
            got = value(moved, weight) if t is x else value(x, moved)
            assert got - base == float(g.reshape(-1)[i])


@on_gpu
def test_empty_batch():
    for layout in (B.DC_NCHW, B.DC_NHWC):
        layer = fp8.Pointwise(0, 8, 4, 5, 5, B.DC_F32, layout)
        layer.load(torch.ones(4, 8, device="cuda"))
        y = layer.forward(torch.empty(layer.x_shape, device="cuda"))
        gx, gw = layer.backward(torch.empty(layer.y_shape, device="cuda"), grad_w=torch.ones(4, 8, device="cuda"))
        assert y.shape == layer.y_shape and gx.shape == layer.x_shape and not gw.any()


@on_gpu
def test_layer_on_other_streams_and_in_a_graph():
    """Two layers on two streams at once, and replays of a captured pass with
    other inputs, give what single calls give."""
    args = (4, 256, 192, 20, 24, B.DC_BF16, B.DC_NHWC)
    layers = [fp8.Pointwise(*args) for _ in range(2)]
    gen = torch.Generator().manual_seed(9)
    ws = [torch.randn(192, 256, generator=gen).bfloat16().cuda() for _ in layers]
    xs = [torch.randn(layers[0].x_shape, generator=gen).bfloat16().cuda() for _ in range(4)]
    gs = [torch.randn(layers[0].y_shape, generator=gen).bfloat16().cuda() for _ in range(4)]

    def single(w, x, g):
        a = fp8.Pointwise(*args)
        a.load(w)
        return (a.forward(x), *a.backward(g))
    want = [[single(w, x, g) for x, g in zip(xs, gs)] for w in ws]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    got = [[], []]
    for i in range(4):
        for k, (layer, st) in enumerate(zip(layers, streams)):
            with torch.cuda.stream(st):
                if i == 0:
                    layer.load(ws[k])
                got[k].append((layer.forward(xs[i]), *layer.backward(gs[i])))
    torch.cuda.synchronize()
    for k in range(2):
        for a, b in zip(got[k], want[k]):
            assert all(torch.equal(u, v) for u, v in zip(a, b))
    x, g = xs[0].clone(), gs[0].clone()
    y, gx, gw = (torch.empty_like(t) for t in want[0][0])
    layer = layers[0]
    layer.load(ws[0])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        layer.forward(x, y)
        layer.backward(g, gx, gw)
    for i in (3, 1, 2):
        x.copy_(xs[i])
        g.copy_(gs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip((y, gx, gw), want[0][i]))
