"""Long reductions of 8-bit products: an error that does not grow with the
length of an accumulator.

The tensor cores cut a float32 sum off after each product of 32, always towards
zero, so a sum of one sign loses up to a unit in the last place each time."""
import pytest
import torch

from deformable_convolution_gb300 import binding as B
from deformable_convolution_gb300 import fp8

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

RUN = 64 * 128  # values of k that an accumulator runs over at most


def factor(batch, rows, k, seed, one_sign):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.empty(batch, rows, k, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    q = fp8.Quantized(B.Fp8Problem(batch, rows, k))
    q.load(x.abs_() if one_sign else x)
    return q


def check(p, one_sign):
    a, b = factor(p.batch, p.m, p.k, 1, one_sign), factor(p.batch, p.n, p.k, 2, one_sign)
    ws = torch.empty(max(1, B.dc_fp8_matmul_workspace_size(p)), dtype=torch.uint8, device="cuda")
    count = 1
    for n in p.shape:
        count *= n
    room = torch.full((count + 64,), 7.0, dtype=p.torch_dtype, device="cuda")
    d = room[32:32 + count].view(p.shape)
    for _ in range(2):  # the second call finds the first one's sums in its workspace
        B.dc_fp8_matmul(p, a.codes, a.scales, b.codes, b.scales, d, ws)
    assert (room[:32] == 7).all() and (room[32 + count:] == 7).all()
    av, bv = a.values(), b.values()
    want = torch.zeros(p.batch, p.m, p.n, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(want)
    for i in range(p.batch):
        for c in range(0, p.k, 1 << 16):
            x, y = av[i, :, c:c + (1 << 16)].double(), bv[i, :, c:c + (1 << 16)].double()
            want[i] += x @ y.T
            size[i] += x.abs() @ y.abs().T
    depth = p.k
    if p.sum:
        want, size, depth = want.sum(0), size.sum(0), p.k * p.batch
    # A run: 4 * 64 products of 32, after each of which less than 2^-23 of the sum so far is cut off; the sums so far add up
    # to half of 256 times the run's magnitudes at most: 128 * 2^-23 of these.  The runs' sums: one float32 addition each,
    # off by half a step of 2^-23.  (Images' reductions end in blocks of their own: one run more for the rest.)
    runs = -(-depth // RUN) + 1
    tol = size * (128 * 2.0 ** -23 + runs * 2.0 ** -24)
    if p.out == B.DC_BF16:
        tol = tol + want.abs() * 2.0 ** -8
    assert ((d.double() - want).abs() <= tol).all(), float(((d.double() - want).abs() / size).max())


@pytest.mark.parametrize("one_sign", (True, False))
@pytest.mark.parametrize("k", (1 << 17, 1 << 20))
@pytest.mark.parametrize("size", [(1, 200, 136), (2, 130, 70), (1, 300, 600)])
def test_a_long_side(size, k, one_sign):
    check(B.Fp8Product(*size, k, out=B.DC_F32), one_sign)


def test_a_long_side_of_whole_rows_and_bf16():
    check(B.Fp8Product(1, 256, 512, 1 << 17, out=B.DC_BF16), True)
    check(B.Fp8Product(3, 33, 47, (1 << 17) + 40, out=B.DC_BF16), True)


@pytest.mark.parametrize("size", [(1, 2048, 2048, 1 << 18), (1, 2000, 2051, 200_000), (32, 1000, 2048, 12_544),
                                  (1, 256, 256, 1 << 22), (5, 64, 72, 1 << 19)])
def test_sums_of_many_tiles_and_of_few(size):
    """Tiles that fill the GPU, whose reductions are not split, and few of them."""
    check(B.Fp8Product(*size, sum=1, out=B.DC_F32), True)


def test_a_weights_gradient_of_many_pixels():
    """Activations of one sign (behind a ReLU) and a gradient of one sign."""
    n, c_in, c_out, h, w = 2, 1024, 1024, 300, 500
    layer = fp8.Pointwise(n, c_in, c_out, h, w, B.DC_BF16, B.DC_NHWC)
    gen = torch.Generator(device="cuda").manual_seed(0)
    x, gy = (torch.empty(s, dtype=torch.bfloat16, device="cuda").normal_(generator=gen).abs_()
             for s in (layer.x_shape, layer.y_shape))
    layer.load(torch.ones(c_out, c_in, dtype=torch.bfloat16, device="cuda"))
    layer.forward(x)
    _, gw = layer.backward(gy)
    xv, gv = (q.values(transposed=True)[0] for q in (layer.x, layer.gy))
    want = sum((g.double() @ x.double().T for g, x in zip(gv.split(50_000, 1), xv.split(50_000, 1))),
               torch.zeros(c_out, c_in, dtype=torch.float64, device="cuda"))
    runs = -(-n * h * w // RUN) + 1
    assert ((gw.double() - want).abs() <= want * (128 * 2.0 ** -23 + runs * 2.0 ** -24)).all()


@pytest.mark.parametrize("layout", (B.DC_NCHW, B.DC_NHWC))
def test_more_channels_than_a_run(layout):
    """Both products of the backward pass have sums in the layer's workspace: the
    weight's gradient does not start beside the other one."""
    c_in, c_out = RUN + 300, RUN + 72
    layer = fp8.Pointwise(2, c_in, c_out, 9, 11, B.DC_BF16, layout)
    apart = fp8.Pointwise(2, c_in, c_out, 9, 11, B.DC_BF16, layout)
    gen = torch.Generator(device="cuda").manual_seed(0)
    w, x, gy = (torch.empty(s, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
                for s in ((c_out, c_in), layer.x_shape, layer.y_shape))
    layer.load(w), apart.load(w)
    y = apart.forward(x)
    torch.cuda.synchronize()
    gx, gw = apart.backward(gy)
    torch.cuda.synchronize()
    gw = gw.clone()
    for _ in range(5):
        y2 = layer.forward(x)
        gx2, gw2 = layer.backward(gy)
        assert torch.equal(y, y2) and torch.equal(gx, gx2) and torch.equal(gw, gw2)
    # the input's gradient and the output against 64 bits, on the codes
    last = layout == B.DC_NHWC
    wv = layer.weight.values()[0].double()
    xv = layer.x.values(transposed=not last).double()
    gv = layer.gy.values(transposed=not last).double()
    for got, factor, weight in ((y, xv, wv.T), (gx, gv, wv)):
        got = got.reshape(factor.shape[0], factor.shape[1], -1) if last else got.flatten(2).transpose(1, 2)
        want, size = factor @ weight, factor.abs() @ weight.abs()
        tol = size * (128 * 2.0 ** -23 + 2 * 2.0 ** -24) + want.abs() * 2.0 ** -8
        assert ((got.double() - want).abs() <= tol).all()
