"""Pointwise layers at the ends of their ranges: sizes that a layer takes, and
which of its two forward passes it takes them with."""
import pytest
import torch

from deformable_convolution_gb300 import binding as B
from deformable_convolution_gb300 import fp8


def on_gpu(f):
    f = pytest.mark.gpu(f)
    return pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")(f)


MANY = (17, 8, 8, 1024, 1024)  # 17.8 million pixels: more than the 2^24 rows of a matrix of codes


@pytest.mark.parametrize("layout", (B.DC_NCHW, B.DC_NHWC))
def test_a_layer_that_keeps_no_codes_takes_more_pixels_than_codes_have_rows(layout):
    layer = fp8.Pointwise(*MANY, B.DC_BF16, layout, training=False, device="cpu")
    assert layer.x.codes is None and layer.x.codes_t is None and layer._ws.numel() <= 1


def test_more_pixels_than_codes_have_rows_are_refused_where_codes_are_kept():
    with pytest.raises(B.DcError):
        fp8.Pointwise(*MANY, B.DC_BF16, B.DC_NHWC, training=True, device="cpu")
    with pytest.raises(B.DcError):
        fp8.Pointwise(*MANY, B.DC_F32, B.DC_NHWC, training=False, device="cpu")
    # channels first every image has codes of its own
    fp8.Pointwise(2, 8, 8, 64, 64, B.DC_BF16, B.DC_NCHW, training=True, device="cpu")


@pytest.mark.parametrize("layout", (B.DC_NCHW, B.DC_NHWC))
def test_deep_inputs_of_small_maps_take_two_launches(layout):
    """One launch gives a tile of 128 pixels its whole reduction: 8 x 14 x 14 pixels
    of 2048 channels took 27 to 46 us so, 10 to 15 us in two."""
    def one(n, c_in, h, w):
        return fp8.Pointwise(n, c_in, 64, h, w, B.DC_BF16, layout, training=False, device="cpu")._one is not None
    assert not one(8, 2048, 14, 14) and not one(1, 1024, 7, 7) and not one(8, 512, 28, 28)
    assert one(8, 256, 14, 14) and one(1, 64, 7, 7) and one(16, 256, 100, 168) and one(16, 1024, 100, 168)


@on_gpu
@pytest.mark.parametrize("layout", (B.DC_NCHW, B.DC_NHWC))
@pytest.mark.parametrize("size", [(3, 520, 64, 14, 14), (1, 1030, 128, 7, 7), (2, 264, 8, 120, 130)])
def test_either_way_gives_the_same(size, layout):
    n, c_in, c_out, h, w = size
    gen = torch.Generator(device="cuda").manual_seed(0)
    layer = fp8.Pointwise(*size, B.DC_BF16, layout, training=False)
    wt, x = (torch.empty(s, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
             for s in ((c_out, c_in), layer.x_shape))
    layer.load(wt)
    y = torch.empty(layer.y_shape, dtype=torch.bfloat16, device="cuda")
    p = B.DcFp8Layer(n, h * w, c_in, c_out, layout)
    assert B.lib().dc_fp8_pointwise(p, x.data_ptr(), layer.weight.codes.data_ptr(), layer.weight.scales.data_ptr(),
                                    y.data_ptr(), torch.cuda.current_stream().cuda_stream) == B.DC_OK
    kept = fp8.Pointwise(*size, B.DC_BF16, layout, training=True)
    kept.load(wt)
    assert torch.equal(layer.forward(x), y) and torch.equal(kept.forward(x), y) and y.any()


@pytest.mark.parametrize("training", (True, False))
@pytest.mark.parametrize("layout", (B.DC_NCHW, B.DC_NHWC))
@pytest.mark.parametrize("size", [(-1, 8, 8, 4, 4), (1, 0, 8, 4, 4), (1, 8, 0, 4, 4), (1, 8, 8, 0, 4), (1, 8, 8, 4, -1)])
def test_sizes_that_are_none_are_refused_where_the_layer_is_made(size, layout, training):
    with pytest.raises(B.DcError):
        fp8.Pointwise(*size, B.DC_BF16, layout, training, device="cpu")


@on_gpu
@pytest.mark.parametrize("layout", (B.DC_NCHW, B.DC_NHWC))
def test_more_pixels_than_codes_have_rows(layout):
    """The last image as a layer of its own gives it."""
    n = MANY[0]
    gen = torch.Generator(device="cuda").manual_seed(0)
    layer, one = (fp8.Pointwise(k, *MANY[1:], B.DC_BF16, layout, training=False) for k in (n, 1))
    w = torch.empty(8, 8, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    layer.load(w), one.load(w)
    x = torch.empty(layer.x_shape, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    y = layer.forward(x)
    for i in (0, n // 2, n - 1):
        assert torch.equal(y[i:i + 1], one.forward(x[i:i + 1])) and y[i].any()


def test_reductions_of_more_than_a_run():
    """They take workspace, and the one-launch forward refuses them."""
    long = B.FP8_RUN + 1
    assert B.dc_fp8_matmul_workspace_size(B.Fp8Product(3, 7, 9, B.FP8_RUN)) == 0
    assert B.dc_fp8_matmul_workspace_size(B.Fp8Product(3, 7, 9, long)) == 3 * 7 * 12 * 4
    p, w = B.DcFp8Product(3, 7, 9, long), 0x10000
    assert B.lib().dc_fp8_matmul(p, w, w, w, w, w, None, 0, None) == B.DC_ERR_WORKSPACE
    assert B.lib().dc_fp8_matmul(p, w, w, w, w, w, w, 3 * 7 * 12 * 4 - 1, None) == B.DC_ERR_WORKSPACE
    assert B.lib().dc_fp8_pointwise(B.DcFp8Layer(1, 8, long, 8, B.DC_NCHW), w, w, w, w, None) == B.DC_ERR_UNSUPPORTED
    for layout in (B.DC_NCHW, B.DC_NHWC):
        assert fp8.Pointwise(1, long, 8, 2, 4, B.DC_BF16, layout, training=False, device="cpu")._one is None
        # products whose sums share the layer's workspace do not run side by side
        assert fp8.Pointwise(1, 8, long, 2, 4, B.DC_BF16, layout, device="cpu")._gw.beside == 0
        assert fp8.Pointwise(1, 8, 8, 2, 4, B.DC_BF16, layout, device="cpu")._gw.beside == 1
