"""Pointwise layers at the ends of their ranges: sizes that a layer takes, and
which of its two forward passes it takes them with."""
from deformable_convolution_gb300 import binding as B
from deformable_convolution_gb300 import fp8


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
