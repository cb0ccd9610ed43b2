"""Pointwise (1 x 1) layers as products of matrices in 8-bit floating point.

Marshalling only: the layer keeps codes, scales and workspaces between its
calls; quantising and products run in the library's kernels.  The codes and
their scales are defined in ``include/deform_conv.h``.
"""
from __future__ import annotations

import torch

from . import binding as B


def _empty(shape, dtype, device, stream):
    """A new tensor for a kernel on ``stream``, whose memory no other stream still writes to."""
    with torch.cuda.stream(stream):  # (None: the current one)
        return torch.empty(shape, dtype=dtype, device=device)


class Quantized:
    """Matrices in 8 bits: codes and scales of ``p`` (an ``Fp8Problem``), and
    of their transposes.  direct, transposed: which of the two are kept."""

    def __init__(self, p: B.Fp8Problem, direct=True, transposed=False, device="cuda"):
        self.p = p

        def pair(shapes):
            return [torch.empty(s, dtype=torch.uint8, device=device) for s in shapes]
        self.codes, self.scales = pair(p.shapes) if direct else (None, None)
        self.codes_t, self.scales_t = pair(p.shapes_t) if transposed else (None, None)

    def load(self, x, stream=None):
        """Quantises x (a tensor of the problem's values, any shape)."""
        B.dc_fp8_quantize(self.p, x.view(self.p.shape), self.codes, self.scales, self.codes_t,
                          self.scales_t, stream)

    def values(self, transposed=False, stream=None):
        """The float32 values that the codes stand for, as a new tensor."""
        codes, scales = (self.codes_t, self.scales_t) if transposed else (self.codes, self.scales)
        shape = (self.p.batch, self.p.cols, self.p.rows) if transposed else self.p.shape
        out = _empty(shape, torch.float32, codes.device, stream)
        B.dc_fp8_values(self.p, codes, scales, out, transposed, stream)
        return out


class Pointwise:
    """y = W x over the channels of every pixel: x [n, c_in, h, w], y
    [n, c_out, h, w] (DC_NHWC: channels last) in ``dtype``, W [c_out, c_in].

    ``load`` quantises the weight (E4M3, a scale for each 128 x 128 block),
    ``forward`` the input (E4M3, a scale for each 128 channels of a pixel, and,
    ``training``, each 128 pixels of a channel for the weight's gradient; else,
    where one launch is faster, on its way into the product),
    ``backward`` the gradient of y (``grad_format``, in ``grad_dtype``) likewise.
    Products are exact and summed in float32 (``dc_fp8_matmul``).  Codes that are
    kept have at most 2^24 rows: channels last that many pixels of all images,
    channels first of one; a forward in one launch takes 2^30 of all.

    The layer keeps the codes of its weight and of the last forward's input,
    and workspaces: its calls belong on one stream, or on streams that wait for
    one another."""

    def __init__(self, n, c_in, c_out, h, w, dtype=B.DC_BF16, layout=B.DC_NCHW, training=True,
                 grad_dtype=None, grad_format=B.DC_E4M3, device="cuda"):
        grad_dtype = dtype if grad_dtype is None else grad_dtype
        last = layout == B.DC_NHWC
        self.training = training
        self.x_shape, self.y_shape = ((n, h, w, c) if last else (n, c, h, w) for c in (c_in, c_out))
        self.w_shape, self.dtype, self.grad_dtype = (c_out, c_in), B._TORCH_DTYPE[dtype], B._TORCH_DTYPE[grad_dtype]
        pixels = max(n, 1) * h * w if last else h * w
        batch, q = min(n, 1) if last else n, B.Fp8Product

        def maps(c, kind, fmt):
            return B.Fp8Problem(batch, pixels, c, kind, fmt) if last else B.Fp8Problem(batch, c, pixels, kind, fmt)
        # codes by channel (runs of channels) and by pixel: direct and transposed, or the other way round
        self.weight = Quantized(B.Fp8Problem(1, c_out, c_in, dtype, B.DC_E4M3, 1), True, training, device)
        # Without a backward pass the input's codes need not be kept, and one launch is faster (in us, one against
        # two): channels last 16 x 100 x 168, 256 -> 256: 57, 75; 4 x 112 x 112, 128 -> 64: 7.8, 10.1; channels first
        # the latter 10.0, 13.0.  Not where rows of y are no whole 16-byte pieces (9 x 22 x 4, 144 -> 71: 13.7, 7.1),
        # and channels first not for many output channels (8 x 56 x 56, 256 -> 256: 16.4, 11.3).  A tile of 128 pixels
        # runs through all of c_in by itself: deep inputs take two launches unless there are tiles for more than one
        # and a half rounds of the 152 SMs (channels last, -> 128: 8 x 14 x 14, 512: 8.9, 6.8, 2048: 26.8, 10.2;
        # 8 x 56 x 56, 1024: 25.4, 20.7; 2 x 100 x 168, 1024: 26.5, 30.7; 8 x 14 x 14, 256: 5.8, 6.3).
        self._one = None
        few = batch * -(-pixels // 128) <= 228
        takes = n >= 0 and h * w > 0 and n * h * w <= 1 << 30 and c_in <= B.FP8_RUN  # (dc_fp8_pointwise)
        if not training and dtype == B.DC_BF16 and takes and not (few and c_in > 256) and \
                (c_out <= 256 and c_out % 8 == 0 if last else c_out <= 128):
            self._one = B.DcFp8Layer(n, h * w, c_in, c_out, layout)
        kept = self._one is None
        self.x = Quantized(maps(c_in, dtype, B.DC_E4M3), kept and (last or training), kept and (not last or training),
                           device)
        e, g = B.DC_E4M3, grad_format
        # products over channels: pixels are the rows of D (channels last) or its columns
        self._fwd = q(batch, pixels, c_out, c_in, b_shared=1, out=dtype) if last else \
            q(batch, c_out, pixels, c_in, a_shared=1, out=dtype)
        products = [self._fwd] if kept else []
        if training:
            self.gy = Quantized(maps(c_out, grad_dtype, g), True, True, device)
            self._gx = q(batch, pixels, c_in, c_out, g, e, b_shared=1, out=dtype) if last else \
                q(batch, c_in, pixels, c_out, e, g, a_shared=1, out=dtype)
            # (beside the product ahead of it: 3 x 29 x 43, 200 -> 328: 17.8 us in place of 21.8; none where that one
            # fills the GPU; not where that one's sums stand in the workspace that both share)
            alone = B.dc_fp8_matmul_workspace_size(self._gx) == 0
            self._gw = q(batch, c_out, c_in, pixels, g, e, sum=1, out=B.DC_F32, beside=int(alone))
            products += [self._gx, self._gw]
        need = max((B.dc_fp8_matmul_workspace_size(p) for p in products), default=0)
        self._ws = torch.empty(max(need, 1), dtype=torch.uint8, device=device)
        # addresses of what the layer keeps, in the order that the calls take them
        self._lib = B.lib()
        w, x = self.weight, self.x

        def addresses(*tensors):
            return tuple(None if t is None else t.data_ptr() for t in tensors)
        self._w = addresses(w.codes, w.scales)
        self._x_to = addresses(x.codes, x.scales, x.codes_t, x.scales_t)
        self._fwd_from = addresses(x.codes, x.scales, w.codes, w.scales) if last else \
            addresses(w.codes, w.scales, x.codes_t, x.scales_t)
        if training:
            g = self.gy
            self._gy_to = addresses(g.codes, g.scales, g.codes_t, g.scales_t)
            self._gx_from = addresses(g.codes, g.scales, w.codes_t, w.scales_t) if last else \
                addresses(w.codes_t, w.scales_t, g.codes_t, g.scales_t)
            self._gw_from = addresses(g.codes_t, g.scales_t, x.codes_t, x.scales_t) if last else \
                addresses(g.codes, g.scales, x.codes, x.scales)
        self._ws_args = self._ws.data_ptr(), self._ws.numel()
        self._loaded = self._kept = False

    def load(self, w, stream=None):
        """The weight [c_out, c_in] (or [c_out, c_in, 1, 1]), for the calls that follow."""
        B._arg(w, "w", w.shape, self.dtype)
        if tuple(w.shape) not in (self.w_shape, self.w_shape + (1, 1)):  # (a 1 x 1 convolution's)
            raise ValueError(f"w: expected shape {self.w_shape}, got {tuple(w.shape)}")
        self.weight.load(w, stream)
        self._loaded = True

    def forward(self, x, y=None, stream=None):
        """y (a new tensor of ``stream``'s if not given) = W x."""
        if not self._loaded:
            raise ValueError("the layer has no weight yet (load)")
        x_ptr = B._arg(x, "x", self.x_shape, self.dtype)
        y = _empty(self.y_shape, self.dtype, x.device, stream) if y is None else y
        y_ptr = B._arg(y, "y", self.y_shape, self.dtype)
        s = B._raw_stream(stream)
        if self._one is not None:
            status = self._lib.dc_fp8_pointwise(self._one, x_ptr, *self._w, y_ptr, s)
            if status:
                raise B.DcError(status, "dc_fp8_pointwise")
            return y
        self._run(self.x.p, x_ptr, self._x_to, s)
        self._product(self._fwd, self._fwd_from, y_ptr, s)
        self._kept = True
        return y

    def backward(self, grad_y, grad_x=None, grad_w=None, stream=None):
        """(grad_x, grad_w) of the last forward's input and of the weight: in
        ``dtype`` and float32, new tensors if not given."""
        if not self.training:
            raise ValueError("a layer made with training=False keeps nothing for a backward pass")
        if not self._kept:
            raise ValueError("no forward pass before the backward pass")
        g_ptr = B._arg(grad_y, "grad_y", self.y_shape, self.grad_dtype)
        if grad_x is None:
            grad_x = _empty(self.x_shape, self.dtype, grad_y.device, stream)
        if grad_w is None:
            grad_w = _empty(self.w_shape, torch.float32, grad_y.device, stream)
        gx_ptr = B._arg(grad_x, "grad_x", self.x_shape, self.dtype)
        gw_ptr = B._arg(grad_w, "grad_w", self.w_shape if grad_w.dim() == 2 else self.w_shape + (1, 1), torch.float32)
        s = B._raw_stream(stream)
        self._run(self.gy.p, g_ptr, self._gy_to, s)
        self._product(self._gx, self._gx_from, gx_ptr, s)
        self._product(self._gw, self._gw_from, gw_ptr, s)
        return grad_x, grad_w

    def _run(self, p, ptr, to, s):
        status = self._lib.dc_fp8_quantize(p, ptr, *to, s)
        if status:
            raise B.DcError(status, "dc_fp8_quantize")

    def _product(self, p, factors, out, s):
        status = self._lib.dc_fp8_matmul(p, *factors, out, *self._ws_args, s)
        if status:
            raise B.DcError(status, "dc_fp8_matmul")
