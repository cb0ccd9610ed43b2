"""Thin Python binding of the C ABI in ``include/deform_conv.h``.

Argument marshalling only: every function here checks tensor shapes and
dtypes, passes raw device pointers and the current CUDA stream to the library
and turns a non-OK status into ``DcError``.  All arithmetic runs in the CUDA
kernels of ``libdeformconv.so``; nothing here computes any part of the layer.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass
from functools import cached_property

import torch

from . import _native

DC_OK, DC_ERR_INVALID_ARG, DC_ERR_UNSUPPORTED, DC_ERR_WORKSPACE, DC_ERR_CUDA, DC_ERR_TIMEOUT = range(6)
DC_F32, DC_BF16 = 0, 1
_TORCH_DTYPE = {DC_F32: torch.float32, DC_BF16: torch.bfloat16}

# every symbol include/deform_conv.h declares
EXPORTED_SYMBOLS = (
    "dc_out_h", "dc_out_w", "deform_conv_workspace_size", "deform_conv_fwd",
    "deform_conv_bwd", "deform_conv_sample", "dc_status_string", "dc_build_info",
    "dc_launch_count", "deform_conv_fwd_noalloc", "dc_device_error", "dc_kernel_timing",
    "dc_kernel_times", "deform_conv_offsets", "deform_conv_margin_histogram", "dc_suggest_margin",
    "deform_conv_bwd_after_fwd", "deform_conv_fwd_sampled_gemm", "dc_relu_fwd", "dc_relu_bwd",
    "dc_col_layout", "dc_sample_tile", "dc_selftest_wait_timeout", "dc_test_fail_launches",
    "dc_group_norm_workspace_size", "dc_group_norm_fwd", "dc_group_norm_bwd",
    "dc_adamw_step", "dc_adamw_state_values", "dc_grad_norm_workspace_size", "dc_grad_norm",
    "dc_fp8_sizes", "dc_fp8_quantize", "dc_fp8_values", "dc_fp8_matmul_workspace_size",
    "dc_fp8_matmul", "dc_fp8_pointwise", "dc_orthogonalize_workspace_size", "dc_orthogonalize",
    "dc_muon_workspace_size", "dc_muon_step",
)
DC_NCHW, DC_NHWC = 0, 1
DC_ACT_NONE, DC_ACT_RELU, DC_ACT_SILU, DC_ACT_GELU = range(4)
DC_STATE_F32, DC_STATE_Q8 = 0, 1
DC_E4M3, DC_E5M2 = 0, 1
DC_ORTHO_16, DC_ORTHO_32 = 0, 1
FP8_BLOCK = 128    # values that share a scale
FP8_RUN = 8192     # most values of k that a product sums in one accumulator
STATE_BLOCK = 256  # elements of an 8-bit state that share a scale
DC_COL_PLANE_MAJOR, DC_COL_PIXEL_MAJOR = 0, 1
MARGIN_BINS = 64
NOALLOC_SCRATCH_BYTES = 32 << 20


class DcProblem(ctypes.Structure):
    """Mirror of ``dc_problem``."""
    _fields_ = [(name, ctypes.c_int) for name in (
        "n", "c_in", "h", "w", "c_out", "kh", "kw", "stride_h", "stride_w",
        "pad_h", "pad_w", "dil_h", "dil_w", "offset_groups", "dtype", "halo_margin", "out_relu",
        "in_relu")]


class DcNormProblem(ctypes.Structure):
    """Mirror of ``dc_norm_problem``."""
    _fields_ = [(name, ctypes.c_int) for name in (
        "n", "c", "h", "w", "groups", "dtype", "layout", "act")] + \
        [("eps", ctypes.c_float), ("grad_dtype", ctypes.c_int)]


class DcAdamwTensor(ctypes.Structure):
    """Mirror of ``dc_adamw_tensor``."""
    _fields_ = [(name, ctypes.c_void_p) for name in (
        "param", "master", "grad", "m", "v", "m_scale", "v_scale")] + \
        [("count", ctypes.c_longlong), ("param_dtype", ctypes.c_int),
         ("grad_dtype", ctypes.c_int), ("state", ctypes.c_int), ("weight_decay", ctypes.c_float)]


class DcAdamwHyper(ctypes.Structure):
    """Mirror of ``dc_adamw_hyper``."""
    _fields_ = [(name, ctypes.c_double) for name in ("lr", "beta1", "beta2", "eps")] + \
        [("step", ctypes.c_longlong)]


class DcFp8Problem(ctypes.Structure):
    """Mirror of ``dc_fp8_problem``."""
    _fields_ = [(name, ctypes.c_int) for name in ("batch", "rows", "cols", "dtype", "format", "square")]


class DcFp8Product(ctypes.Structure):
    """Mirror of ``dc_fp8_product``."""
    _fields_ = [(name, ctypes.c_int) for name in (
        "batch", "m", "n", "k", "a_format", "b_format", "a_shared", "b_shared", "sum", "out", "beside")]


class DcFp8Layer(ctypes.Structure):
    """Mirror of ``dc_fp8_layer``."""
    _fields_ = [(name, ctypes.c_int) for name in ("n", "pixels", "c_in", "c_out", "layout")]


class DcMatrix(ctypes.Structure):
    """Mirror of ``dc_matrix``."""
    _fields_ = [("in_", ctypes.c_void_p), ("out", ctypes.c_void_p)] + \
        [(name, ctypes.c_int) for name in ("rows", "cols", "in_dtype", "out_dtype")]


class DcMuonTensor(ctypes.Structure):
    """Mirror of ``dc_muon_tensor``."""
    _fields_ = [(name, ctypes.c_void_p) for name in ("param", "master", "grad", "m")] + \
        [(name, ctypes.c_int) for name in ("rows", "cols", "param_dtype", "grad_dtype")] + \
        [("weight_decay", ctypes.c_float), ("rate", ctypes.c_float)]


class DcMuonHyper(ctypes.Structure):
    """Mirror of ``dc_muon_hyper``."""
    _fields_ = [("lr", ctypes.c_double), ("momentum", ctypes.c_double)] + \
        [(name, ctypes.c_int) for name in ("nesterov", "steps", "precision")]


class DcError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)}")


_configured = None  # the library, once its functions' types are set


def lib() -> ctypes.CDLL:
    global _configured
    if _configured is not None:
        return _configured
    L = _native.load()
    vp, sz, i = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
    pp = ctypes.POINTER(DcProblem)
    L.dc_out_h.argtypes = [pp]
    L.dc_out_h.restype = i
    L.dc_out_w.argtypes = [pp]
    L.dc_out_w.restype = i
    L.deform_conv_workspace_size.argtypes = [pp, i, ctypes.POINTER(sz)]
    L.deform_conv_workspace_size.restype = i
    L.deform_conv_fwd.argtypes = [pp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.deform_conv_fwd.restype = i
    L.deform_conv_bwd.argtypes = [pp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.deform_conv_bwd.restype = i
    L.deform_conv_bwd_after_fwd.argtypes = [pp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.deform_conv_bwd_after_fwd.restype = i
    L.deform_conv_sample.argtypes = [pp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.deform_conv_sample.restype = i
    L.dc_col_layout.argtypes = [pp]
    L.dc_col_layout.restype = i
    L.dc_sample_tile.argtypes = [pp, ctypes.POINTER(i), ctypes.POINTER(i)]
    L.dc_sample_tile.restype = i
    L.deform_conv_offsets.argtypes = [pp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.deform_conv_offsets.restype = i
    L.deform_conv_fwd_sampled_gemm.argtypes = [pp, vp, vp, vp, vp, vp, vp, vp, vp]
    L.deform_conv_fwd_sampled_gemm.restype = i
    L.deform_conv_margin_histogram.argtypes = [pp, vp, vp, vp]
    L.deform_conv_margin_histogram.restype = i
    L.dc_suggest_margin.argtypes = [pp, ctypes.POINTER(ctypes.c_ulonglong), ctypes.c_double, i]
    L.dc_suggest_margin.restype = i
    L.dc_status_string.argtypes = [i]
    L.dc_status_string.restype = ctypes.c_char_p
    L.dc_build_info.argtypes = []
    L.dc_build_info.restype = ctypes.c_char_p
    L.deform_conv_fwd_noalloc.argtypes = [pp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    L.deform_conv_fwd_noalloc.restype = i
    L.dc_kernel_timing.argtypes = [i]
    L.dc_kernel_timing.restype = None
    L.dc_kernel_times.argtypes = [ctypes.POINTER(ctypes.c_char_p), ctypes.POINTER(ctypes.c_float), i]
    L.dc_kernel_times.restype = i
    L.dc_device_error.argtypes = [i]
    L.dc_device_error.restype = i
    L.dc_selftest_wait_timeout.argtypes = [ctypes.c_uint, vp]
    L.dc_selftest_wait_timeout.restype = i
    L.dc_test_fail_launches.argtypes = [i]
    L.dc_test_fail_launches.restype = i
    L.dc_relu_fwd.argtypes = [vp, vp, sz, i, vp]
    L.dc_relu_fwd.restype = i
    L.dc_relu_bwd.argtypes = [vp, vp, vp, sz, i, vp]
    L.dc_relu_bwd.restype = i
    pn, pt = ctypes.POINTER(DcNormProblem), ctypes.POINTER(DcAdamwTensor)
    ph, pv = ctypes.POINTER(DcAdamwHyper), ctypes.POINTER(vp)
    L.dc_group_norm_workspace_size.argtypes = [pn, i, ctypes.POINTER(sz)]
    L.dc_group_norm_workspace_size.restype = i
    L.dc_group_norm_fwd.argtypes = [pn, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.dc_group_norm_fwd.restype = i
    L.dc_group_norm_bwd.argtypes = [pn, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.dc_group_norm_bwd.restype = i
    L.dc_adamw_step.argtypes = [pt, i, ph, vp, vp, vp]
    L.dc_adamw_step.restype = i
    L.dc_adamw_state_values.argtypes = [pt, i, pv, pv, vp]
    L.dc_adamw_state_values.restype = i
    L.dc_grad_norm_workspace_size.argtypes = [i, ctypes.POINTER(sz)]
    L.dc_grad_norm_workspace_size.restype = i
    L.dc_grad_norm.argtypes = [pt, i, ctypes.c_float, vp, vp, vp, sz, vp]
    L.dc_grad_norm.restype = i
    pq, pm = ctypes.POINTER(DcFp8Problem), ctypes.POINTER(DcFp8Product)
    po, pw, ps = ctypes.POINTER(DcMatrix), ctypes.POINTER(DcMuonTensor), ctypes.POINTER(sz)
    for name, types in dict(
            dc_fp8_sizes=[pq, i, ps, ps], dc_fp8_quantize=[pq, vp, vp, vp, vp, vp, vp],
            dc_fp8_values=[pq, i, vp, vp, vp, vp], dc_fp8_matmul_workspace_size=[pm, ps],
            dc_fp8_matmul=[pm, vp, vp, vp, vp, vp, vp, sz, vp],
            dc_fp8_pointwise=[ctypes.POINTER(DcFp8Layer), vp, vp, vp, vp, vp],
            dc_orthogonalize_workspace_size=[po, i, ps],
            dc_orthogonalize=[po, i, i, i, vp, sz, vp], dc_muon_workspace_size=[pw, i, ps],
            dc_muon_step=[pw, i, ctypes.POINTER(DcMuonHyper), vp, vp, vp, sz, vp]).items():
        f = getattr(L, name)
        f.argtypes, f.restype = types, i
    L.dc_launch_count.argtypes = []
    L.dc_launch_count.restype = ctypes.c_ulonglong
    _configured = L
    return L


def status_string(status: int) -> str:
    return lib().dc_status_string(int(status)).decode()


def build_info() -> str:
    return lib().dc_build_info().decode()


def device_error(clear: bool = False) -> int:
    """DC_ERR_TIMEOUT if a bounded device wait expired (synchronises)."""
    return int(lib().dc_device_error(1 if clear else 0))


def selftest_wait_timeout(spins: int, stream=None) -> int:
    """Test hook: a kernel whose bounded wait on an mbarrier nothing arrives on
    expires after `spins` polls (the next device_error() is DC_ERR_TIMEOUT)."""
    return int(lib().dc_selftest_wait_timeout(spins, _stream(stream)))


def test_fail_launches(count: int) -> int:
    """Test hook: the next `count` launches of the layer entry points fail
    with DC_ERR_CUDA without being made (0 cancels)."""
    return int(lib().dc_test_fail_launches(count))


def kernel_timing(enable: bool) -> None:
    """Start/stop CUDA-event timing of every launch the library enqueues."""
    lib().dc_kernel_timing(1 if enable else 0)


def kernel_times(capacity: int = 256):
    """[(kernel name, ms)] of the launches recorded since timing was enabled
    (waits for them); clears the record."""
    names = (ctypes.c_char_p * capacity)()
    ms = (ctypes.c_float * capacity)()
    n = lib().dc_kernel_times(names, ms, capacity)
    return [(names[i].decode(), float(ms[i])) for i in range(n)]


def launch_count() -> int:
    return int(lib().dc_launch_count())


@dataclass(frozen=True)
class Problem:
    """One deformable layer: NCHW input, 3x3-style kernel geometry, dtype."""
    n: int
    c_in: int
    h: int
    w: int
    c_out: int
    kh: int = 3
    kw: int = 3
    stride: tuple = (1, 1)
    pad: tuple = (1, 1)
    dil: tuple = (1, 1)
    offset_groups: int = 1
    dtype: int = DC_F32
    halo_margin: int = -1
    out_relu: int = 0  # 1: the forward writes relu(y) (a following ReLU fused into its epilogue)
    in_relu: int = 0   # 1: x = relu(z); the backward writes dL/dz in the dtype as grad_x

    def __post_init__(self):
        for f in ("stride", "pad", "dil"):
            v = getattr(self, f)
            if isinstance(v, int):
                object.__setattr__(self, f, (v, v))

    def c_struct(self) -> DcProblem:
        return DcProblem(self.n, self.c_in, self.h, self.w, self.c_out, self.kh, self.kw,
                         self.stride[0], self.stride[1], self.pad[0], self.pad[1],
                         self.dil[0], self.dil[1], self.offset_groups, self.dtype,
                         self.halo_margin, self.out_relu, self.in_relu)

    @property
    def torch_dtype(self):
        return _TORCH_DTYPE[self.dtype]

    @property
    def ho(self):
        return (self.h + 2 * self.pad[0] - self.dil[0] * (self.kh - 1) - 1) // self.stride[0] + 1

    @property
    def wo(self):
        return (self.w + 2 * self.pad[1] - self.dil[1] * (self.kw - 1) - 1) // self.stride[1] + 1

    @property
    def n_off(self):
        return 2 * self.offset_groups * self.kh * self.kw

    def shapes(self):
        return dict(x=(self.n, self.c_in, self.h, self.w),
                    w_off=(self.n_off, self.c_in, self.kh, self.kw),
                    b_off=(self.n_off,),
                    w=(self.c_out, self.c_in, self.kh, self.kw),
                    offset=(self.n, self.n_off, self.ho, self.wo),
                    y=(self.n, self.c_out, self.ho, self.wo),
                    col=(self.c_in * self.kh * self.kw, self.n, self.ho * self.wo))

    # (the deformed map's shape depends on the path the library takes for the
    # problem: binding.col_shape)


def _ptr(t, name, shape=None, dtype=None, optional=False):
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _check(status, what):
    if status != DC_OK:
        raise DcError(status, what)


def deform_conv_workspace_size(p: Problem, backward: bool) -> int:
    out = ctypes.c_size_t(0)
    st = p.c_struct()
    _check(lib().deform_conv_workspace_size(ctypes.byref(st), 1 if backward else 0,
                                            ctypes.byref(out)), "deform_conv_workspace_size")
    return int(out.value)


def out_hw(p: Problem):
    st = p.c_struct()
    return lib().dc_out_h(ctypes.byref(st)), lib().dc_out_w(ctypes.byref(st))


def deform_conv_fwd(p: Problem, x, w_off, b_off, w, offset_add, y, offset_out=None,
                    slowpath_count=None, ws=None, stream=None):
    s = p.shapes()
    dt, f32 = p.torch_dtype, torch.float32
    st = p.c_struct()
    ws_ptr = _ptr(ws, "ws", dtype=torch.uint8)
    _check(lib().deform_conv_fwd(
        ctypes.byref(st), _ptr(x, "x", s["x"], dt), _ptr(w_off, "w_off", s["w_off"], dt),
        _ptr(b_off, "b_off", s["b_off"], f32, True), _ptr(w, "w", s["w"], dt),
        _ptr(offset_add, "offset_add", s["offset"], f32, True), _ptr(y, "y", s["y"], dt),
        _ptr(offset_out, "offset_out", s["offset"], f32, True),
        _ptr(slowpath_count, "slowpath_count", (1,), torch.int64, True),
        ws_ptr, ctypes.c_size_t(ws.numel()), _stream(stream)), "deform_conv_fwd")


def deform_conv_fwd_noalloc(p: Problem, x, w_off, b_off, w, offset_add, y, offset_out=None,
                            slowpath_count=None, stream=None):
    """Forward pass with the library's fixed scratch array instead of a
    workspace (for callers that cannot allocate device memory)."""
    s = p.shapes()
    dt, f32 = p.torch_dtype, torch.float32
    st = p.c_struct()
    _check(lib().deform_conv_fwd_noalloc(
        ctypes.byref(st), _ptr(x, "x", s["x"], dt), _ptr(w_off, "w_off", s["w_off"], dt),
        _ptr(b_off, "b_off", s["b_off"], f32, True), _ptr(w, "w", s["w"], dt),
        _ptr(offset_add, "offset_add", s["offset"], f32, True), _ptr(y, "y", s["y"], dt),
        _ptr(offset_out, "offset_out", s["offset"], f32, True),
        _ptr(slowpath_count, "slowpath_count", (1,), torch.int64, True),
        _stream(stream)), "deform_conv_fwd_noalloc")


def deform_conv_bwd(p: Problem, x, w_off, w, offset, grad_y, grad_x, grad_w_off, grad_b_off,
                    grad_w, grad_offset=None, ws=None, stream=None, after_fwd=False):
    """after_fwd: `ws` still holds the deformed map of the deform_conv_fwd call
    for these inputs (deform_conv_bwd_after_fwd); the map is not replayed.
    grad_x is float32, or of the problem dtype when ``p.in_relu``."""
    s = p.shapes()
    dt, f32 = p.torch_dtype, torch.float32
    st = p.c_struct()
    ws_ptr = _ptr(ws, "ws", dtype=torch.uint8)
    fn = lib().deform_conv_bwd_after_fwd if after_fwd else lib().deform_conv_bwd
    _check(fn(
        ctypes.byref(st), _ptr(x, "x", s["x"], dt), _ptr(w_off, "w_off", s["w_off"], dt),
        _ptr(w, "w", s["w"], dt), _ptr(offset, "offset", s["offset"], f32),
        _ptr(grad_y, "grad_y", s["y"], dt), _ptr(grad_x, "grad_x", s["x"], dt if p.in_relu else f32),
        _ptr(grad_w_off, "grad_w_off", s["w_off"], f32),
        _ptr(grad_b_off, "grad_b_off", s["b_off"], f32, True),
        _ptr(grad_w, "grad_w", s["w"], f32),
        _ptr(grad_offset, "grad_offset", s["offset"], f32, True),
        ws_ptr, ctypes.c_size_t(ws.numel()), _stream(stream)), "deform_conv_bwd")


def col_layout(p: Problem) -> int:
    """DC_COL_PLANE_MAJOR or DC_COL_PIXEL_MAJOR (the deformed map's layout)."""
    st = p.c_struct()
    v = int(lib().dc_col_layout(ctypes.byref(st)))
    if v < 0:
        raise DcError(DC_ERR_INVALID_ARG, "dc_col_layout")
    return v


def col_shape(p: Problem):
    """Shape of the deformed map in the problem's layout."""
    if col_layout(p) == DC_COL_PIXEL_MAJOR:
        return (p.n, p.ho * p.wo, p.kh * p.kw, p.c_in)
    return (p.c_in * p.kh * p.kw, p.n, p.ho * p.wo)


def sample_tile(p: Problem):
    """(tile_h, tile_w): the output tile the sampling stage stages a window for."""
    st = p.c_struct()
    th, tw = ctypes.c_int(0), ctypes.c_int(0)
    _check(lib().dc_sample_tile(ctypes.byref(st), ctypes.byref(th), ctypes.byref(tw)),
           "dc_sample_tile")
    return th.value, tw.value


def deform_conv_sample(p: Problem, x, w_off, b_off, offset_add, offset_in, col,
                       offset_out=None, slowpath_count=None, ws=None, stream=None):
    s = p.shapes()
    dt, f32 = p.torch_dtype, torch.float32
    st = p.c_struct()
    if ws is None:
        ws = workspace(p, False, x.device)
    _check(lib().deform_conv_sample(
        ctypes.byref(st), _ptr(x, "x", s["x"], dt),
        _ptr(w_off, "w_off", s["w_off"], dt, True),
        _ptr(b_off, "b_off", s["b_off"], f32, True),
        _ptr(offset_add, "offset_add", s["offset"], f32, True),
        _ptr(offset_in, "offset_in", s["offset"], f32, True),
        _ptr(col, "col", col_shape(p), dt),
        _ptr(offset_out, "offset_out", s["offset"], f32, True),
        _ptr(slowpath_count, "slowpath_count", (1,), torch.int64, True),
        _ptr(ws, "ws", dtype=torch.uint8), ctypes.c_size_t(ws.numel()),
        _stream(stream)), "deform_conv_sample")


def deform_conv_offsets(p: Problem, x, w_off, b_off, offset_add, offset_out, ws=None,
                        stream=None):
    s = p.shapes()
    dt, f32 = p.torch_dtype, torch.float32
    st = p.c_struct()
    if ws is None:
        ws = workspace(p, False, x.device)
    _check(lib().deform_conv_offsets(
        ctypes.byref(st), _ptr(x, "x", s["x"], dt), _ptr(w_off, "w_off", s["w_off"], dt),
        _ptr(b_off, "b_off", s["b_off"], f32, True),
        _ptr(offset_add, "offset_add", s["offset"], f32, True),
        _ptr(offset_out, "offset_out", s["offset"], f32),
        _ptr(ws, "ws", dtype=torch.uint8), ctypes.c_size_t(ws.numel()),
        _stream(stream)), "deform_conv_offsets")


def deform_conv_fwd_sampled_gemm(p: Problem, x, w_off, b_off, w, offset_add, y, offset_out,
                                 stream=None):
    s = p.shapes()
    dt, f32 = p.torch_dtype, torch.float32
    st = p.c_struct()
    _check(lib().deform_conv_fwd_sampled_gemm(
        ctypes.byref(st), _ptr(x, "x", s["x"], dt), _ptr(w_off, "w_off", s["w_off"], dt),
        _ptr(b_off, "b_off", s["b_off"], f32, True), _ptr(w, "w", s["w"], dt),
        _ptr(offset_add, "offset_add", s["offset"], f32, True), _ptr(y, "y", s["y"], dt),
        _ptr(offset_out, "offset_out", s["offset"], f32), _stream(stream)),
        "deform_conv_fwd_sampled_gemm")


def deform_conv_margin_histogram(p: Problem, offset, hist, stream=None):
    st = p.c_struct()
    _check(lib().deform_conv_margin_histogram(
        ctypes.byref(st), _ptr(offset, "offset", p.shapes()["offset"], torch.float32),
        _ptr(hist, "hist", (MARGIN_BINS,), torch.int64), _stream(stream)),
        "deform_conv_margin_histogram")


def dc_suggest_margin(p: Problem, hist_host, max_slow_fraction: float, for_backward: bool) -> int:
    """hist_host: MARGIN_BINS counts on the host (any integer sequence)."""
    arr = (ctypes.c_ulonglong * MARGIN_BINS)(*[int(v) for v in hist_host])
    st = p.c_struct()
    return int(lib().dc_suggest_margin(ctypes.byref(st), arr, float(max_slow_fraction),
                                       int(bool(for_backward))))


def _dc_dtype(t):
    for k, v in _TORCH_DTYPE.items():
        if t.dtype == v:
            return k
    raise ValueError(f"unsupported dtype {t.dtype}")


def dc_relu_fwd(y, out, stream=None):
    """out = max(y, 0) (float32 or bfloat16 tensors of one shape; out may be y)."""
    if out.shape != y.shape or out.dtype != y.dtype:
        raise ValueError("y and out must have the same shape and dtype")
    _check(lib().dc_relu_fwd(_ptr(y, "y"), _ptr(out, "out"), ctypes.c_size_t(y.numel()),
                             _dc_dtype(y), _stream(stream)), "dc_relu_fwd")


def dc_relu_bwd(act, grad_out, grad_in, stream=None):
    """grad_in = grad_out where act > 0 else 0, in act's dtype; grad_out float32."""
    if grad_out.shape != act.shape or grad_in.shape != act.shape or grad_in.dtype != act.dtype:
        raise ValueError("act, grad_out and grad_in must have one shape; grad_in act's dtype")
    _check(lib().dc_relu_bwd(_ptr(act, "act"), _ptr(grad_out, "grad_out", dtype=torch.float32),
                             _ptr(grad_in, "grad_in"), ctypes.c_size_t(act.numel()),
                             _dc_dtype(act), _stream(stream)), "dc_relu_bwd")


def _arg(t, name, shape, dtype, optional=False):
    """As ``_ptr``, a plain address: one pass over the usual case, ``_ptr`` for
    what is missing or wrong (these calls are short: a check of a tensor costs
    as much as a kernel's launch)."""
    if t.__class__ in _TENSORS and t.dtype is dtype and t.shape == shape and t.is_cuda and \
            t.is_contiguous():
        return t.data_ptr()
    p = _ptr(t, name, shape, dtype, optional)
    return None if p is None else p.value


_TENSORS = (torch.Tensor, torch.nn.Parameter)


def _raw_stream(stream):
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


# ---------------------------------------------------------------- group norm

@dataclass(frozen=True)
class NormProblem:
    """Group norm with an activation over [n, c, h, w] (DC_NCHW) or
    [n, h, w, c] (DC_NHWC) tensors; a torch channels-last tensor ``t`` is
    ``t.permute(0, 2, 3, 1)`` here.  grad_dtype: grad_y's type, DC_F32 (a
    deformable layer's grad_x) or ``dtype``."""
    n: int
    c: int
    h: int
    w: int
    groups: int
    dtype: int = DC_F32
    layout: int = DC_NCHW
    act: int = DC_ACT_NONE
    eps: float = 1e-5
    grad_dtype: int = DC_F32

    def c_struct(self) -> DcNormProblem:
        return DcNormProblem(self.n, self.c, self.h, self.w, self.groups, self.dtype, self.layout,
                             self.act, self.eps, self.grad_dtype)

    @cached_property
    def _as_parameter_(self):
        return ctypes.byref(self.c_struct())

    @cached_property
    def torch_dtype(self):
        return _TORCH_DTYPE[self.dtype]

    @cached_property
    def shape(self):
        """Of x, y, grad_y and grad_x."""
        if self.layout == DC_NHWC:
            return (self.n, self.h, self.w, self.c)
        return (self.n, self.c, self.h, self.w)

    @cached_property
    def stat_shape(self):
        """Of mean and rstd."""
        return (self.n, self.groups)

    @cached_property
    def channel_shape(self):
        """Of gamma, beta and their gradients."""
        return (self.c,)


def dc_group_norm_workspace_size(p: NormProblem, backward: bool) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().dc_group_norm_workspace_size(p, 1 if backward else 0, ctypes.byref(out)),
           "dc_group_norm_workspace_size")
    return int(out.value)


def _ws(ws):
    """(pointer, bytes) of a workspace that may be None."""
    if ws is None:
        return None, 0
    return _arg(ws, "ws", ws.shape, torch.uint8), ws.numel()


def dc_group_norm_fwd(p: NormProblem, x, gamma, beta, y, mean=None, rstd=None, ws=None,
                      stream=None):
    """y = act(group norm of x); mean and rstd [n, groups] for the backward.
    gamma, beta: float32 [c] or None; y may be x."""
    dt, f32, sh, ss, cs = p.torch_dtype, torch.float32, p.shape, p.stat_shape, p.channel_shape
    ws_ptr, ws_bytes = _ws(ws)
    status = lib().dc_group_norm_fwd(
        p, _arg(x, "x", sh, dt), _arg(gamma, "gamma", cs, f32, True),
        _arg(beta, "beta", cs, f32, True), _arg(y, "y", sh, dt),
        _arg(mean, "mean", ss, f32, True), _arg(rstd, "rstd", ss, f32, True),
        ws_ptr, ws_bytes, _raw_stream(stream))
    if status:
        raise DcError(status, "dc_group_norm_fwd")


def dc_group_norm_bwd(p: NormProblem, x, gamma, beta, mean, rstd, grad_y, grad_x,
                      grad_gamma=None, grad_beta=None, ws=None, stream=None):
    """grad_x (x's dtype; may be grad_y where the types agree), grad_gamma and
    grad_beta (float32 [c] or None) from grad_y in ``p.grad_dtype``."""
    dt, f32, sh, ss, cs = p.torch_dtype, torch.float32, p.shape, p.stat_shape, p.channel_shape
    ws_ptr, ws_bytes = _ws(ws)
    status = lib().dc_group_norm_bwd(
        p, _arg(x, "x", sh, dt), _arg(gamma, "gamma", cs, f32, True),
        _arg(beta, "beta", cs, f32, True), _arg(mean, "mean", ss, f32),
        _arg(rstd, "rstd", ss, f32), _arg(grad_y, "grad_y", sh, _TORCH_DTYPE[p.grad_dtype]),
        _arg(grad_x, "grad_x", sh, dt), _arg(grad_gamma, "grad_gamma", cs, f32, True),
        _arg(grad_beta, "grad_beta", cs, f32, True), ws_ptr, ws_bytes, _raw_stream(stream))
    if status:
        raise DcError(status, "dc_group_norm_bwd")


# ---------------------------------------------------------------- AdamW

def adamw_tensors(entries):
    """A host array of ``dc_adamw_tensor`` from dicts of tensors: param, grad
    (required for a step), m, v, and optionally master, m_scale, v_scale,
    weight_decay.  8-bit states are an int8 m and a uint8 v.  The array holds
    plain pointers: the caller keeps the tensors."""
    out = (DcAdamwTensor * max(len(entries), 1))()
    for t, q in zip(out, entries):
        count = q["grad"].numel()
        shape = tuple(q["grad"].shape)
        t.count = count
        t.grad = _addr(q["grad"], "grad", shape)
        t.grad_dtype = _dc_dtype(q["grad"])
        if q.get("param") is None:
            continue
        t.param, t.param_dtype = _addr(q["param"], "param", shape), _dc_dtype(q["param"])
        t.master = _addr(q.get("master"), "master", shape, torch.float32)
        eight = q["m"].dtype == torch.int8
        t.state = DC_STATE_Q8 if eight else DC_STATE_F32
        t.m = _addr(q["m"], "m", shape, torch.int8 if eight else torch.float32)
        t.v = _addr(q["v"], "v", shape, torch.uint8 if eight else torch.float32)
        if eight:
            blocks = (-(-count // STATE_BLOCK),)
            t.m_scale = _addr(q["m_scale"], "m_scale", blocks, torch.float32)
            t.v_scale = _addr(q["v_scale"], "v_scale", blocks, torch.float32)
        t.weight_decay = q.get("weight_decay", 0.0)
    return out


def _addr(t, name, shape=None, dtype=None):
    p = _ptr(t, name, shape, dtype, True)
    return None if p is None else p.value


def dc_adamw_step(tensors, count: int, hyper: DcAdamwHyper, grad_scale=None, schedule=None,
                  stream=None):
    """One AdamW step over ``tensors`` (``adamw_tensors``).  grad_scale: a
    float32 device scalar or None; schedule: float32 [3] {lr, 1 - beta1^step,
    1 - beta2^step} on the device or None."""
    status = lib().dc_adamw_step(
        tensors, count, hyper, _scalar(grad_scale, "grad_scale"),
        None if schedule is None else _arg(schedule, "schedule", (3,), torch.float32),
        _raw_stream(stream))
    if status:
        raise DcError(status, "dc_adamw_step")


def _scalar(t, name):
    """The address of a one-element float32 device tensor, None for None."""
    if t is None:
        return None
    if t.numel() != 1:
        raise ValueError(f"{name} must hold one value")
    return _arg(t, name, t.shape, torch.float32)


def pointers(tensors, name, shapes, dtype):
    """A host array of the tensors' device pointers (None: a null pointer),
    each checked against its shape.  The caller keeps the tensors."""
    a = (ctypes.c_void_p * max(len(tensors), 1))()
    for k, (t, shape) in enumerate(zip(tensors, shapes)):
        a[k] = _addr(t, f"{name}[{k}]", shape, dtype)
    return a


def dc_adamw_state_values(tensors, count: int, m, v, stream=None):
    """The states as float32 values: m[i] and v[i] (``pointers``, either may be
    None) receive tensor i's."""
    status = lib().dc_adamw_state_values(tensors, count, m, v, _raw_stream(stream))
    if status:
        raise DcError(status, "dc_adamw_state_values")


def dc_grad_norm_workspace_size(count: int) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().dc_grad_norm_workspace_size(count, ctypes.byref(out)),
           "dc_grad_norm_workspace_size")
    return int(out.value)


def dc_grad_norm(tensors, count: int, max_norm: float, norm=None, scale=None, ws=None,
                 stream=None):
    """norm: the gradients' global 2-norm; scale: the factor that clips it to
    max_norm (float32 device scalars or None)."""
    ws_ptr, ws_bytes = _ws(ws)
    status = lib().dc_grad_norm(tensors, count, max_norm, _scalar(norm, "norm"),
                                _scalar(scale, "scale"), ws_ptr, ws_bytes, _raw_stream(stream))
    if status:
        raise DcError(status, "dc_grad_norm")


# ---------------------------------------------------------------- matrices in 8 bits

@dataclass(frozen=True)
class Fp8Problem:
    """``batch`` matrices [rows, cols] of ``dtype`` values to be held as 8-bit
    codes with a scale for each run of 128 columns (square: for each block of
    128 x 128).  Codes are uint8 tensors [batch, rows, cols rounded up to 128],
    scales flat uint8 tensors."""
    batch: int
    rows: int
    cols: int
    dtype: int = DC_BF16
    format: int = DC_E4M3
    square: int = 0

    @cached_property
    def _as_parameter_(self):
        return ctypes.byref(DcFp8Problem(self.batch, self.rows, self.cols, self.dtype, self.format,
                                         self.square))

    @cached_property
    def torch_dtype(self):
        return _TORCH_DTYPE[self.dtype]

    @cached_property
    def shape(self):
        """Of x."""
        return (self.batch, self.rows, self.cols)

    def _shapes(self, transposed):
        r, c = (self.cols, self.rows) if transposed else (self.rows, self.cols)
        nbytes = dc_fp8_sizes(self, transposed)
        return (self.batch, r, -(-c // FP8_BLOCK) * FP8_BLOCK), (nbytes[1],)

    @cached_property
    def shapes(self):
        """Of codes and scales."""
        return self._shapes(False)

    @cached_property
    def shapes_t(self):
        """Of the transposes' codes and scales."""
        return self._shapes(True)


@dataclass(frozen=True)
class Fp8Product:
    """D[i] = A[i] B[i]^T for matrices in 8 bits, A[i] [m, k], B[i] [n, k]
    (``Fp8Problem``s with cols = k); a_shared, b_shared: one matrix for all i;
    sum: D is the sum over i.  out: D's type.  beside: the stream's last launch
    was another product that has nothing to do with what this one reads or writes."""
    batch: int
    m: int
    n: int
    k: int
    a_format: int = DC_E4M3
    b_format: int = DC_E4M3
    a_shared: int = 0
    b_shared: int = 0
    sum: int = 0
    out: int = DC_BF16
    beside: int = 0

    @cached_property
    def _as_parameter_(self):
        return ctypes.byref(DcFp8Product(self.batch, self.m, self.n, self.k, self.a_format,
                                         self.b_format, self.a_shared, self.b_shared, self.sum,
                                         self.out, self.beside))

    @cached_property
    def torch_dtype(self):
        return _TORCH_DTYPE[self.out]

    @cached_property
    def shape(self):
        """Of D."""
        return (self.m, self.n) if self.sum else (self.batch, self.m, self.n)

    def _operand(self, shared, rows):
        p = Fp8Problem(1 if shared else self.batch, rows, max(self.k, 1))
        return p.shapes

    @cached_property
    def a_shapes(self):
        """Of A's codes and scales."""
        return self._operand(self.a_shared, self.m)

    @cached_property
    def b_shapes(self):
        return self._operand(self.b_shared, self.n)


def dc_fp8_sizes(p: Fp8Problem, transposed: bool):
    """(bytes of codes, bytes of scales)."""
    codes, scales = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check(lib().dc_fp8_sizes(p, 1 if transposed else 0, ctypes.byref(codes), ctypes.byref(scales)),
           "dc_fp8_sizes")
    return int(codes.value), int(scales.value)


def _codes(codes, scales, shapes, name, optional=False):
    return (_arg(codes, name, shapes[0], torch.uint8, optional),
            _arg(scales, f"{name}'s scales", shapes[1], torch.uint8, optional))


def dc_fp8_quantize(p: Fp8Problem, x, codes=None, scales=None, codes_t=None, scales_t=None,
                    stream=None):
    """x's codes and scales and, from the same read, its transposes'; either
    pair may be None."""
    status = lib().dc_fp8_quantize(
        p, _arg(x, "x", p.shape, p.torch_dtype), *_codes(codes, scales, p.shapes, "codes", True),
        *_codes(codes_t, scales_t, p.shapes_t, "codes_t", True), _raw_stream(stream))
    if status:
        raise DcError(status, "dc_fp8_quantize")


def dc_fp8_values(p: Fp8Problem, codes, scales, out, transposed=False, stream=None):
    """out: the float32 values that codes stand for (transposed: codes_t's)."""
    shape = (p.batch, p.cols, p.rows) if transposed else p.shape
    status = lib().dc_fp8_values(
        p, 1 if transposed else 0,
        *_codes(codes, scales, p.shapes_t if transposed else p.shapes, "codes"),
        _arg(out, "out", shape, torch.float32), _raw_stream(stream))
    if status:
        raise DcError(status, "dc_fp8_values")


def dc_fp8_matmul_workspace_size(p: Fp8Product) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().dc_fp8_matmul_workspace_size(p, ctypes.byref(out)), "dc_fp8_matmul_workspace_size")
    return int(out.value)


def dc_fp8_matmul(p: Fp8Product, a, a_scales, b, b_scales, d, ws=None, stream=None):
    """d[i] = a[i] b[i]^T (their sum over i where ``p.sum``)."""
    ws_ptr, ws_bytes = _ws(ws)
    status = lib().dc_fp8_matmul(
        p, *_codes(a, a_scales, p.a_shapes, "a"), *_codes(b, b_scales, p.b_shapes, "b"),
        _arg(d, "d", p.shape, p.torch_dtype), ws_ptr, ws_bytes, _raw_stream(stream))
    if status:
        raise DcError(status, "dc_fp8_matmul")


def dc_fp8_pointwise(p: DcFp8Layer, x, w_codes, w_scales, y, stream=None):
    """y = W x over the channels of every pixel, x quantised on the way: bf16
    tensors [n, channels, pixels] (DC_NCHW) or [n, pixels, channels]."""
    w = Fp8Problem(1, p.c_out, p.c_in, DC_BF16, DC_E4M3)
    shapes = [(p.n, p.pixels, c) if p.layout == DC_NHWC else (p.n, c, p.pixels) for c in (p.c_in, p.c_out)]
    status = lib().dc_fp8_pointwise(
        p, _arg(x, "x", shapes[0], torch.bfloat16), *_codes(w_codes, w_scales, w.shapes, "w"),
        _arg(y, "y", shapes[1], torch.bfloat16), _raw_stream(stream))
    if status:
        raise DcError(status, "dc_fp8_pointwise")


# ---------------------------------------------------------------- Muon

def _matrix_shape(t, name):
    """A weight as a matrix: its first dimension by all others."""
    if t.dim() < 2:
        raise ValueError(f"{name} must have two dimensions or more")
    rows = t.shape[0]
    return rows, (t.numel() // rows if rows else 0)


def matrices(ins, outs):
    """A host array of ``dc_matrix`` from input and output tensors of equal
    shapes (the first dimension by all others).  The array holds plain
    pointers: the caller keeps the tensors."""
    if len(ins) != len(outs):
        raise ValueError(f"{len(ins)} inputs and {len(outs)} outputs")
    table = (DcMatrix * max(len(ins), 1))()
    for k, (t, a, b) in enumerate(zip(table, ins, outs)):
        t.rows, t.cols = _matrix_shape(a, f"in[{k}]")
        t.in_, t.in_dtype = _addr(a, f"in[{k}]"), _dc_dtype(a)
        t.out, t.out_dtype = _addr(b, f"out[{k}]", tuple(a.shape)), _dc_dtype(b)
    return table


def muon_tensors(entries):
    """A host array of ``dc_muon_tensor`` from dicts of tensors: param, grad, m,
    and optionally master, weight_decay, rate.  The array holds plain pointers:
    the caller keeps the tensors."""
    table = (DcMuonTensor * max(len(entries), 1))()
    for t, q in zip(table, entries):
        shape = tuple(q["param"].shape)
        t.rows, t.cols = _matrix_shape(q["param"], "param")
        t.param, t.param_dtype = _addr(q["param"], "param"), _dc_dtype(q["param"])
        t.master = _addr(q.get("master"), "master", shape, torch.float32)
        if q.get("grad") is None:
            raise ValueError("grad is required")
        t.grad, t.grad_dtype = _addr(q["grad"], "grad", shape), _dc_dtype(q["grad"])
        t.m = _addr(q["m"], "m", shape, torch.float32)
        t.weight_decay, t.rate = q.get("weight_decay", 0.0), q.get("rate", 1.0)
    return table


def dc_orthogonalize_workspace_size(table, count: int) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().dc_orthogonalize_workspace_size(table, count, ctypes.byref(out)),
           "dc_orthogonalize_workspace_size")
    return int(out.value)


def dc_orthogonalize(table, count: int, steps: int, precision: int, ws=None, stream=None):
    """Orthogonalises the matrices of ``table`` (``matrices``)."""
    ws_ptr, ws_bytes = _ws(ws)
    status = lib().dc_orthogonalize(table, count, steps, precision, ws_ptr, ws_bytes,
                                    _raw_stream(stream))
    if status:
        raise DcError(status, "dc_orthogonalize")


def dc_muon_workspace_size(table, count: int) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().dc_muon_workspace_size(table, count, ctypes.byref(out)), "dc_muon_workspace_size")
    return int(out.value)


def dc_muon_step(table, count: int, hyper: DcMuonHyper, grad_scale=None, lr=None, ws=None,
                 stream=None):
    """One Muon step over ``table`` (``muon_tensors``).  grad_scale, lr: float32
    device scalars or None."""
    ws_ptr, ws_bytes = _ws(ws)
    status = lib().dc_muon_step(table, count, hyper, _scalar(grad_scale, "grad_scale"),
                                _scalar(lr, "lr"), ws_ptr, ws_bytes, _raw_stream(stream))
    if status:
        raise DcError(status, "dc_muon_step")


# ---------------------------------------------------------------- conveniences
# Allocate outputs with torch (device memory is PyTorch's job) and call the ABI.

def workspace(p: Problem, backward: bool, device="cuda"):
    return torch.empty(max(deform_conv_workspace_size(p, backward), 1), dtype=torch.uint8,
                       device=device)


def forward(p: Problem, x, w_off, b_off, w, offset_add=None, ws=None, stream=None,
            slowpath_count=None):
    """Returns (y, offsets)."""
    s = p.shapes()
    y = torch.empty(s["y"], dtype=p.torch_dtype, device=x.device)
    off = torch.empty(s["offset"], dtype=torch.float32, device=x.device)
    if ws is None:
        ws = workspace(p, False, x.device)
    deform_conv_fwd(p, x, w_off, b_off, w, offset_add, y, off, slowpath_count, ws, stream)
    return y, off


def backward(p: Problem, x, w_off, w, offset, grad_y, ws=None, stream=None):
    """Returns dict(grad_x, grad_w_off, grad_b_off, grad_w, grad_offset)."""
    s = p.shapes()
    dev = x.device
    out = dict(grad_x=torch.empty(s["x"], dtype=p.torch_dtype if p.in_relu else torch.float32,
                                  device=dev),
               grad_w_off=torch.empty(s["w_off"], dtype=torch.float32, device=dev),
               grad_b_off=torch.empty(s["b_off"], dtype=torch.float32, device=dev),
               grad_w=torch.empty(s["w"], dtype=torch.float32, device=dev),
               grad_offset=torch.empty(s["offset"], dtype=torch.float32, device=dev))
    if ws is None:
        ws = workspace(p, True, dev)
    deform_conv_bwd(p, x, w_off, w, offset, grad_y, out["grad_x"], out["grad_w_off"],
                    out["grad_b_off"], out["grad_w"], out["grad_offset"], ws, stream)
    return out


def norm_workspace(p: NormProblem, backward: bool, device="cuda"):
    return torch.empty(max(dc_group_norm_workspace_size(p, backward), 1), dtype=torch.uint8,
                       device=device)


def group_norm(p: NormProblem, x, gamma=None, beta=None, ws=None, stream=None):
    """Returns (y, mean, rstd)."""
    y = torch.empty(p.shape, dtype=p.torch_dtype, device=x.device)
    mean, rstd = (torch.empty(p.stat_shape, dtype=torch.float32, device=x.device) for _ in range(2))
    if ws is None:
        ws = norm_workspace(p, False, x.device)
    dc_group_norm_fwd(p, x, gamma, beta, y, mean, rstd, ws, stream)
    return y, mean, rstd


def group_norm_backward(p: NormProblem, x, gamma, beta, mean, rstd, grad_y, ws=None, stream=None):
    """Returns dict(grad_x, grad_gamma, grad_beta)."""
    out = dict(grad_x=torch.empty(p.shape, dtype=p.torch_dtype, device=x.device),
               grad_gamma=torch.empty(p.c, dtype=torch.float32, device=x.device),
               grad_beta=torch.empty(p.c, dtype=torch.float32, device=x.device))
    if ws is None:
        ws = norm_workspace(p, True, x.device)
    dc_group_norm_bwd(p, x, gamma, beta, mean, rstd, grad_y, out["grad_x"], out["grad_gamma"],
                      out["grad_beta"], ws, stream)
    return out
