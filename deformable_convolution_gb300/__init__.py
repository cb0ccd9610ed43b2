"""GB300-native deformable convolution layer (sm_103a CUDA behind a C ABI).

The layer is the one the explainer page "DefT: Boosting Scalability of
Deformable Convolution Operations on GPUs" describes: an offset convolution,
a bilinear-interpolation gather that builds the deformed feature map (the two
fused in one kernel), and the main convolution over that map.

``binding`` mirrors ``include/deform_conv.h`` one function per entry point;
``stack`` and ``train`` chain them over stacks of layers (``train``: with group
norm between layers, pointwise layers in 8 bits, ``fp8``, and clipped AdamW or
Muon steps, ``optim``); ``workloads`` holds the seeded synthetic inputs used by the tests and the
benchmark.  The library is built in-tree by ``_native.build()``.
"""
from .binding import (DC_ACT_GELU, DC_ACT_NONE, DC_ACT_RELU, DC_ACT_SILU, DC_BF16, DC_E4M3, DC_E5M2,
                      DC_F32, DC_NCHW, DC_NHWC, DcError, Fp8Problem, Fp8Product, NormProblem, Problem,
                      backward, dc_fp8_matmul, dc_fp8_quantize, dc_fp8_values, dc_group_norm_bwd,
                      dc_group_norm_fwd, dc_muon_step, dc_orthogonalize, deform_conv_bwd, deform_conv_fwd, deform_conv_sample,
                      deform_conv_workspace_size, forward, group_norm, group_norm_backward,
                      norm_workspace, workspace)
from .fp8 import Pointwise, Quantized
from .optim import AdamW, GradNorm, Muon, Orthogonalize, StateValues

__all__ = ["AdamW", "DC_ACT_GELU", "DC_ACT_NONE", "DC_ACT_RELU", "DC_ACT_SILU", "DC_BF16", "DC_E4M3",
           "DC_E5M2", "DC_F32", "DC_NCHW", "DC_NHWC", "DcError", "Fp8Problem", "Fp8Product", "GradNorm",
           "Muon", "NormProblem", "Orthogonalize", "Pointwise", "Problem", "Quantized", "StateValues",
           "backward", "dc_fp8_matmul", "dc_fp8_quantize", "dc_fp8_values", "dc_group_norm_bwd",
           "dc_group_norm_fwd", "dc_muon_step", "dc_orthogonalize", "deform_conv_bwd", "deform_conv_fwd",
           "deform_conv_sample", "deform_conv_workspace_size", "forward", "group_norm",
           "group_norm_backward", "norm_workspace", "workspace"]
