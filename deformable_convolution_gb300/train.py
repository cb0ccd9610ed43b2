"""Training of a stack of deformable layers, each followed by group norm and an
activation, with clipped AdamW steps: the whole step through the C ABI.

Per layer: y = deformable conv(x) (``deform_conv_fwd``), x' = act(group norm of
y) (``dc_group_norm_fwd``).  Backward: group norm's backward takes the gradient
of x' (float32 from the layer above, the caller's dtype at the top) and writes
the layer's grad_y in its dtype; the layer's backward reuses the deformed map
of its forward (``deform_conv_bwd_after_fwd``).  Then ``dc_grad_norm`` over
every gradient and one ``dc_adamw_step`` over every parameter, clipped by the
factor that the former left on the device.  bf16 weights are rounded copies of
float32 masters; biases, offsets' biases and norms' parameters are float32 and
do not decay.

Marshalling only: buffers come from PyTorch, every step of the arithmetic runs
in the library's kernels.  ``python -m deformable_convolution_gb300.train``
fits a small stack to the outputs of another one.
"""
from __future__ import annotations

import argparse
import dataclasses

import torch

from . import binding as B
from . import optim


class Trainer:
    """Buffers and calls of a training step over ``len(params)`` layers.

    p: the layers' problem (C_in = C_out, output size equal to the input size);
    params: per layer a dict of CUDA tensors w_off, b_off, w (as in ``Stack``)
    and gamma, beta (float32 [C]), updated in place.  max_norm: the gradients'
    norm is clipped to it; state_bits: of the optimiser's states."""

    def __init__(self, p: B.Problem, params, groups=32, act=B.DC_ACT_SILU, lr=1e-3,
                 betas=(0.9, 0.999), weight_decay=0.01, max_norm=1.0, state_bits=32, eps=1e-5):
        s = p.shapes()
        if s["x"] != s["y"]:
            raise ValueError("stacked layers need C_in = C_out and an unchanged size")
        self.p, self.params, self.L, self.max_norm = p, list(params), len(params), max_norm
        device, dt, f32 = params[0]["w"].device, p.torch_dtype, torch.float32
        top = B.NormProblem(p.n, p.c_out, p.ho, p.wo, groups, p.dtype, B.DC_NCHW, act, eps, p.dtype)
        below = dataclasses.replace(top, grad_dtype=B.DC_F32)  # grad_x of the layer above
        self.norm = [below] * (self.L - 1) + [top]

        def empty(shape, dtype=f32):
            return torch.empty(shape, dtype=dtype, device=device)
        self.x = [None] + [empty(s["x"], dt) for _ in range(self.L)]  # x[l + 1]: layer l's output
        self.y = [empty(s["y"], dt) for _ in range(self.L)]           # before the norm
        self.off = [empty(s["offset"]) for _ in range(self.L)]
        self.stats = [(empty(top.stat_shape), empty(top.stat_shape)) for _ in range(self.L)]
        self.ws = [B.workspace(p, True, device) for _ in range(self.L)]
        self.norm_ws = empty(max(1, *(B.dc_group_norm_workspace_size(q, b)
                                      for q in (top, below) for b in (False, True))), torch.uint8)
        self.gy = empty(s["y"], dt)
        self.gx = empty(s["x"])
        keys = dict(w_off=s["w_off"], b_off=s["b_off"], w=s["w"], gamma=(p.c_out,), beta=(p.c_out,))
        self.grads = [{k: empty(shape) for k, shape in keys.items()} for _ in range(self.L)]
        entries = []
        for q, g in zip(self.params, self.grads):
            for k in keys:
                e = dict(param=q[k], grad=g[k], weight_decay=weight_decay if k in ("w", "w_off") else 0.0)
                if q[k].dtype == torch.bfloat16:
                    e["master"] = q[k].float()
                entries.append(e)
        self.opt = optim.AdamW(entries, lr=lr, betas=betas, state_bits=state_bits, min_8bit=4096)
        self.grad_norm, self.clip = empty(1), empty(1)

    def forward(self, x0):
        """The stack's output (a buffer that the next call overwrites)."""
        self.x[0] = x0
        for l, q in enumerate(self.params):
            B.deform_conv_fwd(self.p, self.x[l], q["w_off"], q["b_off"], q["w"], None, self.y[l],
                              self.off[l], None, self.ws[l])
            B.dc_group_norm_fwd(self.norm[l], self.y[l], q["gamma"], q["beta"], self.x[l + 1],
                                *self.stats[l], self.norm_ws)
        return self.x[-1]

    def backward(self, grad_out):
        """Gradients of sum(output * grad_out) into ``self.grads``; returns the
        input's (float32)."""
        grad = grad_out
        for l in reversed(range(self.L)):
            q, g = self.params[l], self.grads[l]
            B.dc_group_norm_bwd(self.norm[l], self.y[l], q["gamma"], q["beta"], *self.stats[l], grad,
                                self.gy, g["gamma"], g["beta"], self.norm_ws)
            B.deform_conv_bwd(self.p, self.x[l], q["w_off"], q["w"], self.off[l], self.gy, self.gx,
                              g["w_off"], g["b_off"], g["w"], None, self.ws[l], after_fwd=True)
            grad = self.gx
        return self.gx

    def update(self):
        """The clipped AdamW step; the norm stays in ``self.grad_norm``.  A norm
        that is not finite leaves every parameter as it is."""
        self.opt.grad_norm(self.max_norm, self.grad_norm, self.clip)
        self.opt.step(self.clip)


def initial_params(p: B.Problem, layers, seed=0, device="cuda"):
    """He-initialised main weights, small offset weights, unit norms."""
    gen = torch.Generator().manual_seed(seed)
    s, dt, out = p.shapes(), p.torch_dtype, []
    fan = p.c_in * p.kh * p.kw
    for _ in range(layers):
        q = dict(w_off=(torch.randn(s["w_off"], generator=gen) * 0.5 / fan ** 0.5).to(dt),
                 b_off=torch.zeros(s["b_off"]),
                 w=(torch.randn(s["w"], generator=gen) * (2.0 / fan) ** 0.5).to(dt),
                 gamma=torch.ones(p.c_out), beta=torch.zeros(p.c_out))
        out.append({k: v.to(device) for k, v in q.items()})
    return out


def main(argv=None):
    ap = argparse.ArgumentParser(description="fit a small stack of deformable layers to another one")
    ap.add_argument("--steps", type=int, default=100)
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--channels", type=int, default=64)
    ap.add_argument("--size", type=int, default=28)
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--state-bits", type=int, choices=(8, 32), default=8)
    a = ap.parse_args(argv)
    p = B.Problem(a.batch, a.channels, a.size, a.size, a.channels, dtype=B.DC_BF16)
    teacher = Trainer(p, initial_params(p, a.layers, seed=1), groups=8)
    student = Trainer(p, initial_params(p, a.layers, seed=2), groups=8, state_bits=a.state_bits)
    gen = torch.Generator(device="cuda").manual_seed(0)
    losses = []
    for t in range(a.steps):
        x = torch.randn(p.shapes()["x"], generator=gen, device="cuda").to(p.torch_dtype)
        diff = student.forward(x).float() - teacher.forward(x).float()
        student.backward((diff * (2.0 / diff.numel())).to(p.torch_dtype))
        student.update()
        losses.append(diff.square().mean())
        if t % 10 == 0 or t == a.steps - 1:
            print(f"step {t:4d}  loss {float(losses[-1]):.5f}  gradient norm {float(student.grad_norm):.4f}")
    return [float(v) for v in losses]


if __name__ == "__main__":
    main()
