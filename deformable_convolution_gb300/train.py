"""Training of a stack of deformable layers, each followed by group norm and an
activation (and, where asked for, a pointwise layer in 8 bits), with clipped
AdamW or Muon steps: the whole step through the C ABI.

Per layer: y = deformable conv(x) (``deform_conv_fwd``), x' = act(group norm of
y) (``dc_group_norm_fwd``), with ``w_pw`` among a layer's parameters then
x' = w_pw act(...) over the channels of every pixel (``fp8.Pointwise``).
Backward: group norm's backward takes the gradient
of x' (float32 from the layer above, the caller's dtype at the top) and writes
the layer's grad_y in its dtype; the layer's backward reuses the deformed map
of its forward (``deform_conv_bwd_after_fwd``).  Then ``dc_grad_norm`` over
every gradient and one ``dc_adamw_step`` over every parameter, clipped by the
factor that the former left on the device; with Muon the weights (matrices) go
through ``dc_muon_step`` and AdamW keeps the vectors.  bf16 weights are rounded copies of
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
from . import fp8, optim


class Trainer:
    """Buffers and calls of a training step over ``len(params)`` layers.

    p: the layers' problem (C_in = C_out, output size equal to the input size);
    params: per layer a dict of CUDA tensors w_off, b_off, w (as in ``Stack``)
    and gamma, beta (float32 [C]), updated in place; all layers or none may have
    w_pw [C, C] in the problem's dtype, a pointwise layer behind the activation.
    max_norm: the gradients' norm is clipped to it; state_bits: of AdamW's
    states.  optimizer: "adamw", or "muon" for the weights (``muon``) beside
    AdamW for biases and norms (``opt``)."""

    def __init__(self, p: B.Problem, params, groups=32, act=B.DC_ACT_SILU, lr=1e-3,
                 betas=(0.9, 0.999), weight_decay=0.01, max_norm=1.0, state_bits=32, eps=1e-5,
                 optimizer="adamw"):
        if optimizer not in ("adamw", "muon"):
            raise ValueError("optimizer must be adamw or muon")
        s = p.shapes()
        if s["x"] != s["y"]:
            raise ValueError("stacked layers need C_in = C_out and an unchanged size")
        self.p, self.params, self.L, self.max_norm = p, list(params), len(params), max_norm
        device, dt, f32 = params[0]["w"].device, p.torch_dtype, torch.float32
        top = B.NormProblem(p.n, p.c_out, p.ho, p.wo, groups, p.dtype, B.DC_NCHW, act, eps, p.dtype)
        below = dataclasses.replace(top, grad_dtype=B.DC_F32)  # grad_x of the layer above
        mixed = ["w_pw" in q for q in self.params]
        if any(mixed) != all(mixed):
            raise ValueError("all layers or none have a pointwise layer")
        self.pointwise = None
        if any(mixed):  # takes the gradient from above and hands one in dtype down
            below, above = top, [B.DC_F32] * (self.L - 1) + [p.dtype]
            self.pointwise = [fp8.Pointwise(p.n, p.c_out, p.c_out, p.ho, p.wo, p.dtype, B.DC_NCHW, True, g,
                                            device=device) for g in above]
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
        if self.pointwise:
            keys["w_pw"] = (p.c_out, p.c_out)
            self.z = [empty(s["y"], dt) for _ in range(self.L)]       # before the pointwise layer
            self.gz = empty(s["y"], dt)
        self.grads = [{k: empty(shape) for k, shape in keys.items()} for _ in range(self.L)]
        entries, matrices, weights = [], [], ("w", "w_off", "w_pw")
        for q, g in zip(self.params, self.grads):
            for k in keys:
                e = dict(param=q[k], grad=g[k], weight_decay=weight_decay if k in weights else 0.0)
                if q[k].dtype == torch.bfloat16:
                    e["master"] = q[k].float()
                (matrices if optimizer == "muon" and k in weights else entries).append(e)
        self.opt = optim.AdamW(entries, lr=lr, betas=betas, state_bits=state_bits, min_8bit=4096)
        self.muon = optim.Muon(matrices, lr=lr) if matrices else None
        if matrices:
            self._tables = self.opt.params, self.muon.params
            self._both = optim.GradNorm(self._both_grads())
        self.grad_norm, self.clip = empty(1), empty(1)

    def forward(self, x0):
        """The stack's output (a buffer that the next call overwrites)."""
        self.x[0] = x0
        for l, q in enumerate(self.params):
            B.deform_conv_fwd(self.p, self.x[l], q["w_off"], q["b_off"], q["w"], None, self.y[l],
                              self.off[l], None, self.ws[l])
            out = self.z[l] if self.pointwise else self.x[l + 1]
            B.dc_group_norm_fwd(self.norm[l], self.y[l], q["gamma"], q["beta"], out, *self.stats[l], self.norm_ws)
            if self.pointwise:
                self.pointwise[l].load(q["w_pw"])
                self.pointwise[l].forward(out, self.x[l + 1])
        return self.x[-1]

    def backward(self, grad_out):
        """Gradients of sum(output * grad_out) into ``self.grads``; returns the
        input's (float32)."""
        grad = grad_out
        for l in reversed(range(self.L)):
            q, g = self.params[l], self.grads[l]
            if self.pointwise:
                grad, _ = self.pointwise[l].backward(grad, self.gz, g["w_pw"])
            B.dc_group_norm_bwd(self.norm[l], self.y[l], q["gamma"], q["beta"], *self.stats[l], grad,
                                self.gy, g["gamma"], g["beta"], self.norm_ws)
            B.deform_conv_bwd(self.p, self.x[l], q["w_off"], q["w"], self.off[l], self.gy, self.gx,
                              g["w_off"], g["b_off"], g["w"], None, self.ws[l], after_fwd=True)
            grad = self.gx
        return self.gx

    def _norm(self, max_norm, norm, scale):
        """One norm over both optimisers' gradients, those that their next steps take."""
        if self.muon is None:
            return self.opt.grad_norm(max_norm, norm, scale)
        tables = self.opt.params, self.muon.params  # (new ones after a set_grads)
        if any(a is not b for a, b in zip(self._tables, tables)):
            self._tables = tables
            self._both.set_grads(self._both_grads())
        return self._both(max_norm, norm, scale)

    def _both_grads(self):
        return [q["grad"] for table in self._tables for q in table]

    def update(self):
        """The clipped step; the norm stays in ``self.grad_norm``.  A norm that is
        not finite leaves every parameter as it is."""
        self._norm(self.max_norm, self.grad_norm, self.clip)
        self.opt.step(self.clip)
        if self.muon is not None:
            self.muon.step(self.clip)


def initial_params(p: B.Problem, layers, seed=0, device="cuda", pointwise=False):
    """He-initialised main weights, small offset weights, unit norms (and
    orthogonal pointwise weights)."""
    gen = torch.Generator().manual_seed(seed)
    s, dt, out = p.shapes(), p.torch_dtype, []
    fan = p.c_in * p.kh * p.kw
    for _ in range(layers):
        q = dict(w_off=(torch.randn(s["w_off"], generator=gen) * 0.5 / fan ** 0.5).to(dt),
                 b_off=torch.zeros(s["b_off"]),
                 w=(torch.randn(s["w"], generator=gen) * (2.0 / fan) ** 0.5).to(dt),
                 gamma=torch.ones(p.c_out), beta=torch.zeros(p.c_out))
        if pointwise:
            q["w_pw"] = torch.linalg.qr(torch.randn(p.c_out, p.c_out, generator=gen))[0].contiguous().to(dt)
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
    ap.add_argument("--optimizer", choices=("adamw", "muon"), default="adamw")
    ap.add_argument("--pointwise", action="store_true", help="a pointwise layer in 8 bits behind each activation")
    a = ap.parse_args(argv)
    p = B.Problem(a.batch, a.channels, a.size, a.size, a.channels, dtype=B.DC_BF16)
    teacher, student = (initial_params(p, a.layers, seed, pointwise=a.pointwise) for seed in (1, 2))
    teacher = Trainer(p, teacher, groups=8)
    student = Trainer(p, student, groups=8, state_bits=a.state_bits, optimizer=a.optimizer)
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
