"""AdamW, Muon and gradient clipping over all parameters of a network at once.

Marshalling only: the optimiser keeps a host table of its tensors' pointers
(``binding.adamw_tensors``) and hands it to the library, which updates every
tensor in one launch; the gradient norm and the factor that clips it stay on
the device.  The update and the 8-bit state code are defined in
``include/deform_conv.h``.
"""
from __future__ import annotations

from types import MappingProxyType

import torch

from . import binding as B


class GradNorm:
    """Global norm of a list of gradients (float32 or bfloat16 CUDA tensors),
    and the factor that clips it.  Their addresses are taken here and by
    ``set_grads``.  The object keeps one workspace: its calls belong on one
    stream, or on streams that wait for one another."""

    def __init__(self, grads):
        self._set(grads)
        device = self.grads[0].device if self.grads else "cuda"
        need = B.dc_grad_norm_workspace_size(len(self.grads))
        self._ws = torch.empty(max(need, 1), dtype=torch.uint8, device=device)

    def _set(self, grads):
        grads = tuple(grads)
        self._table = B.adamw_tensors([dict(grad=g) for g in grads])
        self.grads = grads

    def set_grads(self, grads):
        """Other gradients, as many as there were."""
        grads = tuple(grads)
        if len(grads) != len(self.grads):
            raise ValueError(f"expected {len(self.grads)} gradients, got {len(grads)}")
        if any(g is None for g in grads):
            raise ValueError("a gradient is missing")
        self._set(grads)

    def __call__(self, max_norm, norm, scale, stream=None):
        """norm, scale: one-element float32 tensors (or None)."""
        B.dc_grad_norm(self._table, len(self.grads), max_norm, norm, scale, self._ws, stream)


class StateValues:
    """Writes an optimiser's states as float32 values into ``out``: per tensor
    an (m, v) pair of float32 tensors, either of which may be None."""

    def __init__(self, opt, out):
        self.opt, self.out = opt, tuple(tuple(pair) for pair in out)
        if len(self.out) != len(opt.params):
            raise ValueError(f"expected {len(opt.params)} pairs, got {len(self.out)}")
        shapes = [tuple(q["param"].shape) for q in opt.params]
        self._m, self._v = (B.pointers([pair[k] for pair in self.out], name, shapes, torch.float32)
                            for k, name in enumerate(("m", "v")))

    def __call__(self, stream=None):
        B.dc_adamw_state_values(self.opt._table, len(self.out), self._m, self._v, stream)


class AdamW:
    """AdamW over ``params``: dicts with

      param    float32 or bfloat16 CUDA tensor, updated in place
      grad     float32 or bfloat16 tensor of its shape, read by every step
      master   optional float32 tensor that a bfloat16 ``param`` is a rounded
               copy of: the update is made there
      weight_decay   optional, else the optimiser's
      m, v (m_scale, v_scale)   optional state tensors, else made here (zeros)

    state_bits: 32 (float32 states) or 8 (int8 m, uint8 v and a float32 scale
    for each 256 elements; tensors below ``min_8bit`` elements keep float32
    states).  step: steps already taken.

    The optimiser reads and writes its tensors by the addresses they have when
    it is made; ``params`` is therefore read-only, and gradients that autograd
    allocates anew are handed over by ``set_grads``."""

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01,
                 state_bits=32, min_8bit=0, step=0):
        if state_bits not in (8, 32):
            raise ValueError("state_bits must be 8 or 32")
        entries = []
        for q in params:
            q = dict(q)
            q.setdefault("weight_decay", weight_decay)
            p = q["param"]
            if q.get("m") is None:
                eight = state_bits == 8 and p.numel() >= min_8bit
                q["m"] = torch.zeros(p.shape, dtype=torch.int8 if eight else torch.float32,
                                     device=p.device)
                q["v"] = torch.zeros(p.shape, dtype=torch.uint8 if eight else torch.float32,
                                     device=p.device)
                if eight:
                    blocks = -(-p.numel() // B.STATE_BLOCK)
                    q["m_scale"], q["v_scale"] = (torch.zeros(blocks, device=p.device)
                                                  for _ in range(2))
            entries.append(q)
        self._hyper = B.DcAdamwHyper(lr, betas[0], betas[1], eps, step)
        self._norm = None
        self._set(entries)

    def _set(self, entries):
        self._table = B.adamw_tensors(entries)
        self.params = tuple(MappingProxyType(q) for q in entries)

    def set_grads(self, grads):
        """Other gradients for the next steps and norms, one for each parameter."""
        grads = tuple(grads)
        if len(grads) != len(self.params):
            raise ValueError(f"expected {len(self.params)} gradients, got {len(grads)}")
        if any(g is None or g.shape != q["param"].shape for g, q in zip(grads, self.params)):
            raise ValueError("a gradient is missing or of another shape than its parameter")
        self._set([dict(q, grad=g) for q, g in zip(self.params, grads)])
        if self._norm is not None:
            self._norm.set_grads(grads)

    @property
    def step_count(self):
        return self._hyper.step

    @property
    def lr(self):
        return self._hyper.lr

    @lr.setter
    def lr(self, value):
        self._hyper.lr = value

    def grad_norm(self, max_norm, norm=None, scale=None, stream=None):
        """The gradients' global norm and the factor that clips it to max_norm
        (for ``step``): one-element device tensors, made here if not given."""
        if self._norm is None:
            self._norm = GradNorm([q["grad"] for q in self.params])
        device = self._norm._ws.device
        norm = torch.empty(1, device=device) if norm is None else norm
        scale = torch.empty(1, device=device) if scale is None else scale
        self._norm(max_norm, norm, scale, stream)
        return norm, scale

    def step(self, grad_scale=None, schedule=None, stream=None):
        """One step with the gradients times grad_scale (a device scalar; a
        step whose scale is not finite changes no tensor, and counts).
        schedule: see ``schedule``."""
        self._hyper.step += 1
        try:
            B.dc_adamw_step(self._table, len(self.params), self._hyper, grad_scale, schedule, stream)
        except Exception:
            self._hyper.step -= 1
            raise

    def schedule(self, step=None, lr=None):
        """Host float32 [3] {lr, 1 - beta1^step, 1 - beta2^step} for the next
        step (or the given one): what a replayed CUDA graph's ``step(schedule=
        device copy)`` reads."""
        h = self._hyper
        t = h.step + 1 if step is None else step
        return torch.tensor([h.lr if lr is None else lr, 1.0 - h.beta1 ** t, 1.0 - h.beta2 ** t])

    def state_values(self, stream=None):
        """[(m, v)] of every tensor as new float32 tensors."""
        out = [tuple(torch.empty(q["param"].shape, device=q["param"].device) for _ in range(2))
               for q in self.params]
        StateValues(self, out)(stream)
        return out

    def state_dict(self):
        """The state as tensors (not copies): for saving between steps.  The
        masters are part of it: a bfloat16 ``param`` lacks their low bits."""
        keys = ("m", "v", "m_scale", "v_scale", "master")
        return dict(step=self._hyper.step, lr=self._hyper.lr,
                    state=[{k: q[k] for k in keys if q.get(k) is not None} for q in self.params])

    def load_state_dict(self, d):
        """Copies a ``state_dict`` of the same parameters into this state.  A
        parameter with a master becomes its rounded copy; a state that holds no
        masters leaves both as they are."""
        if len(d["state"]) != len(self.params):
            raise ValueError("state of another number of tensors")
        for q, s in zip(self.params, d["state"]):
            for k in ("m", "v", "m_scale", "v_scale", "master"):
                a, b = q.get(k), s.get(k)
                if b is None and k == "master":
                    continue
                if (a is None) != (b is None) or (a is not None and (a.dtype != b.dtype or a.shape != b.shape)):
                    raise ValueError(f"state {k} of another kind or shape")
        for q, s in zip(self.params, d["state"]):
            for k, t in s.items():
                q[k].copy_(t)
            if s.get("master") is not None:
                q["param"].copy_(q["master"])
        self._hyper.step, self._hyper.lr = d["step"], d["lr"]


class Orthogonalize:
    """Writes the matrices ``ins`` (float32 or bfloat16 CUDA tensors, the first
    dimension by all others) orthogonalised into ``outs`` (either type; a tensor
    may be both) by ``steps`` Newton-Schulz steps.  precision: 16, where X's
    products take its high 16 bits only (errors below a bfloat16's rounding, also
    for float32 results), or 32.

    Addresses are taken here.  The object keeps one workspace, about 8 to 16
    bytes a value of up to 40 matrices: its calls belong on one stream, or on streams that
    wait for one another."""

    def __init__(self, ins, outs, steps=5, precision=16):
        self.ins, self.outs = tuple(ins), tuple(outs)
        self._table = B.matrices(self.ins, self.outs)
        self._how = steps, _precision(precision)
        self._ws = _bytes(B.dc_orthogonalize_workspace_size(self._table, len(self.ins)), self.ins)

    def __call__(self, stream=None):
        B.dc_orthogonalize(self._table, len(self.ins), *self._how, self._ws, stream)


def _precision(bits):
    if bits not in (16, 32):
        raise ValueError("precision must be 16 or 32")
    return B.DC_ORTHO_16 if bits == 16 else B.DC_ORTHO_32


def _bytes(count, like):
    return torch.empty(max(count, 1), dtype=torch.uint8, device=like[0].device if like else "cuda")


class Muon:
    """Muon over ``params``, weights of two dimensions or more (a matrix: the
    first by all others): dicts as AdamW's, with

      m        optional momentum, float32, else made here (zeros)
      rate     optional factor on lr, else rms * sqrt(the longer side): a step
               of AdamW's usual size for rms = 0.2

    and param, grad, master, weight_decay as there.  precision: of the
    orthogonalisation (see ``Orthogonalize``).  Biases, norms' parameters and
    other vectors belong to AdamW.  As there, ``params`` is read-only and
    ``set_grads`` hands over gradients at other addresses.  The workspace is
    ``Orthogonalize``'s (40 weights of 2048 x 2048: 2.7 GB, as long as the object)."""

    def __init__(self, params, lr=1e-3, momentum=0.95, nesterov=True, weight_decay=0.01, steps=5,
                 rms=0.2, precision=16):
        entries = []
        for q in params:
            q = dict(q)
            q.setdefault("weight_decay", weight_decay)
            if q.get("rate") is None:
                q["rate"] = rms * max(B._matrix_shape(q["param"], "param")) ** 0.5
            if q.get("m") is None:
                q["m"] = torch.zeros(q["param"].shape, device=q["param"].device)
            entries.append(q)
        self._hyper = B.DcMuonHyper(lr, momentum, int(bool(nesterov)), steps, _precision(precision))
        self._set(entries)
        self._ws = _bytes(B.dc_muon_workspace_size(self._table, len(entries)),
                          [q["param"] for q in entries])

    def _set(self, entries):
        self._table = B.muon_tensors(entries)
        self.params = tuple(MappingProxyType(q) for q in entries)

    def set_grads(self, grads):
        """Other gradients for the next steps, one for each parameter."""
        grads = tuple(grads)
        if len(grads) != len(self.params):
            raise ValueError(f"expected {len(self.params)} gradients, got {len(grads)}")
        if any(g is None or g.shape != q["param"].shape for g, q in zip(grads, self.params)):
            raise ValueError("a gradient is missing or of another shape than its parameter")
        self._set([dict(q, grad=g) for q, g in zip(self.params, grads)])

    @property
    def lr(self):
        return self._hyper.lr

    @lr.setter
    def lr(self, value):
        self._hyper.lr = value

    def step(self, grad_scale=None, lr=None, stream=None):
        """One step with the gradients times grad_scale (a device scalar; a step
        whose scale is not finite changes no tensor).  lr: a device scalar that
        takes the place of ``self.lr`` (for a replayed CUDA graph)."""
        B.dc_muon_step(self._table, len(self.params), self._hyper, grad_scale, lr, self._ws, stream)

    def state_dict(self):
        """The state as tensors (not copies), the masters among it."""
        return dict(lr=self._hyper.lr, state=[{k: q[k] for k in ("m", "master") if q.get(k) is not None}
                                              for q in self.params])

    def load_state_dict(self, d):
        """Copies a ``state_dict`` of the same parameters into this state.  A
        parameter with a master becomes its rounded copy; a state that holds no
        masters leaves both as they are."""
        if len(d["state"]) != len(self.params):
            raise ValueError("state of another number of tensors")
        for q, s in zip(self.params, d["state"]):
            for k in ("m", "master"):
                a, b = q.get(k), s.get(k)
                if b is None and k == "master":
                    continue
                if (a is None) != (b is None) or (a is not None and (a.dtype != b.dtype or a.shape != b.shape)):
                    raise ValueError(f"state {k} of another kind or shape")
        for q, s in zip(self.params, d["state"]):
            for k, t in s.items():
                q[k].copy_(t)
            if s.get("master") is not None:
                q["param"].copy_(q["master"])
        self._hyper.lr = d["lr"]
