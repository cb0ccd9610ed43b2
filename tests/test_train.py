"""A training step over deformable layers with group norm between them: the
chain against the 64-bit oracle and the plain forms, and that it learns (GPU)."""
import numpy as np
import pytest
import torch

import norm_plain as P
import oracle
from deformable_convolution_gb300 import binding as B
from deformable_convolution_gb300 import train as T

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


def f64(t):
    return t.detach().cpu().double().numpy()


def oracle_step(p, np_problem, params, x0, grad_out):
    """Output and gradients of the chain in 64 bits (offsets rounded to float32
    for the backward, as the layer's are)."""
    op = oracle.Problem(p.n, p.c_in, p.h, p.w, p.c_out, p.kh, p.kw, p.stride, p.pad, p.dil, p.offset_groups)
    x, saved = f64(x0), []
    for q in params:
        y, off = oracle.forward(op, x, f64(q["w_off"]), f64(q["b_off"]), f64(q["w"]), None)
        yt = torch.from_numpy(np.ascontiguousarray(y))
        f = P.forward(np_problem, yt, q["gamma"].cpu(), q["beta"].cpu())
        saved.append((x, yt, off, f))
        x = f["y"].contiguous().numpy()
    out, grad, grads = x, torch.from_numpy(f64(grad_out)), []
    for q, (x, yt, off, f) in zip(reversed(params), reversed(saved)):
        g = P.backward(np_problem, yt, q["gamma"].cpu(), q["beta"].cpu(), f["mean"], f["rstd"], grad)
        off32 = off.astype(np.float32).astype(np.float64)
        r = oracle.backward(op, x, f64(q["w_off"]), f64(q["w"]), off32, g["grad_x"].contiguous().numpy())
        grads.append(dict(w=r["grad_w"], w_off=r["grad_w_off"], b_off=r["grad_b_off"],
                          gamma=g["grad_gamma"].numpy(), beta=g["grad_beta"].numpy()))
        grad = torch.from_numpy(np.ascontiguousarray(r["grad_x"]))
    return out, grads[::-1], grad.numpy()


def test_step_matches_the_oracle_chain():
    p = B.Problem(2, 16, 12, 12, 16)
    params = T.initial_params(p, 2, seed=3)
    tr = T.Trainer(p, params, groups=4, act=B.DC_ACT_SILU, lr=1e-2, max_norm=0.5)
    gen = torch.Generator().manual_seed(5)
    x0, grad_out = (torch.randn(p.shapes()[k], generator=gen).cuda() for k in ("x", "y"))
    before = [{k: v.clone() for k, v in q.items()} for q in params]
    out = tr.forward(x0).clone()
    gx = tr.backward(grad_out).clone()
    want_out, want, want_gx = oracle_step(p, tr.norm[0], params, x0, grad_out)

    def close(a, b, tol):
        assert np.max(np.abs(f64(a) - b)) <= tol * np.max(np.abs(b))
    # each layer is good to 1e-4 of its maximum (the layer's own bar); two of
    # them, each passed on by slopes and norms of order one, and the gradients
    # taken at activations that far off: an order of magnitude
    close(out, want_out, 1e-3)
    close(gx, want_gx, 1e-3)
    for g, w in zip(tr.grads, want):
        for k in w:
            close(g[k], w[k], 1e-3)

    # the update: the formula in 64 bits on the gradients found
    tr.update()
    norm = np.sqrt(sum(float((g[k].double() ** 2).sum()) for g in tr.grads for k in g))
    assert abs(float(tr.grad_norm) - norm) <= 1e-5 * norm
    scale = min(1.0, 0.5 / (norm + 1e-6))
    for q, old, g in zip(params, before, tr.grads):
        for k in g:
            v = g[k].double() * scale
            wd = 0.01 if k in ("w", "w_off") else 0.0
            new = old[k].double() * (1 - 1e-2 * wd) - 1e-2 * v / (v.abs() + 1e-8)
            # the first step is lr times a quotient of order one: 1e-5 of lr, but
            # where the gradient is so small that eps counts
            tol = 1e-5 * 1e-2 + 4e-7 * old[k].double().abs() + (v.abs() < 1e-6).double() * 1e-2
            assert ((q[k].double() - new).abs() <= tol).all(), k


@pytest.mark.parametrize("bits", (32, 8))
def test_bf16_stack_learns(bits):
    losses = T.main(["--steps", "60", "--layers", "2", "--channels", "64", "--size", "16", "--batch", "4",
                     "--state-bits", str(bits)])
    assert all(np.isfinite(losses))
    # (60 steps of 1e-3: the loss falls well below its start; no precise figure is claimed)
    assert np.mean(losses[-5:]) < 0.8 * np.mean(losses[:5])


def test_a_gradient_that_is_not_finite_leaves_the_parameters():
    p = B.Problem(1, 64, 8, 8, 64, dtype=B.DC_BF16)
    params = T.initial_params(p, 1, seed=4)
    tr = T.Trainer(p, params, groups=8)
    x = torch.randn(p.shapes()["x"], device="cuda").to(torch.bfloat16)
    g = torch.randn(p.shapes()["y"], device="cuda").to(torch.bfloat16)
    g[0, 0, 0, 0] = float("inf")
    old = [{k: v.clone() for k, v in q.items()} for q in params]
    tr.forward(x)
    tr.backward(g)
    tr.update()
    assert not np.isfinite(float(tr.grad_norm))
    for q, o in zip(params, old):
        assert all(torch.equal(q[k], o[k]) for k in q)


@pytest.mark.parametrize("bits", (32, 8))
def test_a_saved_state_resumes_bit_for_bit(bits):
    p = B.Problem(2, 64, 8, 8, 64, dtype=B.DC_BF16)
    first, again = (T.Trainer(p, T.initial_params(p, 2, seed=s), groups=8, state_bits=bits) for s in (5, 6))
    gen = torch.Generator().manual_seed(7)
    x, g = (torch.randn(p.shapes()[k], generator=gen).to(torch.bfloat16).cuda() for k in ("x", "y"))

    def step(tr):
        tr.forward(x)
        tr.backward(g)
        tr.update()
    for _ in range(3):
        step(first)
    for q, r in zip(first.params, again.params):
        for k in q:
            r[k].copy_(q[k])
    again.opt.load_state_dict(first.opt.state_dict())
    for _ in range(3):
        # the layer's weight gradients are sums in an order of their own: the update's input is made the same
        for tr in (first, again):
            tr.forward(x)
            tr.backward(g)
        for a, b in zip(first.grads, again.grads):
            for k in a:
                b[k].copy_(a[k])
        first.update(), again.update()
        for q, r in zip(first.params, again.params):
            assert all(torch.equal(q[k], r[k]) for k in q)
    for q, r in zip(first.opt.params, again.opt.params):
        if q.get("master") is not None:
            assert torch.equal(q["master"], r["master"])
