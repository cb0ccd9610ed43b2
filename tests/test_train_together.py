"""Both optimisers of a training step at once: their gradients' norm, whole steps
captured and replayed, gradients of the pointwise and norm parameters against
differences of a loss (GPU)."""
import pytest
import torch

from deformable_convolution_gb300 import binding as B
from deformable_convolution_gb300 import train as T

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


def trainer(dtype=B.DC_F32, layers=1, n=2, c=64, size=12, seed=3, **kw):
    p = B.Problem(n, c, size, size, c, dtype=dtype)
    params = T.initial_params(p, layers, seed=seed, pointwise=True)
    return p, params, T.Trainer(p, params, groups=8, act=B.DC_ACT_SILU, optimizer="muon", **kw)


def data(p, gen):
    return [torch.randn(p.shapes()[k], generator=gen).to(p.torch_dtype).cuda() for k in ("x", "y")]


def norm_of(tensors):
    return sum(float((t.double() ** 2).sum()) for t in tensors) ** 0.5


@pytest.mark.parametrize("which", ("muon", "opt", "both"))
def test_the_norm_is_that_of_the_gradients_that_are_stepped_with(which):
    """Gradients at other addresses (averages over replicas, say), handed to
    either optimiser: the norm and the clip factor follow."""
    p, params, tr = trainer(max_norm=0.5, lr=1e-2)
    x, g = data(p, torch.Generator().manual_seed(1))
    tr.forward(x)
    tr.backward(g)
    tr.update()
    for opt, factor in ((tr.muon, 3.0), (tr.opt, 5.0)):
        if which == "both" or opt is getattr(tr, which):
            opt.set_grads([q["grad"] * factor for q in opt.params])
    tr.forward(x)
    tr.backward(g)
    tr.update()
    want = norm_of([q["grad"] for opt in (tr.muon, tr.opt) for q in opt.params])
    assert abs(float(tr.grad_norm) - want) <= 1e-5 * want
    assert abs(float(tr.clip) - 0.5 / (want + 1e-6)) <= 1e-5 * float(tr.clip)


def test_a_captured_step_of_both_optimisers_follows_single_ones():
    """Forward, backward, norm, Muon and AdamW in one graph, replayed with other
    data, learning rates and bias corrections from the device, beside the same
    calls one by one."""
    runs = [trainer(B.DC_BF16, lr=1e-2, seed=9) for _ in range(2)]
    gen = torch.Generator().manual_seed(11)
    p, single, tr = runs[0]
    _, replayed, captured = runs[1]
    steps = [data(p, gen) for _ in range(3)]
    start = [{k: v.float().clone() for k, v in q.items()} for q in single]
    x, g = (t.clone() for t in steps[0])
    schedule, lr = torch.zeros(3, device="cuda"), torch.zeros(1, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        captured.forward(x)
        captured.backward(g)
        captured._norm(captured.max_norm, captured.grad_norm, captured.clip)
        captured.opt.step(captured.clip, schedule=schedule)
        captured.muon.step(captured.clip, lr=lr)
    for k, (a, b) in enumerate(steps):
        tr.opt.lr = tr.muon.lr = 1e-2 / (1 + k)
        tr.forward(a)
        tr.backward(b)
        tr.update()
        schedule.copy_(captured.opt.schedule(step=k + 1, lr=1e-2 / (1 + k)))
        lr.fill_(1e-2 / (1 + k))
        x.copy_(a)
        g.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        assert abs(float(captured.grad_norm) - float(tr.grad_norm)) <= 1e-2 * float(tr.grad_norm)
    for q, r, s in zip(single, replayed, start):
        for k in q:
            moved, apart = q[k].float() - s[k], q[k].float() - r[k].float()
            # every parameter has moved; the layer's backward adds with atomics, whose order moves last bits of the weight's
            # gradients: bf16 values of the chain flip by 2^-8 at most, its quotients and directions with them
            assert float(moved.norm()) > 0.0 and float(apart.norm()) <= 0.05 * float(moved.norm()), k


def test_gradients_against_differences_of_the_loss():
    """(L(q + h d) - L(q - h d)) / 2 against h times the gradient along d, for d the
    gradient itself, L = sum(output * g) as the layer computes it.

    L moves by h |grad|^2 each way.  The forward's codes are off by at most 2^-4 of
    a value, at random 2^-4 / sqrt(3): of L that is the root of the sum over the
    products w z g of their squares (each of both factors' codes), times sqrt(2) for
    two evaluations, over 2 for the difference; four of these are allowed, and the
    gradient's own codes 2 * 2^-4 of it.  h is a tenth of the parameter's size: for
    gamma and beta, whose L bends, the third derivative's share stays below 2 %."""
    p, params, tr = trainer(n=8, size=16)
    q = params[0]
    x, g = data(p, torch.Generator().manual_seed(6))
    tr.forward(x)
    tr.backward(g)
    grads = {k: tr.grads[0][k].clone() for k in ("w_pw", "gamma", "beta")}
    z = tr.z[0].flatten(2).double()
    gz = g.flatten(2).double()
    products = float(((q["w_pw"].double() ** 2) @ (z ** 2) * gz ** 2).sum()) ** 0.5
    noise = 2 * 2.0 ** -4 / 3 ** 0.5 * products * 2 ** 0.5 / 2

    def loss():
        return float((tr.forward(x).double() * g.double()).sum())
    for k, d in grads.items():
        size = max(float(q[k].float().norm()), 0.5 * d.numel() ** 0.5 if k == "beta" else 0.0)
        h = 0.1 * size / float(d.norm())
        kept = q[k].clone()
        q[k].copy_(kept + h * d)
        up = loss()
        q[k].copy_(kept - h * d)
        down = loss()
        q[k].copy_(kept)
        want = h * float(d.double().square().sum())
        assert abs((up - down) / 2 - want) <= 4 * noise + (2 * 2.0 ** -4 + 0.02) * want, k
        assert want > 8 * noise, f"{k}: the difference says nothing"
