"""Both optimisers of a training step at once: the norm of their gradients (GPU)."""
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
