"""Training steps with pointwise layers in 8 bits and Muon: the operators in the
order that a step runs them, against the formulas (GPU)."""
import pytest
import torch

import matrix_plain as P
import norm_plain
from deformable_convolution_gb300 import binding as B
from deformable_convolution_gb300 import fp8
from deformable_convolution_gb300 import train as T

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

WEIGHTS = ("w", "w_off", "w_pw")


def trainer(dtype=B.DC_F32, layers=2, seed=3, optimizer="muon", n=2, c=16, size=12, groups=4, **kw):
    p = B.Problem(n, c, size, size, c, dtype=dtype)
    params = T.initial_params(p, layers, seed=seed, pointwise=True)
    return p, params, T.Trainer(p, params, groups=groups, act=B.DC_ACT_SILU, optimizer=optimizer, **kw)


@pytest.mark.parametrize("dtype", (B.DC_F32, B.DC_BF16))
def test_pointwise_layers_in_the_chain(dtype):
    """Each pointwise layer's output and gradients from what its neighbours left
    in the step's buffers, by the quantised formula in 64 bits."""
    p, params, tr = trainer(dtype, c=64, groups=8)
    gen = torch.Generator().manual_seed(5)
    x0, grad_out = (torch.randn(p.shapes()[k], generator=gen).to(p.torch_dtype).cuda() for k in ("x", "y"))
    out = tr.forward(x0).clone()
    z = [t.clone() for t in tr.z]
    xs = [t.clone() for t in tr.x[1:]]
    tr.backward(grad_out)
    half = 2.0 ** -8 if dtype == B.DC_BF16 else 0.0
    c, hw = p.c_out, p.ho * p.wo
    for l in range(tr.L):
        w = P.quantize(params[l]["w_pw"][None], 0, True)[0][0]
        zq = P.quantize(z[l].flatten(2).transpose(1, 2), 0, False)[0].transpose(1, 2)
        want, size = w @ zq, w.abs() @ zq.abs()
        got = xs[l].flatten(2).cpu().double()
        # float32 sums of c exact products, rounded to the dtype
        assert ((got - want).abs() <= size * c * 2.0 ** -23 + want.abs() * half).all()
    assert torch.equal(out, xs[-1])
    # the top layer's gradients
    gq = P.quantize(grad_out.flatten(2), 0, False)[0]
    zq = P.quantize(z[-1].flatten(2), 0, False)[0]
    want, size = (gq @ zq.transpose(1, 2)).sum(0), (gq.abs() @ zq.abs().transpose(1, 2)).sum(0)
    assert ((tr.grads[-1]["w_pw"].cpu().double() - want).abs() <= size * p.n * hw * 2.0 ** -23).all()


def test_gradients_of_the_stack_against_differences():
    """One layer's loss sum(output * grad_out) in the directions of the pointwise
    and the norm's parameters.  The forward quantises to 3 mantissa bits, so its
    steps are averaged: a difference over many directions at once, against the
    gradient's own prediction, both off by the codes' relative error of 2^-4 at
    most a value, independent over the 64 x 144 x 2 values that the loss sums."""
    p, params, tr = trainer(layers=1, c=64, groups=8)
    gen = torch.Generator().manual_seed(6)
    x0, g = (torch.randn(p.shapes()[k], generator=gen).cuda() for k in ("x", "y"))
    tr.forward(x0)
    tr.backward(g)
    # the plain chain behind the convolution in 64 bits, not quantised: the norm, SiLU and the product
    y = tr.y[0].cpu().double()
    w, gamma, beta = (params[0][k].cpu().double() for k in ("w_pw", "gamma", "beta"))
    f = norm_plain.forward(tr.norm[0], y, gamma, beta)
    z = f["y"].flatten(2)
    gw = (g.cpu().double().flatten(2) @ z.transpose(1, 2)).sum(0)
    gz = (w.T @ g.cpu().double().flatten(2)).view(y.shape)
    back = norm_plain.backward(tr.norm[0], y, gamma, beta, f["mean"], f["rstd"], gz)
    for got, want in ((tr.grads[0]["w_pw"], gw), (tr.grads[0]["gamma"], back["grad_gamma"]), (tr.grads[0]["beta"], back["grad_beta"])):
        # each factor of each product is off by 2^-4 of itself at most, 2^-4 / sqrt(3) as a rule: two factors, summed at
        # random over 288 pixels (64 channels), and the sums' own terms at random: 2 * 2^-4 / sqrt(3) of the sum's size
        assert float((got.cpu().double() - want).norm() / want.norm()) <= 2 * 2.0 ** -4


def test_steps_match_the_formulas():
    """Gradient norm, Muon for the weights and AdamW for the rest, by the
    formulas in 64 bits on the gradients found."""
    p, params, tr = trainer(lr=1e-2, max_norm=0.5)
    gen = torch.Generator().manual_seed(7)
    x0, g = (torch.randn(p.shapes()[k], generator=gen).cuda() for k in ("x", "y"))
    before = [{k: v.clone() for k, v in q.items()} for q in params]
    tr.forward(x0)
    tr.backward(g)
    tr.update()
    norm = sum(float((t.double() ** 2).sum()) for q in tr.grads for t in q.values()) ** 0.5
    assert abs(float(tr.grad_norm) - norm) <= 1e-5 * norm
    scale = float(tr.clip)
    assert abs(scale - min(1.0, 0.5 / (norm + 1e-6))) <= 1e-5 * scale
    assert len(tr.muon.params) == 3 * tr.L and len(tr.opt.params) == 3 * tr.L
    for q, old, g in zip(params, before, tr.grads):
        for k in g:
            got = q[k].cpu().double()
            if k in WEIGHTS:
                rows = old[k].shape[0]
                rate = 0.2 * max(rows, old[k].numel() // rows) ** 0.5
                want, _ = P.muon(old[k], torch.zeros_like(old[k]), g[k], scale, 1e-2, 0.95, True, 0.01, rate)
                # precision 16, relative error 4.2e-3 of the direction's norm at most (1.21 * sqrt(short side))
                tol = 1e-2 * rate * 4.2e-3 * 1.21 * min(rows, old[k].numel() // rows) ** 0.5
                assert float((got - want).norm()) <= tol + 1e-6
            else:
                v = g[k].cpu().double() * scale
                want = old[k].cpu().double() - 1e-2 * v / (v.abs() + 1e-8)
                # AdamW's first step: lr times a quotient of order one, but where the gradient is so small that eps counts
                tol = 1e-5 * 1e-2 + 4e-7 * old[k].cpu().double().abs() + (v.abs() < 1e-6).double() * 1e-2
                assert ((got - want).abs() <= tol).all(), k


def test_a_gradient_that_is_not_finite_leaves_the_parameters():
    p, params, tr = trainer(B.DC_BF16, layers=1, c=64, groups=8)
    x, g = (torch.randn(p.shapes()[k], device="cuda").to(torch.bfloat16) for k in ("x", "y"))
    g[0, 0, 0, 0] = float("inf")
    old = [{k: v.clone() for k, v in q.items()} for q in params]
    tr.forward(x)
    tr.backward(g)
    tr.update()
    assert not torch.isfinite(tr.grad_norm).item()
    for q, o in zip(params, old):
        assert all(torch.equal(q[k], o[k]) for k in q)


def test_a_captured_step_follows_single_ones():
    """Forward, backward and update of a stack in a graph, replayed, beside the
    same calls one by one."""
    runs = [trainer(B.DC_BF16, c=64, size=8, groups=8, seed=9) for _ in range(2)]
    gen = torch.Generator().manual_seed(11)
    p = runs[0][0]
    data = [[torch.randn(p.shapes()[k], generator=gen).to(torch.bfloat16).cuda() for k in ("x", "y")] for _ in range(3)]
    x, g = (t.clone() for t in data[0])
    _, single, tr = runs[0]
    _, replayed, captured = runs[1]
    before = [{k: v.clone() for k, v in q.items()} for q in replayed]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        captured.forward(x)
        captured.backward(g)
        captured._norm(captured.max_norm, captured.grad_norm, captured.clip)
        captured.muon.step(captured.clip)
    assert all(torch.equal(q[k], b[k]) for q, b in zip(replayed, before) for k in q)
    for a, b in data:
        tr.forward(a)
        tr.backward(b)
        tr._norm(tr.max_norm, tr.grad_norm, tr.clip)
        tr.muon.step(tr.clip)
        x.copy_(a)
        g.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
    for q, r in zip(single, replayed):
        for k in WEIGHTS:
            # the layer's own backward adds with atomics, whose order moves last bits
            d = (q[k].float() - r[k].float()).abs()
            assert float(d.max()) <= 0.1 * float(q[k].float().abs().max())
        assert torch.equal(q["gamma"], r["gamma"])


@pytest.mark.parametrize("argv", [["--optimizer", "muon"], ["--pointwise"], ["--optimizer", "muon", "--pointwise"]])
def test_the_example_runs(argv):
    losses = T.main(["--steps", "12", "--layers", "2", "--channels", "64", "--size", "12", "--batch", "2"] + argv)
    assert all(v == v and abs(v) < 1e30 for v in losses)


def test_refusals():
    p = B.Problem(1, 16, 8, 8, 16)
    with pytest.raises(ValueError):
        T.Trainer(p, T.initial_params(p, 1), groups=4, optimizer="sgd")
    mixed = T.initial_params(p, 1) + T.initial_params(p, 1, pointwise=True)
    with pytest.raises(ValueError):
        T.Trainer(p, mixed, groups=4)


def test_a_layer_and_its_optimiser_together():
    """A pointwise layer trained alone, as a user's loop runs it: codes of the
    weight, forward, backward, Muon, codes of the new weight."""
    gen = torch.Generator().manual_seed(1)
    w = (torch.randn(96, 128, generator=gen) * 0.1).bfloat16().cuda()
    master, grad = w.float(), torch.empty(96, 128, device="cuda")
    from deformable_convolution_gb300 import optim
    layer = fp8.Pointwise(2, 128, 96, 9, 11, B.DC_BF16, B.DC_NHWC)
    opt = optim.Muon([dict(param=w, master=master, grad=grad)], lr=1e-2, precision=32)
    m = torch.zeros(96, 128)
    for step in range(3):
        x = torch.randn(layer.x_shape, generator=gen).bfloat16().cuda()
        gy = torch.randn(layer.y_shape, generator=gen).bfloat16().cuda()
        layer.load(w)
        layer.forward(x)
        layer.backward(gy, grad_w=grad)
        xq, gq = (P.quantize(t.reshape(1, -1, t.shape[3]).transpose(1, 2), 0, False)[0][0] for t in (x, gy))
        want = gq @ xq.T
        size = gq.abs() @ xq.abs().T
        assert ((grad.cpu().double() - want).abs() <= size * 198 * 2.0 ** -23).all()
        old = master.clone()
        opt.step()
        new, m = P.muon(old, m, grad, 1.0, 1e-2, 0.95, True, 0.01, 0.2 * 128 ** 0.5)
        assert float((master.cpu().double() - new).abs().max()) <= 1e-6 + 1e-2 * 0.2 * 128 ** 0.5 * 4e-5
        assert torch.equal(w, master.bfloat16())
