"""Orthogonalisation and the Muon step: refusals (CPU), and the kernels against
plain forms in 64 bits (GPU)."""
import ctypes
import math

import pytest
import torch

import matrix_plain as P
from deformable_convolution_gb300 import binding as B
from deformable_convolution_gb300 import optim


def on_gpu(f):
    f = pytest.mark.gpu(f)
    return pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")(f)


F32, BF16 = torch.float32, torch.bfloat16
INVALID, UNSUPPORTED, WORKSPACE = B.DC_ERR_INVALID_ARG, B.DC_ERR_UNSUPPORTED, B.DC_ERR_WORKSPACE


# ---------------------------------------------------------------- refusals

def ortho_status(count=1, steps=5, precision=0, ws=0x10000, nbytes=1 << 40, table=True, **kw):
    d = dict(in_=0x1000, out=0x2000, rows=80, cols=80, in_dtype=B.DC_F32, out_dtype=B.DC_F32)
    d.update(kw)
    t = (B.DcMatrix * 1)(B.DcMatrix(**d)) if table else None
    return B.lib().dc_orthogonalize(t, count, steps, precision, ws, nbytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(count=-1), INVALID), (dict(table=False), INVALID), (dict(steps=0), INVALID), (dict(steps=21), INVALID),
    (dict(precision=2), INVALID), (dict(rows=-1), INVALID), (dict(in_=None), INVALID), (dict(out=None), INVALID),
    (dict(in_dtype=2), INVALID), (dict(out_dtype=-1), INVALID), (dict(in_=0x1002), UNSUPPORTED),
    (dict(out_dtype=B.DC_BF16, out=0x2001), UNSUPPORTED), (dict(rows=16385, cols=16385), UNSUPPORTED),
    (dict(cols=(1 << 22) + 1), UNSUPPORTED), (dict(ws=None), WORKSPACE), (dict(ws=0x10010), WORKSPACE),
    (dict(nbytes=100), WORKSPACE), (dict(count=0, table=False), B.DC_OK), (dict(rows=0, in_=None), B.DC_OK),
])
def test_orthogonalize_checks_its_arguments(kw, status):
    assert ortho_status(**kw) == status


def muon_status(count=1, scale=None, lr_device=None, ws=0x10000, nbytes=1 << 40, **kw):
    h = dict(lr=1e-3, momentum=0.95, nesterov=1, steps=5, precision=0)
    d = dict(param=0x1000, master=None, grad=0x2000, m=0x3000, rows=80, cols=80, param_dtype=B.DC_F32,
             grad_dtype=B.DC_F32, weight_decay=0.0, rate=1.0)
    for k, v in kw.items():
        (h if k in h else d)[k] = v
    t = (B.DcMuonTensor * 1)(B.DcMuonTensor(**d))
    return B.lib().dc_muon_step(t, count, ctypes.byref(B.DcMuonHyper(**h)), scale, lr_device, ws, nbytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(count=-1), INVALID), (dict(lr=-1.0), INVALID), (dict(lr=math.nan), INVALID), (dict(lr=math.inf), INVALID),
    (dict(momentum=1.0), INVALID), (dict(momentum=-0.1), INVALID), (dict(nesterov=2), INVALID), (dict(steps=0), INVALID),
    (dict(precision=-1), INVALID), (dict(param=None), INVALID), (dict(grad=None), INVALID), (dict(m=None), INVALID),
    (dict(master=0x4000), INVALID), (dict(param_dtype=3), INVALID), (dict(grad_dtype=-1), INVALID),
    (dict(weight_decay=-0.1), INVALID), (dict(weight_decay=math.inf), INVALID), (dict(rate=math.nan), INVALID),
    (dict(rate=math.inf), INVALID), (dict(cols=-1), INVALID), (dict(param=0x1002), UNSUPPORTED),
    (dict(grad=0x2001), UNSUPPORTED), (dict(m=0x3002), UNSUPPORTED),
    (dict(param_dtype=B.DC_BF16, master=0x4002), UNSUPPORTED), (dict(scale=0x5002), UNSUPPORTED),
    (dict(lr_device=0x5001), UNSUPPORTED), (dict(ws=None), WORKSPACE), (dict(nbytes=10), WORKSPACE),
    (dict(rows=0, param=None, grad=None, m=None), B.DC_OK),
])
def test_muon_checks_its_arguments(kw, status):
    assert muon_status(**kw) == status


def test_other_refusals():
    L = B.lib()
    out = ctypes.c_size_t(0)
    t = (B.DcMatrix * 1)(B.DcMatrix(None, None, 80, 80, 0, 0))
    assert L.dc_orthogonalize_workspace_size(t, 1, None) == INVALID
    assert L.dc_orthogonalize_workspace_size(None, 1, ctypes.byref(out)) == INVALID
    assert L.dc_orthogonalize_workspace_size(t, 1, ctypes.byref(out)) == B.DC_OK and out.value % 256 == 0 and out.value
    assert L.dc_muon_workspace_size(None, 1, ctypes.byref(out)) == INVALID
    assert L.dc_muon_step(None, 0, None, None, None, None, 0, None) == INVALID
    with pytest.raises(ValueError):
        optim.Orthogonalize([torch.zeros(3, 4)], [torch.zeros(3, 4)])  # not on the GPU
    with pytest.raises(ValueError):
        optim.Muon([dict(param=torch.zeros(5), grad=torch.zeros(5))])  # a vector
    with pytest.raises(ValueError):
        optim.Muon([], precision=8)


# ---------------------------------------------------------------- orthogonalisation

def matrix(m, n, kind, seed):
    gen = torch.Generator().manual_seed(seed)
    g = torch.randn(m, n, generator=gen, dtype=torch.float64)
    if kind == "falling":  # singular values over three orders of magnitude
        u, s, v = torch.linalg.svd(g, full_matrices=False)
        g = u * torch.exp(-7.0 * torch.arange(len(s)) / max(1, len(s) - 1)).double() @ v
    if kind == "deficient":
        r = max(1, min(m, n) // 3)
        g = torch.randn(m, r, generator=gen, dtype=torch.float64) @ torch.randn(r, n, generator=gen, dtype=torch.float64)
    return (g * 10.0 ** torch.randint(-6, 4, (1,), generator=gen).item()).float()


def off(got, want):
    return float((got.cpu().double() - want).norm() / want.norm())


SIZES = [(1, 1), (1, 300), (300, 1), (3, 5), (18, 2304), (2304, 18), (64, 64), (130, 70), (70, 131), (128, 128), (129, 513),
         (256, 2304), (640, 200), (384, 390)]


@on_gpu
@pytest.mark.parametrize("kind", ("full", "falling", "deficient"))
@pytest.mark.parametrize("size", SIZES)
def test_orthogonalize(size, kind):
    g = matrix(*size, kind, sum(size))
    want = P.orthogonal(g)
    # float32 arithmetic's own distance from 64 bits is the yardstick of precision 32, whose pairs of 16-bit floats hold
    # a number to 2^-24 as float32 does, but whose products leave low times low out and whose sums are truncated: four
    # times that.  A matrix of few elements may come out exact in float32 by luck; there the bound is the arithmetic's:
    # a step's roundings of X, A and P and of three products, eight of 2^-24 of |X|, of which the first step's grow by
    # 3.4445 a step in the directions of small singular values
    e32 = off(P.orthogonal(g, dtype=F32), want)
    x = g.cuda()
    outs = {b: torch.full_like(x, 5.0) for b in (16, 32)}
    for b in (16, 32):
        optim.Orthogonalize([x], [outs[b]], precision=b)()
    few = 8 * 3.4445 ** 5 * 2.0 ** -24 if g.numel() < 4096 else 0.0
    assert off(outs[32], want) <= max(4 * e32 + 2e-6, few)
    # precision 16 rounds X's factors to 11 bits (2^-12): A by 2 * 2^-12 of itself at most, which moves p(X) by
    # X p'(X) / 2 * that, |x p'(x)| <= 3.4 on [0, 1.21], and each later step carries it on with a slope of about one:
    # five times 3.4 * 2^-12 = 4.2e-3 were the roundings all one way
    assert off(outs[16], want) <= 4.2e-3
    again = torch.empty_like(x)
    optim.Orthogonalize([x], [again], precision=32)()
    assert torch.equal(again, outs[32])


@on_gpu
@pytest.mark.parametrize("size", [(8, 40000), (40000, 5), (64, 5000), (33, 9000), (65, 64), (64, 65), (1100, 1030), (1030, 1100),
                                  (2048, 2304), (2100, 2049)])
def test_orthogonalize_at_the_paths_borders(size):
    """Short sides whose long ones fit a cluster or not, several rows of tiles,
    tiles of every width: as above, the 64-bit form computed on the GPU."""
    g = matrix(*size, "full", sum(size))

    def plain(dtype):
        a, b, c = P.NS
        x = g.cuda().to(dtype)
        x = x / (x.square().sum().sqrt() + 1e-7)
        x = x.T if size[0] > size[1] else x
        for _ in range(5):
            p = x @ x.T
            x = a * x + (b * p + c * (p @ p)) @ x
        return (x.T if size[0] > size[1] else x).cpu()
    want = plain(torch.float64)
    e32 = off(plain(F32), want)
    x = g.cuda()
    outs = {b: torch.full_like(x, 5.0) for b in (16, 32)}
    for b in (16, 32):
        optim.Orthogonalize([x], [outs[b]], precision=b)()
    # an accumulator of A is truncated after every 16 products, after a split's 64 at most (or, with 1024 values a side
    # and more, after all): half a unit in the last place of the sum each time on the diagonal, twice that of X
    # by the steps' slopes
    long = max(size) / 16
    truncated = 2 * (long if min(size) > 512 else min(long, 64 * max(1, long / 64 / 48))) * 2.0 ** -25
    assert off(outs[32], want) <= 4 * e32 + 2e-6 + truncated
    assert off(outs[16], want) <= 4.2e-3
    # beside others of its kind and of the small ones' the same bits
    y, more = torch.empty_like(x), [torch.randn(s, device="cuda") for s in ((18, 200), (300, 300), (130, 700))]
    optim.Orthogonalize(more + [x], [torch.empty_like(t) for t in more] + [y], precision=32)()
    assert torch.equal(y, outs[32])


@on_gpu
@pytest.mark.parametrize("kinds", [(F32, BF16), (BF16, F32), (BF16, BF16)])
def test_types_and_in_place(kinds):
    g = matrix(96, 200, "full", 1).to(kinds[0])
    want = P.orthogonal(g)
    x, y = g.cuda(), torch.empty(96, 200, dtype=kinds[1], device="cuda")
    optim.Orthogonalize([x], [y], precision=32)()
    # a rounding to bf16 is off by 2^-8 of the value at most
    assert off(y, want) <= (2.0 ** -8 if kinds[1] is BF16 else 2e-5)
    if kinds[0] is kinds[1]:
        optim.Orthogonalize([x], [x], precision=32)()
        assert torch.equal(x, y)


@on_gpu
def test_steps():
    g = matrix(60, 90, "full", 2)
    for steps in (1, 2, 3, 8, 20):
        y = torch.empty(60, 90, device="cuda")
        optim.Orthogonalize([g.cuda()], [y], steps=steps, precision=32)()
        # later steps carry an error on with a slope of at most 1.6 around one: 20 of them by 1.6^15 from 1e-6
        assert off(y, P.orthogonal(g, steps)) <= (2e-5 if steps <= 8 else 1e-2)


@on_gpu
def test_zeros_and_what_is_not_finite():
    zero, bad, inf, big, small = (matrix(40, 300, "full", k).cuda() for k in range(5))
    zero.zero_()
    bad[3, 7] = float("nan")
    inf[39, 299] = float("-inf")
    big.fill_(1e30)
    small.mul_(1e-30)
    ins = [zero, bad, inf, big, small]
    outs = [torch.ones_like(t) for t in ins]
    optim.Orthogonalize(ins, outs, precision=32)()
    assert not outs[0].any()
    assert all(torch.isnan(t).all() for t in outs[1:4])
    # far below eps: X starts at g / 1e-7, which five steps raise by 3.4445^5 at most
    assert float(outs[4].abs().max()) <= 485 * 1e-20


@on_gpu
def test_many_matrices_at_once():
    """More than one launch's table holds, of every shape, some empty."""
    gen = torch.Generator().manual_seed(0)
    sizes = [tuple(int(v) for v in torch.randint(1, 90, (2,), generator=gen)) for _ in range(101)]
    sizes[5], sizes[60], sizes[100] = (0, 7), (9, 0), (0, 0)
    ins = [torch.randn(s, generator=gen).cuda() for s in sizes]
    outs = [torch.empty_like(t) for t in ins]
    call = optim.Orthogonalize(ins, outs, precision=32)
    call()
    for x, y in zip(ins, outs):
        if x.numel():
            alone = torch.empty_like(x)
            optim.Orthogonalize([x], [alone], precision=32)()
            assert torch.equal(y, alone)  # a matrix's result does not depend on its company


@on_gpu
def test_unaligned_tensors_and_guards():
    for off_by, kind in ((1, F32), (3, BF16)):
        room = torch.full((70 * 91 + 32,), 3.0, dtype=kind, device="cuda")
        g = matrix(70, 91, "full", 3).to(kind)
        flat = torch.cat([torch.zeros(off_by, dtype=kind), g.flatten()]).cuda()
        x, y = flat[off_by:].view(70, 91), room[off_by:off_by + 70 * 91].view(70, 91)
        optim.Orthogonalize([x], [y], precision=32)()
        assert off(y, P.orthogonal(g)) <= (2.0 ** -8 if kind is BF16 else 2e-5)
        assert (room[:off_by] == 3).all() and (room[off_by + 70 * 91:] == 3).all()


# ---------------------------------------------------------------- the step

def weights(kind, grad, shapes, seed):
    gen = torch.Generator().manual_seed(seed)
    params = []
    for s in shapes:
        p = torch.randn(s, generator=gen) * 0.05
        q = dict(param=p.cuda() if kind == "f32" else p.bfloat16().cuda(), grad=(torch.randn(s, generator=gen) * 1e-3).to(grad).cuda(),
                 m=(torch.randn(s, generator=gen) * 1e-3).cuda())
        if kind == "master":
            q["master"] = p.cuda()
        params.append(q)
    return params


SHAPES = [(16, 8, 3, 3), (18, 72), (130, 40), (1, 5), (64, 64, 1, 1), (80, 70), (72, 16, 3, 3), (200, 131)]


@on_gpu
@pytest.mark.parametrize("nesterov", (True, False))
@pytest.mark.parametrize("grad", (F32, BF16))
@pytest.mark.parametrize("kind", ("f32", "master", "bf16"))
def test_step(kind, grad, nesterov):
    lr, mu, decay, scale = 2e-2, 0.9, 0.05, 0.37
    params = weights(kind, grad, SHAPES, 4)
    old = [{k: v.clone() for k, v in q.items()} for q in params]
    opt = optim.Muon(params, lr=lr, momentum=mu, nesterov=nesterov, weight_decay=decay, precision=32)
    s = torch.full((1,), scale, device="cuda")
    opt.step(grad_scale=s)
    for q, o in zip(opt.params, old):
        rate = 0.2 * max(o["param"].shape[0], o["param"][0].numel()) ** 0.5
        assert q["rate"] == pytest.approx(rate)
        kept = "master" if kind == "master" else "param"
        want, m = P.muon(o[kept], o["m"], o["grad"], float(s), lr, mu, nesterov, decay, rate)
        # m: three operations' roundings of terms no larger than the sum of their magnitudes
        size = o["m"].cpu().double().abs() + o["grad"].cpu().double().abs()
        assert ((q["m"].cpu().double() - m).abs() <= 4 * 2.0 ** -24 * size).all()
        # p: three roundings, and the direction's error: 2e-5 of its largest value (1.21, a singular value)
        tol = 3 * 2.0 ** -24 * o[kept].cpu().double().abs() + (2e-5 + 4 * 2.0 ** -24) * lr * rate * 1.21
        got = q[kept].cpu().double()
        half = 2.0 ** -8 * want.abs() if kind == "bf16" else 0.0
        assert ((got - want).abs() <= tol + half).all()
        if kind == "master":
            assert torch.equal(q["param"], q["master"].bfloat16())


@on_gpu
def test_a_scale_that_is_not_finite_skips_the_step():
    params = weights("master", F32, SHAPES, 5)
    old = [{k: v.clone() for k, v in q.items()} for q in params]
    opt = optim.Muon(params)
    for v in (float("nan"), float("inf")):
        opt.step(grad_scale=torch.full((1,), v, device="cuda"))
        for q, o in zip(opt.params, old):
            assert all(torch.equal(q[k], o[k]) for k in o)
    params[1]["grad"][0, 0] = float("nan")  # one weight's gradient: that weight alone
    opt.step()
    for i, q in enumerate(opt.params):
        assert torch.isnan(q["param"]).all() if i == 1 else torch.isfinite(q["param"]).all()


@on_gpu
def test_replayed_steps_follow_single_ones():
    """A captured step with lr and scale on the device, replayed with other
    gradients, beside the same steps called one by one."""
    a, b = (weights("master", BF16, SHAPES, 6) for _ in range(2))
    one, graphed = (optim.Muon(q, precision=16) for q in (a, b))
    gen = torch.Generator().manual_seed(8)
    steps = [([torch.randn(s, generator=gen).bfloat16().cuda() for s in SHAPES], lr) for lr in (1e-2, 3e-3, 1e-3)]
    scale, lr = torch.ones(1, device="cuda"), torch.zeros(1, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        graphed.step(grad_scale=scale, lr=lr)
    for k, (grads, rate) in enumerate(steps):
        for q, r, g in zip(a, b, grads):
            q["grad"].copy_(g)
            r["grad"].copy_(g)
        scale.fill_(0.5 + k)
        lr.fill_(rate)
        one.lr = rate
        one.step(grad_scale=scale)
        graph.replay()
    torch.cuda.synchronize()
    for q, r in zip(one.params, graphed.params):
        assert all(torch.equal(q[k], r[k]) for k in ("param", "master", "m"))


@on_gpu
def test_state_and_gradients_at_other_addresses():
    a, b = weights("master", F32, SHAPES, 10), weights("master", F32, SHAPES, 11)
    first, again = optim.Muon(a), optim.Muon(b)
    first.step()
    saved = {k: ([{n: t.clone() for n, t in s.items()} for s in v] if k == "state" else v)
             for k, v in first.state_dict().items()}
    again.load_state_dict(saved)
    grads = [torch.randn_like(q["grad"]) for q in a]
    for opt in (first, again):
        opt.set_grads(grads)
        opt.step()
    for q, r in zip(first.params, again.params):
        assert all(torch.equal(q[k], r[k]) for k in ("param", "master", "m"))
    with pytest.raises(ValueError):
        first.set_grads(grads[:-1])
    with pytest.raises(ValueError):
        first.set_grads([None] * len(grads))
    with pytest.raises(ValueError):
        again.load_state_dict(dict(lr=1.0, state=saved["state"][:-1]))
