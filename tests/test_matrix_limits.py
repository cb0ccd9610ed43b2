"""Matrices in 8 bits, orthogonalisation and Muon where their calls meet others
(two streams at once, graphs that share a workspace) and where an element's
place passes 32 bits."""
import dataclasses

import pytest
import torch

import matrix_plain as P
from deformable_convolution_gb300 import binding as B
from deformable_convolution_gb300 import fp8, optim

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]
F32, BF16 = torch.float32, torch.bfloat16


def normal(*shape, dtype=BF16, seed=0):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(seed))


def in_bits(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


# ---------------------------------------------------------------- calls beside others

def calls():
    """Independent calls of every kind with results of their own: (call, results)."""
    out = []
    for seed, sizes in enumerate([[(300, 700), (18, 500), (64, 64)], [(1024, 600), (700, 130)], [(40, 40)] * 45]):
        ins = [normal(*s, dtype=F32, seed=seed) for s in sizes]
        outs = [torch.zeros_like(t) for t in ins]
        out.append((optim.Orthogonalize(ins, outs, precision=32 if seed else 16), outs))
    for seed, (layout, training) in enumerate([(B.DC_NCHW, True), (B.DC_NHWC, True), (B.DC_NHWC, False)]):
        layer = fp8.Pointwise(4, 200, 120, 30, 40, B.DC_BF16, layout, training)
        layer.load(normal(120, 200, seed=seed))
        x, gy = normal(*layer.x_shape, seed=5), normal(*layer.y_shape, seed=6)
        y, gx, gw = torch.zeros_like(gy), torch.zeros_like(x), torch.zeros(120, 200, device="cuda")

        def call(stream=None, layer=layer, x=x, gy=gy, y=y, gx=gx, gw=gw):
            layer.forward(x, y, stream)
            if layer.training:
                layer.backward(gy, gx, gw, stream)
        out.append((call, [y, gx, gw]))
    torch.cuda.synchronize()
    return out


def test_calls_on_streams_of_their_own_at_once():
    work = calls()
    want = []
    for call, results in work:
        call()
        torch.cuda.synchronize()
        want.append([t.clone() for t in results])
        assert any(t.any() for t in results)
    streams = [torch.cuda.Stream() for _ in work]
    for _ in range(10):
        for _, results in work:
            for t in results:
                t.zero_()
        torch.cuda.synchronize()
        for _ in range(3):
            for (call, _), s in zip(work, streams):
                call(stream=s)
        torch.cuda.synchronize()
        for (_, results), w in zip(work, want):
            assert all(in_bits(a, b) for a, b in zip(results, w))
    assert B.device_error() == 0


def test_graphs_that_share_a_workspace():
    """Two captured calls of one object (one workspace), replayed in turn on one
    stream and with an eager call between, read what stands in their inputs."""
    x, w = normal(300, 700, dtype=F32), normal(600, 520, dtype=F32, seed=1)
    y, z = torch.zeros_like(x), torch.zeros_like(w)
    call = optim.Orthogonalize([x, w], [y, z])
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g in graphs:
        with torch.cuda.graph(g):
            call()
    for seed, g in enumerate(graphs + graphs):
        x.copy_(normal(300, 700, dtype=F32, seed=seed + 2))
        g.replay()
        got = y.clone(), z.clone()
        y.zero_(), z.zero_()
        call()
        assert torch.equal(got[0], y) and torch.equal(got[1], z) and y.any()


@pytest.mark.parametrize("size", [(1, 512, 32, 64, 64), (3, 40, 72, 9, 11), (2, 64, 300, 40, 33), (8, 256, 256, 56, 56)])
@pytest.mark.parametrize("layout", (B.DC_NCHW, B.DC_NHWC))
def test_backward_products_side_by_side(size, layout):
    """The weight's gradient may start before the product ahead of it has ended:
    what comes after both (the next pass's codes of other inputs, in the same
    place) waits for both, eagerly and in a graph."""
    n, c_in, c_out, h, w = size
    layer = fp8.Pointwise(n, c_in, c_out, h, w, B.DC_BF16, layout)
    layer.load(normal(c_out, c_in))
    sets = [(normal(*layer.x_shape, seed=k), normal(*layer.y_shape, seed=k + 9)) for k in range(3)]
    want = []
    for x, gy in sets:
        layer.forward(x)
        torch.cuda.synchronize()
        want.append([t.clone() for t in layer.backward(gy)])
        torch.cuda.synchronize()
    # the same with the weight's gradient behind the other product
    apart = fp8.Pointwise(n, c_in, c_out, h, w, B.DC_BF16, layout)
    apart._gw = dataclasses.replace(apart._gw, beside=0)
    apart.load(normal(c_out, c_in))
    for (x, gy), r in zip(sets, want):
        apart.forward(x)
        assert all(in_bits(a, b) for a, b in zip(apart.backward(gy), r))

    def passes(times):
        got = []
        for _ in range(times):
            for x, gy in sets:
                layer.forward(x)
                got.append(layer.backward(gy))
        return got
    got = passes(10)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = passes(2)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for k, r in enumerate(got + captured):
        assert all(in_bits(a, b) for a, b in zip(r, want[k % len(sets)]))


def test_new_results_on_another_stream():
    """A result made for a call on another stream does not take memory that the
    current stream, which has just given it up, has still to write."""
    layer = fp8.Pointwise(2, 64, 64, 64, 64, B.DC_BF16, B.DC_NHWC)
    layer.load(normal(64, 64))
    x, gy = normal(*layer.x_shape, seed=1), normal(*layer.y_shape, seed=2)
    want = [layer.forward(x), *layer.backward(gy)]
    values = layer.x.values()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for k in range(4):
        late = [torch.empty_like(t) for t in want + [values]]
        torch.cuda._sleep(20_000_000)  # about 10 ms
        for t in late:
            t.fill_(7.0)
        del late, t
        got = [layer.forward(x, stream=side), *layer.backward(gy, stream=side)]
        again = layer.x.values(stream=side)
        torch.cuda.synchronize()
        assert all(in_bits(a, b) for a, b in zip(got, want)) and in_bits(again, values)


# ---------------------------------------------------------------- beyond 32 bits

def test_codes_beyond_32_bits():
    rows, cols, last = 260, 8_500_000 // 128 * 128 + 40, 128 * 3 + 40  # 2.2e9 values
    assert rows * (cols - last) > 2 ** 31
    x = normal(1, rows, cols)
    q = fp8.Quantized(B.Fp8Problem(1, rows, cols), True, True)
    q.load(x)
    # a row's last runs, and the last columns' transposes, as of a matrix of their own
    end = x[:, :, -last:].contiguous()
    r = fp8.Quantized(B.Fp8Problem(1, rows, last), True, True)
    r.load(end)
    n = r.codes.shape[2]
    assert torch.equal(q.codes[:, :, -n:], r.codes)
    assert torch.equal(q.codes_t[:, -last:], r.codes_t)
    # values decode to the same numbers, for the last rows
    del x, end
    torch.cuda.empty_cache()
    v = q.values(transposed=True)
    assert torch.equal(v[:, -last:], r.values(transposed=True))


def test_products_beyond_32_bits():
    """D of 2.5e9 values, a sum over 2.1e9 and images 2.1e9 values apart."""
    m, n, k, last = 50_000, 50_000, 130, 300
    a, b = (fp8.Quantized(B.Fp8Problem(1, rows, k)) for rows in (m, n))
    x, y = normal(1, m, k), normal(1, n, k, seed=1)
    a.load(x), b.load(y)
    p = B.Fp8Product(1, m, n, k)
    d = torch.empty(p.shape, dtype=BF16, device="cuda")
    ws = torch.empty(max(1, B.dc_fp8_matmul_workspace_size(p)), dtype=torch.uint8, device="cuda")
    B.dc_fp8_matmul(p, a.codes, a.scales, b.codes, b.scales, d, ws)
    e = fp8.Quantized(B.Fp8Problem(1, last, k))
    e.load(x[:, -last:].contiguous())
    p2 = B.Fp8Product(1, last, n, k)
    d2 = torch.empty(p2.shape, dtype=BF16, device="cuda")
    ws2 = torch.empty(max(1, B.dc_fp8_matmul_workspace_size(p2)), dtype=torch.uint8, device="cuda")
    B.dc_fp8_matmul(p2, e.codes, e.scales, b.codes, b.scales, d2, ws2)
    assert torch.equal(d[:, -last:], d2)


@pytest.mark.parametrize("training", (True, False))
@pytest.mark.parametrize("layout", (B.DC_NCHW, B.DC_NHWC))
def test_layers_beyond_32_bits(layout, training):
    """Two images of 1.1e9 values each: the second as a layer of its own gives it."""
    c_in, c_out, h, w = 136, 72, 2800, 2900
    layer, one = (fp8.Pointwise(n, c_in, c_out, h, w, B.DC_BF16, layout, training) for n in (2, 1))
    assert 2 * c_in * h * w > 2 ** 31
    weight = normal(c_out, c_in)
    layer.load(weight), one.load(weight)
    x = normal(*layer.x_shape, seed=1)
    y = layer.forward(x)
    assert torch.equal(y[1:], one.forward(x[1:]))
    if training:
        gy = y
        gx, gw = layer.backward(gy)
        gx1, gw1 = one.backward(gy[1:].contiguous())
        assert torch.equal(gx[1:], gx1)
        one.forward(x[:1])
        _, gw0 = one.backward(gy[:1].contiguous())
        # the same exact products of 1.8e7 pixels summed in float32 in another order, by runs
        assert float((gw - gw0 - gw1).norm() / gw.norm()) <= 1e-3


def polynomial(x, steps=5):
    """M (64 bits) with M X0 = X after `steps`, for a wide x, and X0's factor."""
    gram = torch.zeros(x.shape[0], x.shape[0], dtype=torch.float64, device="cuda")
    for part in x.split(200_000, 1):
        part = part.double()
        gram += part @ part.T
    squares = gram.diagonal().sum()
    f = 1 / (squares.sqrt() + 1e-7)
    gram *= f * f
    a, b, c = P.NS
    eye = torch.eye(len(gram), dtype=torch.float64, device="cuda")
    m = eye
    for _ in range(steps):
        p = m @ gram @ m.T
        m = (a * eye + b * p + c * (p @ p)) @ m
    return m, f


@pytest.mark.parametrize("size", [(700, 70_000), (600, 3_700_000)])
def test_orthogonalize_long_sides(size):
    """Long sides, one with 2.2e9 values.  An accumulator runs over 8 blocks of 64:
    96 products of 16, each truncated by less than 2^-23 of the sum so far, half
    the run's on average: 96 * 2^-24 = 5.7e-6 of the gram.  A gram that is off by
    d moves these sizes' results by 1.1 d and 1.4 d (the steps evaluated at their
    singular values, within 10 % and 1.3 % of their mean): 8e-6, and 2e-6 for the
    other roundings."""
    x = normal(*size, dtype=F32)
    m, f = polynomial(x)
    out = torch.empty_like(x)
    optim.Orthogonalize([x], [out], precision=32)()
    for cut in (slice(0, 3000), slice(size[1] // 2, size[1] // 2 + 3000), slice(size[1] - 3000, size[1])):
        want = m @ (x[:, cut].double() * f)
        err = float((out[:, cut].double() - want).norm() / want.norm())
        assert err <= 1e-5
