"""Plain forms in 64 bits of the matrices in 8 bits, their products and Muon."""
import torch

BLOCK = 128
# bits of the mantissa, lowest exponent of a normal code, largest code
FORMATS = {0: (3, -6, 448.0), 1: (2, -14, 57344.0)}
NS = (3.4445, -4.7750, 2.0315)


def blocks(t, square):
    """t [batch, rows, cols] (float64) padded with zeros and cut into blocks:
    [batch, row blocks, block rows, column blocks, 128]."""
    b, r, c = t.shape
    h = BLOCK if square else 1
    i, k = -(-r // h), -(-c // BLOCK)
    p = torch.zeros(b, i * h, k * BLOCK, dtype=torch.float64)
    p[:, :r, :c] = t
    return p.view(b, i, h, k, BLOCK)


def quantize(t, fmt, square):
    """(values that the codes stand for, scale byte of each element) of t
    [batch, rows, cols], computed on the CPU."""
    b, r, c = t.shape
    mantissa, low, most = FORMATS[fmt]
    v = blocks(t.detach().cpu().double(), square)
    top = v.abs().amax((2, 4), keepdim=True)
    e = torch.full_like(top, -126.0)
    for k in range(-126, 121):  # the smallest exponent whose range holds the block, by comparisons alone
        e = torch.where(top > most * 2.0 ** k, torch.full_like(e, k + 1.0), e)
    bad = ~torch.isfinite(top)
    s = v / torch.exp2(e)
    quantum = torch.exp2(torch.floor(torch.log2(s.abs().clamp_min(2.0 ** -300))).clamp_min(low) - mantissa)
    q = torch.round(s / quantum) * quantum * torch.exp2(e)
    q = torch.where(bad.expand_as(q), torch.full_like(q, float("nan")), q)
    byte = torch.where(bad, torch.full_like(e, 255.0), e + 127).to(torch.uint8)

    def back(x):
        return x.expand_as(v).reshape(b, v.shape[1] * v.shape[2], -1)[:, :r, :c]
    return back(q), back(byte)


def orthogonal(g, steps=5, dtype=torch.float64):
    """Newton-Schulz steps of g [rows, cols] in the given type, on the CPU."""
    a, b, c = NS
    x = g.detach().cpu().to(dtype)
    x = x / (x.square().sum().sqrt() + 1e-7)
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    for _ in range(steps):
        p = x @ x.T
        x = a * x + (b * p + c * (p @ p)) @ x
    return x.T if tall else x


def muon(p, m, g, scale, lr, momentum, nesterov, decay, rate, steps=5, direction=None):
    """(new p, new m) in 64 bits; direction: an orthogonalised matrix to use."""
    p, m, g = (t.detach().cpu().double() for t in (p, m, g))
    g = g * scale
    m = m * momentum + g * (1 - momentum)
    u = m * momentum + g * (1 - momentum) if nesterov else m
    o = orthogonal(u.reshape(u.shape[0], -1), steps).reshape(u.shape)
    return p * (1 - lr * decay) - o * (lr * rate), m
