"""Sums of the orthogonalisation in 32 bits: runs short enough that what the
tensor cores cut off stays below float32's own roundings (GPU)."""
import pytest
import torch

import matrix_plain as P
from deformable_convolution_gb300 import optim

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


def test_a_large_square_matrix_keeps_its_runs():
    """2048 x 2048 against 64 bits.  A run of 8 blocks of 64 has 96 products of 16,
    after each of which less than 2^-23 of the sum so far is cut off, half of that
    on average, of half the run's sum on average: 96 * 2^-25 = 2.9e-6 of a gram's
    diagonal, which moves the result by 1.4 times as much at most (the steps' slopes
    at these singular values) = 4e-6; 2e-6 for the other roundings.  In one run of
    32 blocks it would be four times the first term."""
    gen = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn(2048, 2048, device="cuda", generator=gen)
    a, b, c = P.NS
    want = x.double() / (x.double().norm() + 1e-7)
    for _ in range(5):
        p = want @ want.T
        want = a * want + (b * p + c * (p @ p)) @ want
    out = torch.empty_like(x)
    optim.Orthogonalize([x], [out], precision=32)()
    assert float((out.double() - want).norm() / want.norm()) <= 6e-6
