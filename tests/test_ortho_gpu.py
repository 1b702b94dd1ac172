"""Newton-Schulz orthogonalisation on the GPU against the iteration in 64 bits.

Errors are relative to the norm of the result.  Its one rounding to BF16 is off
by at most half a step: between 2^-9 and 2^-8 of a value, evenly spread, so at
most 2^-8 / sqrt(3) = 2.26e-3 in the mean square.  Between, X is
exact to 22 bits and what enters a product is rounded to FP16 off the diagonal:
a relative error of at most 2^-11 / sqrt(3) = 2.8e-4 in the mean square.  Five
steps take three products of two operands each, so 30 independent roundings,
sqrt(30) * 2.8e-4 = 1.6e-3.  (A step changes the relative error of a direction
by the factor x p'(x) / p(x), which is 1 for small x and, where x has grown to
0.7 or more, between -1.7 and 1: later steps do not let earlier errors grow.)
The bound is the plain sum, 2.26e-3 + 1.6e-3 = 3.9e-3.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

NS = (3.4445, -4.7750, 2.0315)
BOUND = 3.9e-3


@pytest.fixture(scope="module")
def fp8():
    import fp8_block_scaled_13_b200 as m
    from fp8_block_scaled_13_b200 import build
    build.build()
    return m


def _gradient(n, k, seed, dtype, size=1e-3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = max(1, min(n, k) // 8)
    v = torch.randn(n, r, generator=g, device="cuda") @ torch.randn(r, k, generator=g, device="cuda") / r ** 0.5
    return ((v + torch.randn(n, k, generator=g, device="cuda")) * size).to(dtype)


def _reference(g, steps=5, eps=1e-7, coefficients=NS):
    a, b, c = coefficients
    x = g.double()
    x = x / (x.norm() + eps)
    for _ in range(steps):
        m = x @ x.mT if x.shape[0] <= x.shape[1] else x.mT @ x
        p = b * m + c * m @ m
        x = a * x + (p @ x if x.shape[0] <= x.shape[1] else x @ p)
    return x


def _error(got, want):
    return ((got.double() - want).norm() / want.norm()).item()


@pytest.mark.parametrize("n,k", [(1, 1), (1, 40), (40, 1), (2, 3), (16, 16), (64, 64), (65, 63), (128, 128), (128, 640),
                                 (640, 128), (129, 257), (200, 333), (333, 200), (256, 512), (300, 1000), (1000, 300),
                                 (520, 520), (768, 2048), (2048, 768), (1100, 1537)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_orthogonalize(fp8, n, k, dtype):
    g = _gradient(n, k, n * 3 + k, dtype)
    got = fp8.orthogonalize(g)
    assert fp8.device_status() == 0
    assert got.dtype == torch.bfloat16 and _error(got, _reference(g)) <= BOUND
