"""What the orthogonalisation adds to the rounding of its BF16 result, for gradients of every structure: those whose
roundings would be independent anyway (Gaussian, low rank over a floor), those whose entries are alike (all equal, signs,
blocks, repeated rows) and those that lack directions (exact low rank), which every step lifts by 3.4 if a rounding
leaves any there.

Operands are rounded to FP16 at random: f (1 - f) of a squared step, 1/6 in the mean, a step of 2^-10 to 2^-11 of the
value: 0.41 * 0.74 * 2^-10 = 2.9e-4 in the mean square.  Five steps take three products of two operands each: 30
independent roundings, sqrt(30) * 2.9e-4 = 1.6e-3.  (A step changes the relative error of a direction by x p'(x) / p(x),
1 for small x and between -1.7 and 1 where x has grown.)  The result's own rounding is off by e0, measured, where its
values are many and spread, and by half a step of 2^-8 at most where they are few: then they round alike."""
import pytest
import torch

pytestmark = pytest.mark.gpu

NS = (3.4445, -4.7750, 2.0315)
ADDED = 1.6e-3
HALF = 2.0 ** -8


@pytest.fixture(scope="module")
def fp8():
    import fp8_block_scaled_13_b200 as m
    from fp8_block_scaled_13_b200 import build
    build.build()
    return m


def _gradients(n, k):
    """(name, gradient, whether the result's values are spread)."""
    g = torch.Generator(device="cuda").manual_seed(n * 7 + k)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    sign = lambda *s: torch.where(randn(*s) < 0, -1.0, 1.0)  # noqa: E731
    low = lambda r: randn(n, r) @ randn(r, k) / r ** 0.5  # noqa: E731
    yield "gaussian", randn(n, k), True
    yield "an eighth over a floor", low(max(1, min(n, k) // 8)) + randn(n, k), True
    yield "rank 1", low(1), True
    yield "rank 4", low(4), True
    yield "rank 1 over 1 %", low(1) + 0.01 * randn(n, k), True
    yield "all equal", torch.ones(n, k, device="cuda"), False
    yield "signs", sign(n, 1) * sign(1, k), False
    yield "four of signs", sign(n, 4) @ sign(4, k), False
    yield "blocks", torch.kron(sign(n // 8 + 1, k // 8 + 1), torch.ones(8, 8, device="cuda"))[:n, :k].contiguous(), False
    yield "repeated rows", randn(16, k)[torch.randint(0, 16, (n,), generator=g, device="cuda")], False


def _reference(g, steps=5):
    a, b, c = NS
    x = g.double()
    x = x / (x.norm() + 1e-7)
    wide = x.shape[0] <= x.shape[1]
    for _ in range(steps):
        m = x @ x.mT if wide else x.mT @ x
        p = b * m + c * m @ m
        x = a * x + (p @ x if wide else x @ p)
    return x


def _off(got, want):
    return ((got.double() - want).norm() / want.norm()).item()


@pytest.mark.parametrize("n,k", [(129, 130), (200, 333), (333, 200), (160, 1342), (1342, 160), (256, 768), (640, 640),
                                 (640, 5377), (5377, 640), (1000, 1000), (2048, 2048)])
def test_above_128(fp8, n, k):
    for name, g, spread in _gradients(n, k):
        want = _reference(g)
        off, e0 = _off(fp8.orthogonalize(g), want), _off(want.to(torch.bfloat16), want)
        if spread:
            added = max(0.0, off ** 2 - e0 ** 2) ** 0.5
            assert added <= ADDED, (name, added)
        else:
            assert off <= HALF + ADDED, (name, off)
    assert fp8.device_status() == 0


@pytest.mark.parametrize("n,k", [(2, 3), (3, 2), (8, 8), (16, 40), (40, 16), (64, 64), (128, 128), (100, 1800), (640, 128)])
def test_up_to_128(fp8, n, k):
    for name, g, spread in _gradients(n, k):
        want = _reference(g)
        off = _off(fp8.orthogonalize(g), want)
        assert off <= HALF + ADDED, (name, off)
    assert fp8.device_status() == 0


@pytest.mark.parametrize("n,k", [(64, 64), (100, 300), (129, 400), (300, 200), (640, 640)])
def test_ten_steps_of_what_lacks_directions(fp8, n, k):
    """What an operation leaves in a direction that X lacks is lifted by 3.4445 in each of up to nine later steps, and
    each step leaves as much: 3.4445^9 * (1 + 1/3.4 + ...) = 9.6e4 times.  Held to 22 bits, X is off by 2^-22, and a sum
    over the m rows, added 16 at a time, by m / 16 roundings of 2^-24."""
    bound = (4 + min(n, k) / 16) * 2.0 ** -24 * 9.6e4 + HALF
    for name, g, _ in _gradients(n, k):
        if name in ("rank 1", "rank 4"):
            off = _off(fp8.orthogonalize(g, steps=10), _reference(g, 10))
            assert off <= bound, (name, off)


@pytest.mark.parametrize("n,k", [(1, 5000), (5000, 1), (2, 65536), (65536, 3), (128, 2049), (2049, 128), (33, 10000),
                                 (10000, 31), (127, 4097)])
def test_far_from_square(fp8, n, k):
    """Beyond the sides of the small kernel by one of them only: products of few rows over long sums.  Few rows average
    less: a rounding of O or R, a step of 2^-10 at most, may count whole, 2 in each of 5 steps and what they leave, and the
    bound is that of few values."""
    for name, g, _ in _gradients(n, k):
        want = _reference(g)
        off = _off(fp8.orthogonalize(g), want)
        assert off <= HALF + 10 * 2.0 ** -10, (name, off)
    assert fp8.device_status() == 0


@pytest.mark.parametrize("n,k", [(1, 5000), (5000, 1), (2, 65536), (65536, 3), (23, 2152), (2049, 128), (33, 10000)])
def test_few_rows_meet_all_of_x(fp8, n, k):
    """Up to 128 rows, R multiplies both terms of X.  What X X^T loses averages over its long sums; O, which enters the
    square twice and R, and R itself are rounded, 4 times in each of 5 steps: sqrt(20) * 2.9e-4 = 1.3e-3."""
    for name, g, _ in _gradients(n, k):
        if name in ("gaussian", "an eighth over a floor"):
            want = _reference(g)
            off, e0 = _off(fp8.orthogonalize(g), want), _off(want.to(torch.bfloat16), want)
            assert max(0.0, off ** 2 - e0 ** 2) ** 0.5 <= 1.3e-3, (name, off)
    assert fp8.device_status() == 0
