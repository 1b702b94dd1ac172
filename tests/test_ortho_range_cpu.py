"""Coefficients of the orthogonalisation that leave the range its FP16 form holds are refused, also where only a few
starting values between the points of any grid would leave it.  Without a GPU: an empty gradient is a no-op, after the
checks."""
import numpy as np
import pytest

from fp8_block_scaled_13_b200 import _lib

A = 1 << 20  # an aligned fake device address; never dereferenced


@pytest.fixture(scope="module", autouse=True)
def built():
    from fp8_block_scaled_13_b200 import build
    build.build()


def _status(steps, a, b, c):
    return _lib.puro_fp8_orthogonalize(A, 64, 1, 0, 64, steps, a, b, c, 1e-7, A, 64, A, None)


def test_a_chaotic_quintic_is_refused():
    """From 0.99687 it ends at -2.6 in ten steps, from values beside that beyond 1e10."""
    assert _status(10, 1.5586876728841097, -3.7906957486772406, 1.2235391024963826) == _lib.PURO_ERR_SHAPE


@pytest.mark.parametrize("c", [(3.4445, -4.7750, 2.0315), (2.0, -1.5, 0.5), (1.875, -1.25, 0.375), (1.5, -0.5, 0.0),
                               (1.0, 0.0, 0.0), (0.0, 0.0, 0.0), (0.5, 0.0, -0.25), (0.0, 1.0, -0.5)])
def test_usual_coefficients_are_taken(c):
    for steps in (1, 5, 64):
        assert _status(steps, *c) == _lib.PURO_OK


@pytest.mark.parametrize("c", [(float("nan"), 0, 0), (0, float("nan"), 0), (0, 0, float("nan")), (float("inf"), 0, 0),
                               (0, float("-inf"), 0), (0, 0, float("inf")), (2.0, 0, 0), (0, -2.0, 0), (0, 0, 2.0)])
def test_others_are_refused(c):
    assert _status(1, *c) == _lib.PURO_ERR_SHAPE


def test_against_fine_grids():
    """Whatever any of 20000 starting values shows to leave the range is refused; what a grid keeps well inside, through
    every step and from a slightly wider interval, is taken."""
    rng = np.random.RandomState(1)
    refused = taken = 0
    for _ in range(400):
        a, b, c = (np.float32(v) for v in (rng.uniform(-4, 4), rng.uniform(-8, 8), rng.uniform(-5, 5)))
        steps = int(rng.choice([1, 2, 5, 10]))
        status = _status(steps, a, b, c)
        x = np.linspace(0, 1, 20000)
        top = r_top = 0.0
        for _ in range(steps):
            q = x * x
            r = q * (float(b) + float(c) * q)
            x = np.clip(x * (float(a) + r), -1e3, 1e3)
            top, r_top = max(top, np.abs(x).max()), max(r_top, np.abs(r).max())
        if top >= 2 or r_top >= 15:
            assert status == _lib.PURO_ERR_SHAPE, (a, b, c, steps)
            refused += 1
        elif steps == 1 and top < 1.95 and r_top < 14:
            # (one step: 2^-9 of the interval moves the value by 2^-9 (|a| + 3 |b| + 5 |c|) at most, 0.11)
            assert (status == _lib.PURO_OK) or top > 1.89, (a, b, c, steps)
            taken += status == _lib.PURO_OK
    assert refused > 50 and taken > 20


@pytest.mark.parametrize("steps", [2 ** 32 + 5, -2 ** 32 + 5, 2 ** 31, 2 ** 70, -2 ** 70])
def test_step_counts_beyond_an_int_are_refused(steps):
    """Cut to 32 bits, the first two are 5."""
    import torch
    import fp8_block_scaled_13_b200 as fp8
    with pytest.raises(ValueError, match="steps"):
        fp8.orthogonalize(torch.zeros(8, 8), steps=steps)
