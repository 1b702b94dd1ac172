"""The gated activation where the sigmoid leaves FP32's normal range, against 64 bits, forward and backward.

The sigmoid is 2^-22 / (2^-22 + 2^x) with x = -g log2(e) - 22: x is off by 2^-24 of itself and of g log2(e) (the
constant), which times ln 2 makes (15.3 + 2 |g|) 2^-24 of 2^x; with the 2 units of ex2 and of the quotient, the sum and up
to five products below 2^-19 + |g| 2^-22.  Below FP32's normal range it is rounded to multiples of 2^-149 (and its
factors may flush what is below), off by at most 2^-148, times the factors that each result has; a result below BF16's
range by at most 2^-134."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fp8():
    import fp8_block_scaled_13_b200 as m
    from fp8_block_scaled_13_b200 import build
    build.build()
    return m


def _gu(t, f, reach):
    """g over [-95, 95] and u over powers of two up to 2^reach, and their signs, in every combination of columns."""
    g = torch.linspace(-95, 95, f, device="cuda").expand(t, f)
    e = torch.arange(t, device="cuda")[:, None] * (2.0 * reach / (t - 1)) - reach
    u = torch.exp2(e.double()).expand(t, f) * torch.where(torch.arange(f, device="cuda") % 2 == 0, 1.0, -1.0)
    return torch.cat([g, u.float()], 1).to(torch.bfloat16)


def _inside(got, want, bound):
    got = got.double()
    assert got.isfinite().all()
    worst = ((got - want).abs() - bound).max().item()
    assert worst <= 0, "off by %.3g more than its bound" % worst


def test_forward(fp8):
    t, f = 260, 3840
    gu = _gu(t, f, 100.0)
    g, u = gu[:, :f].double(), gu[:, f:].double()
    want = g * torch.sigmoid(g) * u
    noise = 2.0 ** -19 + 2.0 ** -22 * g.abs()
    _inside(fp8.swiglu(gu, layout="bf16"), want, (2.0 ** -8 + noise) * want.abs() + 2.0 ** -148 * (g * u).abs() + 2.0 ** -134)


def test_backward(fp8):
    t, f = 260, 3840
    gu = _gu(t, f, 60.0)
    da = torch.exp2(torch.arange(f, device="cuda") % 41 - 10.0).expand(t, f).to(torch.bfloat16).contiguous()
    g, u, d = gu[:, :f].double(), gu[:, f:].double(), da.double()
    s = torch.sigmoid(g)
    dg, du = d * u * s * (1 + g * (1 - s)), d * g * s
    # 1 + g (1 - s) cancels: its error is that of its parts, and 1 - s is off by the noise of s and half a unit of 1
    noise = 2.0 ** -19 + 2.0 ** -22 * g.abs()
    parts = (d * u * s).abs() * (1 + g.abs() * (1 - s) + g.abs() * (s + 2.0 ** -4))
    got = fp8.swiglu_backward(da, gu, layout="bf16")
    _inside(got[:, :f], dg, 2.0 ** -8 * dg.abs() + noise * parts + 2.0 ** -148 * (d * u).abs() * (1 + g.abs()) + 2.0 ** -134)
    _inside(got[:, f:], du, (2.0 ** -8 + noise) * du.abs() + 2.0 ** -148 * (d * g).abs() + 2.0 ** -134)
