"""Column gradients of the norms over very many tokens, against 64 bits: the error does not grow with the rows."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fp8():
    import fp8_block_scaled_13_b200 as m
    from fp8_block_scaled_13_b200 import build
    build.build()
    return m


def test_sums_over_a_million_rows(fp8):
    """Rows alike, so that every addition of the CTAs' sums would round the same way."""
    t, d = 1 << 20, 128
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(1, d, generator=g, device="cuda").to(torch.bfloat16).expand(t, d).contiguous()
    dn = torch.rand(1, d, generator=g, device="cuda").to(torch.bfloat16).expand(t, d).contiguous()
    w = torch.ones(d, device="cuda")
    f = fp8.residual_norm(x, w, x, w_post=w, layout="bf16")
    b = fp8.residual_norm_backward(dn, f.y, f.rstd, w, x, w_post=w, rstd_post=f.rstd_post, layout="bf16")
    nh = f.y[0].double() * f.rstd[0].double()
    one = dn[0].double() * nh
    # 4 operations, 32 rows in a thread and one rounding of the result: 2^-18 allows 64 of 2^-24
    assert ((b.dw_pre.double() - t * one).abs() <= 2.0 ** -18 * t * one.abs()).all()
    dY = f.rstd[0].double() * (dn[0].double() - nh * one.mean())
    size = f.rstd[0].double() * (dn[0].double() + nh.abs() * one.abs().mean())
    hh = x[0].double() * f.rstd_post[0].double()
    assert ((b.dw_post.double() - t * dY * hh).abs() <= 2.0 ** -17 * t * size * hh.abs()).all()
