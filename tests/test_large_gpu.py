"""Tensors of more than 2^31 elements: the norms with every input and both kinds of codes, and the orthogonalisation."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fp8():
    import fp8_block_scaled_13_b200 as m
    from fp8_block_scaled_13_b200 import build
    build.build()
    return m


def test_norms(fp8):
    """The last 128 rows, a group of the transposed codes, come out as they do by themselves."""
    t, d, last = 8282 * 128, 2048, 128
    g = torch.Generator(device="cuda").manual_seed(1)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731

    def tall(seed_rows):
        v = torch.zeros(t, d, dtype=torch.bfloat16, device="cuda")
        v[-last:] = seed_rows
        return v

    x, h, gate, dn, dy = (tall(randn(last, d).to(torch.bfloat16)) for _ in range(5))
    w, wp = 1 + 0.1 * randn(d), 1 + 0.1 * randn(d)
    assert x.numel() > 2 ** 31
    end = lambda v: v[-last:].clone()  # noqa: E731
    f = fp8.residual_norm(x, w, h, w_post=wp, gate=gate, scale=0.5)
    s = fp8.residual_norm(end(x), w, end(h), w_post=wp, gate=end(gate), scale=0.5)
    assert torch.equal(f.y[-last:], s.y) and torch.equal(f.rstd[-last:], s.rstd)
    assert torch.equal(f.n.q[-last:], s.n.q) and torch.equal(f.n.qt[:, -last:], s.n.qt)
    f.n = None
    b = fp8.residual_norm_backward(dn, f.y, f.rstd, w, h, dy=dy, w_post=wp, rstd_post=f.rstd_post, gate=gate, scale=0.5)
    r = fp8.residual_norm_backward(end(dn), s.y, s.rstd, w, end(h), dy=end(dy), w_post=wp, rstd_post=s.rstd_post,
                                   gate=end(gate), scale=0.5)
    for name in ("dx", "dgate"):
        assert torch.equal(getattr(b, name)[-last:], getattr(r, name)), name
    assert torch.equal(b.dh.q[-last:], r.dh.q) and torch.equal(b.dh.qt[:, -last:], r.dh.qt)
    # the other rows add zeros; the order of the additions differs: 32 rows in a thread against fewer, 2^-18 of the sums
    for name, rows in (("dw_pre", end(dn).double() * s.y.double() * s.rstd.double()[:, None]),):
        assert ((getattr(b, name).double() - getattr(r, name).double()).abs() <= 2.0 ** -18 * rows.abs().sum(0)).all()
    assert fp8.device_status() == 0


def test_orthogonalize(fp8):
    """A gradient of 2 x 2 blocks on the diagonal: its products stay there, so that each block follows the iteration by
    itself, from the whole gradient's norm.  Entries are few and alike, so the rounding of the result is half a step of
    2^-8 at most, and 30 roundings of the operands add 2^-10 each at most (a step of FP16), two entries to a sum."""
    n, k = 65536, 32896
    block = torch.tensor([[1.0, 0.5], [-0.25, 1.0]], device="cuda")
    g = torch.zeros(n, k, dtype=torch.bfloat16, device="cuda")
    assert g.numel() > 2 ** 31
    i = torch.arange(0, k, 2, device="cuda")
    rows = i + (n - k)   # the last rows: the furthest offsets
    for a in range(2):
        for b in range(2):
            g[rows + a, i + b] = block[a, b].to(torch.bfloat16)
    out = fp8.orthogonalize(g)
    assert fp8.device_status() == 0
    x = block.double() / (k / 2 * block.double().square().sum()) ** 0.5
    for _ in range(5):
        m = x @ x.T
        x = 3.4445 * x + (-4.7750 * m + 2.0315 * m @ m) @ x
    size = x.abs().max()
    for a in range(2):
        for b in range(2):
            got = out[rows + a, i + b].double()
            assert ((got - x[a, b]).abs() <= 2.0 ** -8 * size + 30 * 2.0 ** -10 * size).all(), (a, b)
            out[rows + a, i + b] = 0
    assert not out.any()
