"""The norm's forward pass rounds the residual stream as its definition does, operation by operation in FP32.

The norm's factor follows the stored y, and in a strong channel one y that rounds the other way moves it by far more
than FP32's rounding.  So y is compared bit for bit with separate operations on FP32 tensors, in the order of the
definition, from the factor that the call returned; and the returned factor with 64 bits from the returned y."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fp8():
    import fp8_block_scaled_13_b200 as m
    from fp8_block_scaled_13_b200 import build
    build.build()
    return m


def _inputs(t, d, post, gate, wt, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = randn(t, d)
    x[:, :: max(1, d // 8)] *= 20.0   # strong channels
    kw = {}
    if post:
        kw["w_post"] = (1 + 0.1 * randn(d)).to(wt)
    if gate:
        shape = {"token": (t, 1), "channel": (1, d), "full": (t, d)}[gate]
        kw["gate"] = (1 + 0.3 * randn(*shape)).to(torch.bfloat16 if gate == "full" else wt)
    return x.to(torch.bfloat16), (1 + 0.1 * randn(d)).to(wt), randn(t, d).to(torch.bfloat16), kw


def _stream(x, h, scale, rstd_post, w_post=None, gate=None):
    hn = h.float()
    if w_post is not None:
        hn = hn * rstd_post[:, None] * w_post.float()
    if gate is not None:
        hn = hn * gate.float()
    return (x.float() + scale * hn).to(torch.bfloat16)


@pytest.mark.parametrize("t,d", [(3000, 2048), (9001, 1152), (4500, 4096), (2500, 8192)])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", [None, "token", "channel", "full"])
def test_the_stream_rounds_in_the_definitions_order(fp8, t, d, post, gate):
    wt = torch.float32 if t % 2 else torch.bfloat16
    x, w, h, kw = _inputs(t, d, post, gate, wt, t + d)
    for scale in (0.3, 0.5):
        r = fp8.residual_norm(x, w, h, scale=scale, layout="rowwise", **kw)
        assert torch.equal(r.y, _stream(x, h, scale, r.rstd_post, **kw))
        # a sum of squares in FP32, 45 additions deep, one division and one square root: below 64 operations of 2^-24
        want = (r.y.double().square().mean(1) + 1e-6) ** -0.5
        assert ((r.rstd.double() - want).abs() <= 2.0 ** -18 * want).all()
        if post:
            want = (h.double().square().mean(1) + 1e-6) ** -0.5
            assert ((r.rstd_post.double() - want).abs() <= 2.0 ** -18 * want).all()
    assert fp8.device_status() == 0
