"""The operators around the linear layers together, as a training step of an FFN block uses them: norm, gate+up
projection, gated activation, down projection, norm after the block with a gate, backward through all of them into
FP32 main gradients, and the orthogonalised updates of both weights."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fp8():
    import fp8_block_scaled_13_b200 as m
    from fp8_block_scaled_13_b200 import build
    build.build()
    return m


def _tensors(t, d, f, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    bf = torch.bfloat16
    return dict(x=r(t, d).to(bf), w1=(r(2 * f, d) * d ** -0.5).to(bf), w2=(r(d, f) * f ** -0.5).to(bf),
                n1=1 + 0.1 * r(d), n2=1 + 0.1 * r(d), post=1 + 0.1 * r(d), gate=(1 + 0.1 * r(1, d)),
                dn=(r(t, d) * 1e-2).to(bf), dy=(r(t, d) * 1e-2).to(bf))


def _step(fp8, v, main, codes):
    """One step; with codes=False every result leaves as BF16 and the quantizer takes it from there."""
    layout = "both" if codes else "bf16"
    q = (lambda a: a) if codes else fp8.quant_act
    a = fp8.residual_norm(v["x"], v["n1"], layout=layout)
    gu, xq1, wq1 = fp8.linear_forward(q(a.n), v["w1"])
    h, xq2, wq2 = fp8.linear_forward(q(fp8.swiglu(gu, layout=layout)), v["w2"])
    b = fp8.residual_norm(a.y, v["n2"], h, w_post=v["post"], gate=v["gate"], scale=0.5, layout=layout)
    gb = fp8.residual_norm_backward(v["dn"], b.y, b.rstd, v["n2"], h, dy=v["dy"], w_post=v["post"],
                                    rstd_post=b.rstd_post, gate=v["gate"], scale=0.5, layout=layout)
    da, _ = fp8.linear_backward(q(gb.dh), xq2, wq2, main_grad=main[1])
    dn1, _ = fp8.linear_backward(q(fp8.swiglu_backward(da, gu, layout=layout)), xq1, wq1, main_grad=main[0])
    ga = fp8.residual_norm_backward(dn1, v["x"], a.rstd, v["n1"], dy=gb.dx)
    updates = [fp8.orthogonalize(m) for m in main]
    return [b.y, ga.dx, ga.dw_pre, gb.dw_pre, gb.dw_post, gb.dgate, *main, *updates]


@pytest.mark.parametrize("t,d,f", [(256, 256, 512), (1000, 512, 384), (77, 1152, 640)])
def test_codes_give_what_the_quantizer_gives(fp8, t, d, f):
    v = _tensors(t, d, f, t)
    res = []
    for codes in (True, False):
        main = [torch.zeros(2 * f, d, device="cuda"), torch.zeros(d, f, device="cuda")]
        _step(fp8, v, main, codes)
        res.append(_step(fp8, v, main, codes))   # a second micro-batch is added
    for i, (a, b) in enumerate(zip(*res)):
        assert torch.equal(a, b), i
    assert fp8.device_status() == 0


def test_gradients_against_the_step_in_64_bits(fp8):
    """The FP8 step against autograd through the same block in 64 bits.  Every product takes two E4M3 operands, each
    off by at most 2^-4 of a value, evenly spread over a half step: 2^-4 / sqrt(3) = 3.6 % in the mean square, so 5.1 %
    for a product.  The deepest gradient passes six of them (three forward, whose results it multiplies, and three
    backward), sqrt(6) * 5.1 % = 12.5 % when the roundings are independent; twice that is allowed."""
    t, d, f = 512, 256, 512
    v = _tensors(t, d, f, 1)
    main = [torch.zeros(2 * f, d, device="cuda"), torch.zeros(d, f, device="cuda")]
    got = _step(fp8, v, main, True)
    z = {k: a.double().requires_grad_() for k, a in v.items() if k not in ("dn", "dy")}
    rms = lambda a, w: a * (a.square().mean(1, keepdim=True) + 1e-6) ** -0.5 * w  # noqa: E731
    gu = rms(z["x"], z["n1"]) @ z["w1"].T
    h = (torch.nn.functional.silu(gu[:, :f]) * gu[:, f:]) @ z["w2"].T
    y = z["x"] + 0.5 * z["gate"] * rms(h, z["post"])
    torch.autograd.backward([rms(y, z["n2"]), y], [v["dn"].double(), v["dy"].double()])
    want = [y, z["x"].grad, z["n1"].grad, z["n2"].grad, z["post"].grad, z["gate"].grad, z["w1"].grad, z["w2"].grad]
    for i, (a, b) in enumerate(zip(got, want)):
        err = ((a.double() - b).norm() / b.norm()).item()
        assert err <= 0.25, (i, err)


def test_a_captured_step(fp8):
    """The whole step in a CUDA graph on a side stream, replayed on other inputs, while an eager step runs beside it."""
    t, d, f = 384, 512, 384
    v, other = _tensors(t, d, f, 1), _tensors(t, d, f, 2)
    shapes = [(2 * f, d), (d, f)]
    zeros = lambda: [torch.zeros(s, device="cuda") for s in shapes]  # noqa: E731
    want = [_step(fp8, u, zeros(), True) for u in (v, other)]
    held = {k: a.clone() for k, a in v.items()}
    main = zeros()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for m in main:
            m.zero_()
        res = _step(fp8, held, main, True)
    side = torch.cuda.Stream()
    for u, w in zip((v, other, v), (want[0], want[1], want[0])):
        for k, a in held.items():
            a.copy_(u[k])
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            eager = _step(fp8, other, zeros(), True)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(res, w):
            assert torch.equal(a, b)
        for a, b in zip(eager, want[1]):
            assert torch.equal(a, b)
    assert fp8.device_status() == 0
