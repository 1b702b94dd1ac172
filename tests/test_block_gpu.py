"""Norms around a block and gated activation on the GPU, against 64-bit forms.

BF16 results and sums are held to bounds derived in block_reference.py.  Codes
have to be, bit for bit, what the oracle's quantizer gives for the kernel's own
BF16 result of the same inputs."""
import numpy as np
import pytest
import torch

import block_reference as ref
from helpers import gpu_colwise, gpu_rowwise

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.fixture(scope="module")
def fp8():
    import fp8_block_scaled_13_b200 as m
    from fp8_block_scaled_13_b200 import build
    build.build()
    return m


def _bf(shape, seed, std=1.0, ld=None):
    """A BF16 matrix; with ld, a view into a wider one whose other columns hold NaN."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    v = (torch.randn(*shape, generator=g, device="cuda") * std).to(torch.bfloat16)
    if ld:
        wide = torch.full((shape[0], ld), float("nan"), dtype=torch.bfloat16, device="cuda")
        wide[:, :shape[1]] = v
        v = wide[:, :shape[1]]
    return v


def _close(got, want, bound, what):
    got = got.double()
    assert got.shape == want.shape, what
    worst = ((got - want).abs() - bound).max().item() if want.numel() else -1.0
    assert worst <= 0, "%s: off by %.3g more than its bound" % (what, worst)


def _same_codes(qa, bf, oracle_mod, layout):
    """qa holds the oracle's codes and scales of the BF16 tensor, pads included."""
    host = bf.cpu()
    if layout in ("rowwise", "both"):
        q, s = gpu_rowwise(qa)
        oq, os_ = oracle_mod.quant_rowwise(host)
        assert np.array_equal(s, os_) and np.array_equal(q, oq)
        groups = qa.cols // 128
        rows_up = (qa.rows + 127) // 128 * 128
        from helpers import unblock
        assert (unblock(qa.s, rows_up, groups)[qa.rows:] == 127).all()
    if layout in ("colwise", "both"):
        qt, st, pad = gpu_colwise(qa)
        oqt, ost = oracle_mod.quant_colwise(host)
        assert np.array_equal(st, ost) and np.array_equal(qt, oqt)
        assert not pad.any()


def _inputs(t, d, res, post, gate, w32, seed, ld=None):
    wt = torch.float32 if w32 else torch.bfloat16
    k = {"w_post": (1 + 0.2 * torch.randn(d, device="cuda")).to(wt) if post else None, "gate": None}
    x = _bf((t, d), seed, 2.0, ld)
    h = _bf((t, d), seed + 1, 0.5, ld) if res else None
    if gate == "token":
        k["gate"] = torch.randn(t, 1, device="cuda").to(wt)
    elif gate == "channel":
        k["gate"] = torch.randn(1, d, device="cuda").to(wt)
    elif gate == "full":
        k["gate"] = _bf((t, d), seed + 2, 1.0, ld)
    if res and t > 2:
        h[1] = 0   # a block that adds nothing to a token
        x[2] = 0
        h[2] = 0   # and a token that is zero altogether
    return x, (1 + 0.2 * torch.randn(d, device="cuda")).to(wt), h, k


# variants by width (up to 2048, 4096 and 8192 columns), rows around the 16 of a CTA and the 128 of a group
SHAPES = [(1, 128), (2, 384), (15, 2048), (16, 1152), (17, 2048), (127, 640), (128, 2048), (129, 256), (300, 2176),
          (200, 4096), (130, 4224), (40, 8192), (1000, 1024)]
KINDS = [(False, False, None), (True, False, None), (True, True, None), (True, False, "token"), (True, True, "token"),
         (True, False, "channel"), (True, True, "channel"), (True, False, "full"), (True, True, "full")]


@pytest.mark.parametrize("t,d", SHAPES)
@pytest.mark.parametrize("res,post,gate", KINDS)
def test_norm_forward(fp8, oracle_mod, t, d, res, post, gate):
    seed = t * 7 + d
    torch.manual_seed(seed)
    x, w, h, k = _inputs(t, d, res, post, gate, (t + d // 128) % 2 == 0, seed, ld=d + 64 if t % 2 else None)
    r = fp8.residual_norm(x, w, h, scale=0.75, eps=EPS, layout="bf16", **k)
    y, ybound, r1 = ref.norm_forward(x, h, k["w_post"], k["gate"], 0.75, EPS)
    _close(r.y, y, ybound, "y")
    n, nbound, r2 = ref.norm_of(r.y, w, EPS)
    _close(r.n, n, nbound, "n")
    _close(r.rstd, r2, ref.NOISE * r2, "rstd")
    if post:
        _close(r.rstd_post, r1, ref.NOISE * r1, "rstd_post")
    for layout in ("rowwise", "colwise", "both"):
        c = fp8.residual_norm(x, w, h, scale=0.75, eps=EPS, layout=layout, **k)
        assert torch.equal(c.y, r.y) and torch.equal(c.rstd, r.rstd)
        _same_codes(c.n, r.n, oracle_mod, layout)
    assert fp8.device_status() == 0


@pytest.mark.parametrize("t,d", SHAPES)
@pytest.mark.parametrize("res,post,gate", KINDS)
def test_norm_backward(fp8, oracle_mod, t, d, res, post, gate):
    seed = t * 5 + d
    torch.manual_seed(seed)
    x, w, h, k = _inputs(t, d, res, post, gate, (t + d // 128) % 2 == 1, seed, ld=d + 64 if t % 2 else None)
    f = fp8.residual_norm(x, w, h, scale=0.75, eps=EPS, layout="bf16", **k)
    dn = _bf((t, d), seed + 3, 1e-2)
    dy = _bf((t, d), seed + 4, 1e-2, ld=d + 8) if t % 3 else None
    args = (dn, f.y, f.rstd, w, h)
    kw = dict(dy=dy, rstd_post=f.rstd_post, scale=0.75, **k)
    want = ref.norm_backward(dn, f.y, f.rstd, w, h, dy, k["w_post"], f.rstd_post, k["gate"], 0.75)
    r = fp8.residual_norm_backward(*args, layout="bf16", **kw)
    for name, (value, bound) in want.items():
        _close(getattr(r, name).reshape(value.shape), value, bound, name)
    if not res:
        assert r.dh is None
        return
    for layout in ("rowwise", "colwise", "both"):
        c = fp8.residual_norm_backward(*args, layout=layout, **kw)
        for name in ("dx", "dw_pre", "dw_post", "dgate"):
            a, b = getattr(c, name), getattr(r, name)
            assert (a is None and b is None) or torch.equal(a, b), name
        _same_codes(c.dh, r.dh, oracle_mod, layout)
    assert fp8.device_status() == 0


def test_norm_accumulates_weight_gradients(fp8):
    t, d = 300, 256
    torch.manual_seed(1)
    x, w, h, k = _inputs(t, d, True, True, "channel", True, 1)
    f = fp8.residual_norm(x, w, h, **k)
    dn = _bf((t, d), 5)
    args, kw = (dn, f.y, f.rstd, w, h), dict(rstd_post=f.rstd_post, **k)
    one = fp8.residual_norm_backward(*args, **kw)
    bufs = {n: torch.full_like(getattr(one, n), 0.5) for n in ("dw_pre", "dw_post", "dgate")}
    fp8.residual_norm_backward(*args, accumulate=True, **bufs, **kw)
    for n, b in bufs.items():
        assert torch.equal(b, 0.5 + getattr(one, n)), n


def test_norm_without_rows(fp8):
    x = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(256, device="cuda")
    r = fp8.residual_norm(x, w, x.clone(), w_post=w, gate=w[None])
    assert r.y.shape == (0, 256) and r.n.rows == 0
    g = fp8.residual_norm_backward(x, x, r.rstd, w, x.clone(), w_post=w, rstd_post=r.rstd_post, gate=w[None])
    for v in (g.dw_pre, g.dw_post, g.dgate):
        assert not v.any()


def test_norm_in_place(fp8):
    t, d = 77, 640
    torch.manual_seed(2)
    x, w, h, k = _inputs(t, d, True, True, "full", True, 2)
    want = fp8.residual_norm(x, w, h, **k)
    for dst in (x.clone(), h.clone()):
        a = (dst, h) if dst.data_ptr() and torch.equal(dst, x) else (x, dst)
        got = fp8.residual_norm(a[0], w, a[1], y=dst, **k)
        assert got.y is dst and torch.equal(got.y, want.y) and torch.equal(got.n.q, want.n.q)
    dn, dy = _bf((t, d), 3), _bf((t, d), 4)
    kw = dict(w_post=k["w_post"], gate=k["gate"], rstd_post=want.rstd_post)
    plain = fp8.residual_norm_backward(dn, want.y, want.rstd, w, h, dy=dy, **kw)
    for i in range(3):
        src = [dn.clone(), want.y.clone(), dy.clone()]
        got = fp8.residual_norm_backward(src[0], src[1], want.rstd, w, h, dy=src[2], dx=src[i], **kw)
        assert torch.equal(got.dx, plain.dx) and torch.equal(got.dh.qt, plain.dh.qt)


def test_norm_offsets_past_32_bits(fp8):
    """Over 2^31 elements: the last rows come out as they do by themselves."""
    t, d = 1_060_000, 2048
    x = torch.zeros(t, d, dtype=torch.bfloat16, device="cuda")
    x[-130:] = _bf((130, d), 1)
    w = torch.ones(d, device="cuda")
    q = torch.empty(t, d, dtype=torch.uint8, device="cuda")
    s = torch.empty((t + 127) // 128 * 4 * 512, dtype=torch.uint8, device="cuda")
    r = fp8.residual_norm(x, w, layout="rowwise", out=fp8.QuantAct(t, d, q=q, s=s))
    small = fp8.residual_norm(x[-130:].clone(), w, layout="rowwise")
    assert torch.equal(r.n.q[-130:], small.n.q) and torch.equal(r.rstd[-130:], small.rstd)


GATED = [(1, 128), (7, 256), (128, 128), (129, 384), (300, 1408), (1000, 640), (2000, 2048)]


def _gu(t, f, seed, ld=None):
    gu = _bf((t, 2 * f), seed, 3.0, ld)
    gu[0, :4] = torch.tensor([-90.0, -200.0, 90.0, 0.0], device="cuda")  # sigmoid saturates
    return gu


@pytest.mark.parametrize("t,f", GATED)
def test_swiglu(fp8, oracle_mod, t, f):
    gu = _gu(t, f, t + f, ld=2 * f + 8 if t % 2 else None)
    a = fp8.swiglu(gu, layout="bf16")
    _close(a, *ref.swiglu(gu), "a")
    for layout in ("rowwise", "colwise", "both"):
        _same_codes(fp8.swiglu(gu, layout=layout), a, oracle_mod, layout)
    assert fp8.device_status() == 0


@pytest.mark.parametrize("t,f", GATED)
def test_swiglu_backward(fp8, oracle_mod, t, f):
    gu = _gu(t, f, t + f, ld=2 * f + 8 if t % 2 else None)
    da = _bf((t, f), 9, 1e-2, ld=f + 16 if t % 2 else None)
    d = fp8.swiglu_backward(da, gu, layout="bf16")
    _close(d, *ref.swiglu_backward(da, gu), "dgu")
    for layout in ("rowwise", "colwise", "both"):
        _same_codes(fp8.swiglu_backward(da, gu, layout=layout), d, oracle_mod, layout)
    assert fp8.device_status() == 0


def test_backward_offsets_past_32_bits(fp8):
    """Over 2^31 elements: the last rows' gradients come out as they do by themselves."""
    t, d = 1_060_000, 2048
    x = torch.zeros(t, d, dtype=torch.bfloat16, device="cuda")
    x[-130:] = _bf((130, d), 1)
    dn = torch.zeros(t, d, dtype=torch.bfloat16, device="cuda")
    dn[-130:] = _bf((130, d), 2)
    w = torch.ones(d, device="cuda")
    f = fp8.residual_norm(x, w, layout="bf16")
    big = fp8.residual_norm_backward(dn, x, f.rstd, w, layout="bf16")
    small = fp8.residual_norm_backward(dn[-130:].clone(), x[-130:].clone(), f.rstd[-130:].clone(), w, layout="bf16")
    assert torch.equal(big.dx[-130:], small.dx) and torch.allclose(big.dw_pre, small.dw_pre, rtol=1e-4, atol=1e-3)
    del f, big, x, dn
    t, f = 180_000, 6144
    gu = torch.zeros(t, 2 * f, dtype=torch.bfloat16, device="cuda")
    gu[-130:] = _bf((130, 2 * f), 3)
    # (a group of transposed codes is 128 rows from the start: 180000 = 1406 * 128 + 32)
    a, b = fp8.swiglu(gu), fp8.swiglu(gu[-160:].clone())
    assert torch.equal(a.q[-160:], b.q) and torch.equal(a.qt[:, t - 160:], b.qt[:, :160])


@pytest.mark.parametrize("t,d", [(70, 384), (300, 2176), (129, 4224)])
def test_norm_weights_off_16_byte_boundaries(fp8, t, d):
    torch.manual_seed(t)
    x, _, h, _ = _inputs(t, d, True, True, None, True, t)
    dn = _bf((t, d), 9)
    for wt in (torch.float32, torch.bfloat16):
        w, wp, gate = [(1 + 0.2 * torch.randn(d, device="cuda")).to(wt) for _ in range(3)]
        off = [torch.cat([v[:1], v])[1:] for v in (w, wp, gate)]   # one element into their memory
        assert all(v.data_ptr() % 16 for v in off)
        a = fp8.residual_norm(x, w, h, w_post=wp, gate=gate[None])
        b = fp8.residual_norm(x, off[0], h, w_post=off[1], gate=off[2][None])
        assert torch.equal(a.y, b.y) and torch.equal(a.n.q, b.n.q) and torch.equal(a.n.qt, b.n.qt)
        kw = dict(rstd_post=a.rstd_post)
        ga = fp8.residual_norm_backward(dn, a.y, a.rstd, w, h, w_post=wp, gate=gate[None], **kw)
        gb = fp8.residual_norm_backward(dn, a.y, a.rstd, off[0], h, w_post=off[1], gate=off[2][None], **kw)
        for n in ("dx", "dw_pre", "dw_post", "dgate"):
            assert torch.equal(getattr(ga, n), getattr(gb, n)), n
        assert torch.equal(ga.dh.qt, gb.dh.qt)


def test_a_token_does_not_see_its_neighbours(fp8):
    """A token's result is the same alone and in a batch, and one that is not a number stays by itself."""
    for d in (256, 2048, 4224):
        x, h = _bf((700, d), d), _bf((700, d), d + 1)
        w = 1 + 0.2 * torch.randn(d, device="cuda")
        r = fp8.residual_norm(x, w, h, w_post=w, layout="bf16")
        for i in (0, 15, 16, 333, 699):
            one = fp8.residual_norm(x[i:i + 1], w, h[i:i + 1], w_post=w, layout="bf16")
            assert torch.equal(one.n[0], r.n[i]) and torch.equal(one.y[0], r.y[i])
        x[333] = float("nan")
        bad = fp8.residual_norm(x, w, h, w_post=w, layout="bf16")
        keep = torch.arange(700, device="cuda") != 333
        assert torch.equal(bad.n[keep], r.n[keep]) and bad.n[333].isnan().all()


def test_only_the_results_are_written(fp8):
    """Wider buffers: what lies beside the results keeps its bytes."""
    t, d = 150, 384
    x, h, dn, gu = _bf((t, d), 1), _bf((t, d), 2), _bf((t, d), 3), _bf((t, 2 * d), 4)
    w = torch.ones(d, device="cuda")

    def buffers(cols):
        q = torch.full((t + 9, cols + 32), 9, dtype=torch.uint8, device="cuda")
        qt = torch.full((cols + 3, 160 + 48), 9, dtype=torch.uint8, device="cuda")
        fresh = fp8.quant_act(torch.zeros(t, cols, dtype=torch.bfloat16, device="cuda"))
        return q, qt, fp8.QuantAct(t, cols, q=q[:t, :cols], s=fresh.s, qt=qt[:cols, :160], st=fresh.st)

    def check(q, qt, cols):
        assert (q[t:] == 9).all() and (q[:, cols:] == 9).all() and (qt[cols:] == 9).all() and (qt[:, 160:] == 9).all()

    wide = [torch.full((t + 5, d + 64), -3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    q, qt, out = buffers(d)
    r = fp8.residual_norm(x, w, h, y=wide[0][:t, :d], out=out)
    check(q, qt, d)
    q, qt, out = buffers(d)
    fp8.residual_norm_backward(dn, r.y, r.rstd, w, h, dx=wide[1][:t, :d], out=out)
    check(q, qt, d)
    for v in wide:
        assert (v[t:] == -3).all() and (v[:, d:] == -3).all()
    q, qt, out = buffers(d)
    fp8.swiglu(gu, out=out)
    check(q, qt, d)
    q, qt, out = buffers(2 * d)
    fp8.swiglu_backward(dn, gu, out=out)
    check(q, qt, 2 * d)


def test_repeatable(fp8):
    """Sums over tokens are added in a fixed order, whatever CTA takes which rows or tile."""
    t, d = 5000, 2048
    x, h, dn = _bf((t, d), 1), _bf((t, d), 2), _bf((t, d), 3)
    w = 1 + 0.1 * torch.randn(d, device="cuda")
    f = fp8.residual_norm(x, w, h, w_post=w)
    one = fp8.residual_norm_backward(dn, f.y, f.rstd, w, h, w_post=w, rstd_post=f.rstd_post)
    for _ in range(5):
        r = fp8.residual_norm_backward(dn, f.y, f.rstd, w, h, w_post=w, rstd_post=f.rstd_post)
        assert torch.equal(r.dw_pre, one.dw_pre) and torch.equal(r.dw_post, one.dw_post)
        assert torch.equal(r.dh.q, one.dh.q) and torch.equal(r.dh.qt, one.dh.qt)


def test_wrapper_refusals(fp8):
    """Whatever does not fit is refused before any launch, with the name of the argument."""
    t, d = 16, 256
    x, h, w = _bf((t, d), 1), _bf((t, d), 2), torch.ones(d, device="cuda")
    f = fp8.residual_norm(x, w, h, w_post=w)
    n = lambda *a, **k: lambda: fp8.residual_norm(*a, **k)  # noqa: E731
    b = lambda *a, **k: lambda: fp8.residual_norm_backward(*a, **k)  # noqa: E731
    args = (x, f.y, f.rstd, w, h)
    other = fp8.residual_norm(_bf((t, 128), 1), w[:128]).n
    rowwise = fp8.residual_norm(x, w, layout="rowwise").n
    for match, call in [
            ("layout", n(x, w, layout="columns")), ("eps", n(x, w, eps=0.0)), ("x must", n(x.float(), w)),
            ("x must", n(x.T, w)), ("x must", n(x[0], w)), ("w_pre must", n(x, w[:-1])), ("w_pre must", n(x, w.half())),
            ("w_pre must", n(x, torch.ones(2 * d, device="cuda")[::2])), ("one type", n(x, w, h, w_post=w.bfloat16())),
            ("h must", n(x, w, h[:-1])), ("missing", n(x, w, gate=w[None])), ("missing", n(x, w, w_post=w)),
            ("only written", n(x, w, y=x)), ("y must", n(x, w, h, y=x.float())), ("gate must", n(x, w, h, gate=w)),
            ("gate must", n(x, w, h, gate=w[None].half())), ("per element", n(x, w, h, gate=x.float())),
            ("per token", n(x, w, h, gate=torch.ones(2 * t, 1, device="cuda")[::2])),
            ("QuantAct", n(x, w, out=other)), ("QuantAct", n(x, w, out=x)), ("transposed codes", n(x, w, out=rowwise)),
            ("BF16 tensor", n(x, w, layout="bf16", out=rowwise)), ("out must", n(x, w, layout="bf16", out=x[:-1])),
            ("CUDA", n(x.cpu(), w.cpu())), ("different devices", n(x, w.cpu())),
            ("y must", b(x, f.y[:-1], f.rstd, w)), ("rstd must", b(x, f.y, f.rstd[:-1], w)),
            ("rstd_post", b(*args, w_post=w)), ("rstd_post must", b(*args, w_post=w, rstd_post=f.rstd_post.double())),
            ("missing", b(x, f.y, f.rstd, w, out=rowwise)), ("need w_post", b(*args, dw_post=w)),
            ("need w_post", b(*args, dgate=w)), ("accumulate", b(*args, accumulate=True)),
            ("accumulate", b(*args, gate=w[None], dw_pre=w, accumulate=True)), ("dw_pre must", b(*args, dw_pre=w[:-1])),
            ("dgate must", b(*args, gate=w[None], dgate=w)), ("dx must", b(*args, dx=w)), ("dy must", b(*args, dy=x[:-1])),
            ("two halves", lambda: fp8.swiglu(torch.zeros(4, 257, dtype=torch.bfloat16, device="cuda"))),
            ("gu must", lambda: fp8.swiglu_backward(x, x))]:
        with pytest.raises(ValueError, match=match):
            call()
    for wrong in (None, 3, "x"):
        with pytest.raises(TypeError, match="tensor"):
            fp8.swiglu(wrong)
    with pytest.raises(fp8_error(fp8)):   # a width that the library does not take
        fp8.residual_norm(_bf((4, 200), 1), torch.ones(200, device="cuda"), layout="bf16")
    assert fp8.device_status() == 0


def fp8_error(fp8):
    from fp8_block_scaled_13_b200._lib import PuroError
    return PuroError


def test_on_another_stream_than_the_tensors(fp8):
    """Calls go to the current stream; memory that a side stream still writes is waited for by that stream's order."""
    t, d = 4096, 2048
    w = 1 + 0.1 * torch.randn(d, device="cuda")
    src, da = _bf((t, 2 * d), 1), _bf((t, d), 2)
    want = [fp8.swiglu(src).q.clone(), fp8.residual_norm(src[:, :d].contiguous(), w).n.qt.clone(),
            fp8.swiglu_backward(da, src).qt.clone()]
    side = torch.cuda.Stream()
    x = torch.zeros_like(src)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(20):
            x.mul_(0.5)     # work in front of the copy
        x.copy_(src)
        got = [fp8.swiglu(x).q, fp8.residual_norm(x[:, :d].contiguous(), w).n.qt, fp8.swiglu_backward(da, x).qt]
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
