"""Norms over many rows: a CTA's loop goes round several times, so that every stage of its ring is filled again, with
every tensor in it, on each of the three widths of kernel; and the sums over tokens of long batches.

The bounds are block_reference's.  Its NOISE of 2^-17 allows 128 operations of 2^-24.  A value that a row pass forms
takes at most 20 operations and a sum over a row of depth 45 (8 in a thread, 5 in a warp, 32 warps); a sum over tokens
32 rows in a thread, and the CTAs' sums are added in 64 bits and rounded once, whatever the number of rows."""
import numpy as np
import pytest
import torch

import block_reference as ref
from helpers import gpu_colwise, gpu_rowwise

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fp8():
    import fp8_block_scaled_13_b200 as m
    from fp8_block_scaled_13_b200 import build
    build.build()
    return m


def _inputs(t, d, post, gate, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    bf = torch.bfloat16
    x = randn(t, d)
    x[:, :: max(1, d // 8)] *= 20.0   # strong channels
    kw = {"w_post": 1 + 0.1 * randn(d) if post else None, "gate": None}
    if gate:
        shape = {"token": (t, 1), "channel": (1, d), "full": (t, d)}[gate]
        kw["gate"] = (1 + 0.3 * randn(*shape)).to(bf if gate == "full" else torch.float32)
    # (gradients of non-zero mean: the sums over tokens grow with the rows)
    return x.to(bf), 1 + 0.1 * randn(d), (0.3 + randn(t, d)).to(bf), kw, (0.5 + randn(t, d)).to(bf), randn(t, d).to(bf)


def _inside(got, want, bound, what):
    worst = ((got.double() - want).abs() - bound).max().item()
    assert worst <= 0, "%s: off by %.3g more than its bound" % (what, worst)


def _same_codes(fp8, qa, bf):
    want = fp8.quant_act(bf)
    assert torch.equal(qa.q, want.q) and torch.equal(qa.qt, want.qt)
    for a, b in zip(gpu_rowwise(qa)[1:] + gpu_colwise(qa)[1:2], gpu_rowwise(want)[1:] + gpu_colwise(want)[1:2]):
        assert np.array_equal(a, b)


# as many rows as give a CTA its full share: 16 (32 where it fills an SM) forward, 32 backward; the last one ragged
SHAPES = [(9600, 2048), (9501, 640), (4801, 4096), (4750, 5248)]
KINDS = [(False, None), (True, None), (True, "token"), (False, "channel"), (True, "channel"), (True, "full")]


@pytest.mark.parametrize("t,d", SHAPES)
@pytest.mark.parametrize("post,gate", KINDS)
def test_against_64_bits(fp8, t, d, post, gate):
    x, w, h, kw, dn, dy = _inputs(t, d, post, gate, t + d)
    f = fp8.residual_norm(x, w, h, scale=0.75, layout="bf16", **kw)
    y, bound, r1 = ref.norm_forward(x, h, kw["w_post"], kw["gate"], 0.75, 1e-6)
    _inside(f.y, y, bound, "y")
    n, bound, r2 = ref.norm_of(f.y, w, 1e-6)
    _inside(f.n, n, bound, "n")
    _inside(f.rstd, r2, ref.NOISE * r2, "rstd")
    if post:
        _inside(f.rstd_post, r1, ref.NOISE * r1, "rstd_post")
    c = fp8.residual_norm(x, w, h, scale=0.75, **kw)
    assert torch.equal(c.y, f.y) and torch.equal(c.rstd, f.rstd)
    _same_codes(fp8, c.n, f.n)
    del y, n, bound, c

    args, more = (dn, f.y, f.rstd, w, h), dict(dy=dy, rstd_post=f.rstd_post, scale=0.75, **kw)
    b = fp8.residual_norm_backward(*args, layout="bf16", **more)
    want = ref.norm_backward(dn, f.y, f.rstd, w, h, dy, kw["w_post"], f.rstd_post, kw["gate"], 0.75)
    for name, (value, bound) in want.items():
        _inside(getattr(b, name).reshape(value.shape), value, bound, name)
    c = fp8.residual_norm_backward(*args, **more)
    for name in want:
        if name != "dh":
            assert torch.equal(getattr(c, name), getattr(b, name)), name
    _same_codes(fp8, c.dh, b.dh)
    assert fp8.device_status() == 0
