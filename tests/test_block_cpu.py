"""Norms around a block and gated activation without a GPU: the backward
formulas against central differences and autograd, and the refusals of the C
ABI and of the wrappers (every one before any launch)."""
import ctypes
import os
import re

import pytest
import torch

import block_reference as ref
import fp8_block_scaled_13_b200 as fp8

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 20  # a 16-byte-aligned fake device address; never dereferenced


@pytest.fixture(scope="module")
def lib():
    from fp8_block_scaled_13_b200 import _lib, build
    build.build()
    return _lib


def test_binding_matches_the_header(lib):
    """Every declared argument has the ctypes type of its C type, in order."""
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "puro_fp8.h")).read(), flags=re.S)
    kinds = (("*", ctypes.c_void_p), ("int64_t", ctypes.c_int64), ("int32_t", ctypes.c_int32),
             ("float", ctypes.c_float), ("int", ctypes.c_int))
    for name in lib.EXPORTS:
        args = [a for a in re.search(r"\b%s\s*\((.*?)\);" % name, src, re.S).group(1).split(",")]
        want = [next(t for k, t in kinds if k in a) for a in args]
        assert list(getattr(lib.load(), name).argtypes) == want, name


def _double(shape, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


def _forward(v, scale=0.7, eps=1e-3):
    y, _, _ = ref.norm_forward(v["x"], v.get("h"), v.get("w_post"), v.get("gate"), scale, eps)
    return y, ref.norm_of(y, v["w_pre"], eps)[0]


@pytest.mark.parametrize("res,post,gate", [(False, False, None), (True, False, None), (True, True, None),
                                           (True, True, (5, 1)), (True, False, (1, 6)), (True, True, (5, 6))])
def test_norm_backward_formula_against_differences(res, post, gate):
    t, d, scale, eps = 5, 6, 0.7, 1e-3
    v = {"x": _double((t, d), 1), "w_pre": _double((d,), 2)}
    if res:
        v["h"] = _double((t, d), 3)
    if post:
        v["w_post"] = _double((d,), 4)
    if gate:
        v["gate"] = _double(gate, 5)
    dn, dy = _double((t, d), 6), _double((t, d), 7)
    y, n = _forward(v)
    rstd = (y.square().mean(1) + eps) ** -0.5
    rp = (v["h"].square().mean(1) + eps) ** -0.5 if post else None
    got = ref.norm_backward(dn, y, rstd, v["w_pre"], v.get("h"), dy, v.get("w_post"), rp, v.get("gate"), scale)
    names = {"x": "dx", "w_pre": "dw_pre", "h": "dh", "w_post": "dw_post", "gate": "dgate"}
    step = 1e-5
    for k, tensor in v.items():
        for i in range(tensor.numel()):
            side = []
            for sign in (1, -1):
                moved = dict(v, **{k: tensor.clone()})
                moved[k].view(-1)[i] += sign * step
                yy, nn = _forward(moved)
                side.append(((yy * dy).sum() + (nn * dn).sum()).item())
            # central differences: the error is the third derivative times step^2 / 6, plus 1e-16 * |loss| / step
            assert abs((side[0] - side[1]) / (2 * step) - got[names[k]][0].reshape(-1)[i].item()) < 1e-6, (k, i)


def test_swiglu_backward_formula_against_autograd_and_differences():
    gu, da = _double((4, 6), 1), _double((4, 3), 2)
    assert torch.autograd.gradcheck(lambda z: torch.nn.functional.silu(z[:, :3]) * z[:, 3:], gu.clone().requires_grad_())
    z = gu.clone().requires_grad_()
    (torch.nn.functional.silu(z[:, :3]) * z[:, 3:]).backward(da)
    assert torch.allclose(ref.swiglu_backward(da, gu)[0], z.grad, rtol=1e-12, atol=1e-14)


# ------------------------------------------------------------------ refusals of the C ABI

def _norm(**over):
    a = dict(x=A, ld_x=256, h=A, ld_h=256, w_pre=A, w_post=A, w_f32=0, gate=A, ld_gate=256, kind=3, gate_f32=0,
             scale=1.0, eps=1e-6, rows=64, cols=256, y=A, ld_y=256, rstd=A, rstd_post=A, layout=3, q=A, ld_q=256, s=A,
             qt=A, ld_qt=64, st=A, n=None, ld_n=0, workspace=A)
    assert set(over) <= set(a)
    a.update(over)
    return tuple(a.values())


@pytest.mark.parametrize("over,code", [
    (dict(layout=0), -4), (dict(layout=5), -4), (dict(layout=7), -4),
    (dict(kind=4), -4), (dict(kind=-1), -4), (dict(w_f32=2), -4), (dict(gate_f32=1), -4),  # FP32 per element
    (dict(cols=200), -3), (dict(cols=8320, ld_x=8320), -3), (dict(rows=-1), -3), (dict(rows=1 << 31), -3),
    (dict(eps=0.0), -3), (dict(eps=-1.0), -3), (dict(eps=float("nan")), -3),
    (dict(x=None), -1), (dict(w_pre=None), -1), (dict(y=None), -1), (dict(rstd=None), -1), (dict(rstd_post=None), -1),
    (dict(gate=None), -1), (dict(q=None), -1), (dict(s=None), -1), (dict(qt=None), -1), (dict(st=None), -1),
    (dict(layout=4), -1),                                        # BF16 result without its buffer
    (dict(ld_x=128), -3), (dict(ld_h=128), -3), (dict(ld_y=128), -3), (dict(ld_gate=128), -3),
    (dict(ld_qt=48), -3), (dict(layout=4, n=A, ld_n=128), -3),
    (dict(x=A + 2), -2), (dict(h=A + 8), -2), (dict(ld_x=260), -2), (dict(w_pre=A + 1), -2), (dict(rstd=A + 2), -2),
    (dict(kind=1, gate=A + 1), -2), (dict(w_f32=1, w_post=A + 2), -2), (dict(s=A + 8), -2), (dict(st=A + 4), -2),
])
def test_norm_argument_errors(lib, over, code):
    assert lib.puro_fp8_residual_norm(*_norm(**over), None) == code


@pytest.mark.parametrize("over,code", [
    (dict(workspace=None), -1), (dict(layout=2, workspace=None), -1), (dict(workspace=A + 8), -2)])
def test_norm_wants_its_workspace(lib, over, code):
    big = dict(rows=1 << 18, ld_qt=1 << 18)
    assert lib.puro_fp8_residual_norm(*_norm(**big, **over), None) == code


def _norm_bwd(**over):
    a = dict(dn=A, ld_dn=256, dy=A, ld_dy=256, y=A, ld_y=256, rstd=A, h=A, ld_h=256, rstd_post=A, w_pre=A, w_post=A,
             w_f32=0, gate=A, ld_gate=256, kind=3, gate_f32=0, scale=1.0, rows=64, cols=256, dx=A, ld_dx=256, dw_pre=A,
             dw_post=A, dgate=A, ld_dgate=256, accumulate=0, layout=3, q=A, ld_q=256, s=A, qt=A, ld_qt=64, st=A,
             dh=None, ld_dh=0, ws=A)
    assert set(over) <= set(a)
    a.update(over)
    return tuple(a.values())


@pytest.mark.parametrize("over,code", [
    (dict(layout=0), -4), (dict(accumulate=2), -4), (dict(kind=5), -4), (dict(gate_f32=1), -4),
    (dict(cols=100), -3), (dict(cols=8320), -3), (dict(rows=-5), -3), (dict(ld_dn=128), -3), (dict(ld_dy=128), -3),
    (dict(ld_dx=128), -3), (dict(ld_dgate=128), -3),
    (dict(dn=None), -1), (dict(y=None), -1), (dict(rstd=None), -1), (dict(rstd_post=None), -1), (dict(dx=None), -1),
    (dict(dw_pre=None), -1), (dict(dw_post=None), -1), (dict(dgate=None), -1), (dict(kind=1, dgate=None), -1),
    (dict(kind=2, dgate=None), -1), (dict(ws=None), -1), (dict(q=None), -1),
    (dict(ws=A + 8), -2), (dict(dn=A + 8), -2), (dict(dw_pre=A + 2), -2), (dict(kind=1, dgate=A + 2), -2),
])
def test_norm_backward_argument_errors(lib, over, code):
    assert lib.puro_fp8_residual_norm_backward(*_norm_bwd(**over), None) == code


@pytest.mark.parametrize("over,code", [
    (dict(layout=0), -4), (dict(layout=6), -4), (dict(f=100), -3), (dict(rows=-1), -3), (dict(f=1 << 30), -3),
    (dict(gu=None), -1), (dict(ld_gu=256), -3), (dict(gu=A + 8), -2), (dict(ld_gu=514), -2), (dict(q=None), -1),
    (dict(st=None), -1), (dict(layout=4), -1), (dict(ld_qt=48), -3),
])
def test_swiglu_argument_errors(lib, over, code):
    a = dict(gu=A, ld_gu=512, rows=64, f=256, layout=3, q=A, ld_q=512, s=A, qt=A, ld_qt=64, st=A, a=None, ld_a=0)
    a.update(over)
    assert lib.puro_fp8_swiglu(*a.values(), None) == code
    assert lib.puro_fp8_swiglu_backward(A, 256, *a.values(), None) == code


def test_swiglu_backward_checks_its_gradient(lib):
    rest = (A, 512, 64, 256, 3, A, 512, A, A, 64, A, None, 0, None)
    assert lib.puro_fp8_swiglu_backward(None, 256, *rest) == -1
    assert lib.puro_fp8_swiglu_backward(A, 128, *rest) == -3
    assert lib.puro_fp8_swiglu_backward(A + 4, 256, *rest) == -2


def test_empty_inputs_are_no_ops(lib):
    none = [None] * 4
    assert lib.puro_fp8_residual_norm(*_norm(rows=0, x=None, y=None), None) == 0
    assert lib.puro_fp8_residual_norm(*_norm(cols=0, x=None, w_pre=None), None) == 0
    assert lib.puro_fp8_residual_norm_backward(*_norm_bwd(cols=0, dn=None, dw_pre=None), None) == 0
    assert lib.puro_fp8_swiglu(None, 0, 0, 256, 3, None, 0, *none[:2], 0, *none[:2], 0, None) == 0
    assert lib.puro_fp8_swiglu(None, 0, 5, 0, 3, None, 0, *none[:2], 0, *none[:2], 0, None) == 0


def test_workspace_sizes(lib):
    size = lib.puro_fp8_residual_norm_workspace_bytes
    for layout in (0, 1, 2, 3, 4):
        assert size(0, 256, layout, 0) == size(0, 256, layout, 1) == size(5, 0, layout, 1) == 0
    # forward: a tile counter where transposed codes take more than 2368 tiles
    assert [size(32768, 2048, layout, 0) for layout in (1, 2, 3, 4)] == [0, 256, 256, 0]
    assert size(148 * 128, 2048, 3, 0) == 0 and size(148 * 128 + 1, 2048, 3, 0) == 256
    for rows in (1, 4, 5, 129, 1000, 9471, 9472, 32768, 1 << 24):
        for cols in (128, 2048, 4096, 8192):
            sums = size(rows, cols, 1, 1)
            assert sums == size(rows, cols, 0, 1) == size(rows, cols, 4, 1)
            parts = (sums - 256) // (2 * cols * 4)
            assert -(-rows // 32) <= parts <= max(-(-rows // 32), 4 * 148) + 1 and parts * 2 * cols * 4 + 256 == sums
            assert size(rows, cols, 2, 1) == size(rows, cols, 3, 1) == sums + rows * cols * 2


# ------------------------------------------------------------------ refusals of the wrappers

def _x(rows=4, cols=128, dtype=torch.bfloat16):
    return torch.zeros(rows, cols, dtype=dtype)


def test_wrappers_refuse_host_tensors_and_mixed_devices():
    w = torch.ones(128)
    for call in (lambda: fp8.residual_norm(_x(), w), lambda: fp8.swiglu(_x()), lambda: fp8.swiglu_backward(_x(), _x()),
                 lambda: fp8.residual_norm_backward(_x(), _x(), torch.ones(4), w)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="different devices"):
        fp8.residual_norm(_x(), torch.ones(128, device="meta"))


def test_linear_layers_check_a_quantized_input():
    with pytest.raises(ValueError, match="inner dimensions"):
        fp8.linear_forward(fp8.QuantAct(128, 256), wq=fp8.QuantWeight(128, 128, _x(128, 128, torch.uint8),
                                                                      _x(1, 1, torch.uint8)))
