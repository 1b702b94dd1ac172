"""Torch-facing wrappers of what stands between the FP8 linear layers of a
transformer block: the norms with gate and residual sum, and the gated
activation, forward and backward.  Each one leaves its result as the QuantAct
that linear_forward / linear_backward take, in the bytes quant_act would make
of the BF16 tensor, or as that BF16 tensor (layout="bf16").

As in linear.py: outputs are allocated with torch unless given, pointers and
the current stream go to libpuro_fp8.so, and a non-zero status is raised.
"""
from __future__ import annotations

import functools
from dataclasses import dataclass

import torch

from . import _lib
from .linear import (QuantAct, _LAYOUTS, _blocked, _check, _check_bytes, _check_tensor, _need, _on_operand_device,
                     _require, _round16, _stream, blocked_scale_bytes)

_OUT_LAYOUTS = {**_LAYOUTS, "bf16": _lib.PURO_BF16}


@dataclass
class ResidualNorm:
    """Result of residual_norm."""
    y: torch.Tensor                         # [rows, cols] BF16, the residual stream (x itself without a block output)
    n: QuantAct | torch.Tensor              # the normed stream: codes, or BF16 with layout="bf16"
    rstd: torch.Tensor                      # [rows] FP32, 1 / rms of y
    rstd_post: torch.Tensor | None = None   # [rows] FP32, 1 / rms of h (with w_post)


@dataclass
class ResidualNormGrad:
    """Result of residual_norm_backward."""
    dx: torch.Tensor                        # [rows, cols] BF16
    dw_pre: torch.Tensor                    # [cols] FP32
    dh: QuantAct | torch.Tensor | None = None   # codes, or BF16 with layout="bf16" (None without h)
    dw_post: torch.Tensor | None = None     # [cols] FP32
    dgate: torch.Tensor | None = None       # the gate's shape: FP32 per token or channel, BF16 per element


def _ptr(t):
    return t.data_ptr() if t is not None else None


def _ld(t):
    return t.stride(0) if t is not None else 0


def _bf16(t, shape, name):
    """A row-major BF16 matrix of `shape`, checked: its address and row stride."""
    stride = t.stride()
    if t.dtype is not torch.bfloat16 or t.shape != shape or not t.is_cuda or stride[1] != 1:
        _check_tensor(t, shape, (torch.bfloat16,), name)  # (an empty matrix may have any strides)
    return t.data_ptr(), stride[0]


def _layout_flag(layout):
    flag = _OUT_LAYOUTS.get(layout) if isinstance(layout, str) else None
    if flag is None:
        raise ValueError("layout must be one of %s, got %r" % (", ".join(_OUT_LAYOUTS), layout))
    return flag


def _codes(t, rows, cols, name, what, padded=False):
    """A caller's buffer of codes, checked: its address and row stride."""
    if t is None:
        raise ValueError("out has no %s" % what)
    stride, shape = t.stride(), t.shape
    if (t.dtype is not torch.uint8 or len(shape) != 2 or shape[0] != rows or not t.is_cuda or stride[1] != 1
            or (shape[1] < cols if padded else shape[1] != cols)):
        _check_tensor(t, (rows, cols), (torch.uint8,), name, min_cols=padded)
    return t.data_ptr(), stride[0]


def _scales(t, rows, groups, name, what):
    if t is None:
        raise ValueError("out has no %s" % what)
    if (t.dtype is not torch.uint8 or t.numel() < blocked_scale_bytes(rows, groups) or not t.is_cuda
            or not t.is_contiguous()):
        _check_bytes(t, blocked_scale_bytes(rows, groups), name)
    return t.data_ptr()


def _result(out, rows, cols, flag, dev):
    """`out`, checked, or new memory for a [rows, cols] result in the layout, and the C call's q, ld_q, s, qt, ld_qt,
    st, bf16, ld_bf16 for it."""
    if flag == _lib.PURO_BF16:
        if out is None:
            out = torch.empty((rows, cols), dtype=torch.bfloat16, device=dev)
        elif not isinstance(out, torch.Tensor):
            raise ValueError("out must be a BF16 tensor for layout 'bf16'")
        return out, (None, 0, None, None, 0, None, *_bf16(out, (rows, cols), "out"))
    tiles = (rows + 127) // 128
    if out is None:
        out = QuantAct(rows, cols)
        if flag & _lib.PURO_ROWWISE:
            out.q = torch.empty((rows, cols), dtype=torch.uint8, device=dev)
            out.s = _blocked(rows, cols // 128, dev)
        if flag & _lib.PURO_COLWISE:
            out.qt = torch.empty((cols, _round16(rows)), dtype=torch.uint8, device=dev)
            out.st = _blocked(cols, tiles, dev)
    elif not isinstance(out, QuantAct) or (out.rows, out.cols) != (rows, cols):
        raise ValueError("out must be a QuantAct made for a [%d, %d] input" % (rows, cols))
    q = ld_q = s = qt = ld_qt = st = None
    if flag & _lib.PURO_ROWWISE:
        q, ld_q = _codes(out.q, rows, cols, "out.q", "row-wise codes")
        s = _scales(out.s, rows, cols // 128, "out.s", "row-wise scales")
    if flag & _lib.PURO_COLWISE:
        qt, ld_qt = _codes(out.qt, cols, _round16(rows), "out.qt", "transposed codes", padded=True)
        st = _scales(out.st, cols, tiles, "out.st", "transposed scales")
    return out, (q, ld_q or 0, s, qt, ld_qt or 0, st, None, 0)


_NO_RESULT = (None, 0, None, None, 0, None, None, 0)


def _weight(w, cols, name):
    if (w.dtype is torch.bfloat16 or w.dtype is torch.float32) and w.shape == (cols,) and w.is_cuda and w.is_contiguous():
        return w.data_ptr()
    if not w.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if w.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("%s must be torch.bfloat16 or torch.float32, got %s" % (name, w.dtype))
    raise ValueError("%s must be a contiguous [%d] tensor, got %s" % (name, cols, tuple(w.shape)))


def _vector(t, n, name):
    if t.dtype is not torch.float32 or t.shape != (n,) or not t.is_cuda or not t.is_contiguous():
        raise ValueError("%s must be a contiguous CUDA float32 [%d] tensor" % (name, n))
    return t.data_ptr()


def _gate(gate, rows, cols):
    """(kind, is_f32, row stride) of a gate [rows, 1], [1, cols] or [rows, cols]."""
    if gate is None:
        return _lib.PURO_GATE_NONE, 0, 0
    if not gate.is_cuda:
        raise ValueError("gate must be a CUDA tensor")
    if gate.dim() != 2 or tuple(gate.shape) not in ((rows, 1), (1, cols), (rows, cols)):
        raise ValueError("gate must be [%d, 1], [1, %d] or [%d, %d], got %s"
                         % (rows, cols, rows, cols, tuple(gate.shape)))
    if gate.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("gate must be torch.bfloat16 or torch.float32, got %s" % gate.dtype)
    f32 = int(gate.dtype == torch.float32)
    if gate.shape[1] == 1:
        if not gate.is_contiguous():
            raise ValueError("a gate per token must be contiguous")
        return _lib.PURO_GATE_TOKEN, f32, 0
    if gate.shape[0] == 1:  # also one row of elements: the same products
        if not gate.is_contiguous():
            raise ValueError("a gate per channel must be contiguous")
        return _lib.PURO_GATE_CHANNEL, f32, 0
    if f32:
        raise ValueError("a gate per element must be torch.bfloat16")
    _require(gate, torch.bfloat16, "gate")
    return _lib.PURO_GATE_FULL, 0, gate.stride(0)


def _same_type(w_pre, w_post):
    if w_post is not None and w_post.dtype != w_pre.dtype:
        raise ValueError("w_pre and w_post must have one type, got %s and %s" % (w_pre.dtype, w_post.dtype))
    return int(w_pre.dtype == torch.float32)


@functools.lru_cache(maxsize=1024)
def _norm_workspace(rows, cols, flag, backward):
    return _lib.puro_fp8_residual_norm_workspace_bytes(rows, cols, flag, backward)


def _branch(h, w_post, gate):
    if h is None and (w_post is not None or gate is not None):
        raise ValueError("w_post and gate act on the block output h, which is missing")


@_on_operand_device
def residual_norm(x: torch.Tensor, w_pre: torch.Tensor, h: torch.Tensor | None = None, *,
                  w_post: torch.Tensor | None = None, gate: torch.Tensor | None = None, scale: float = 1.0,
                  eps: float = 1e-6, layout: str = "both", y: torch.Tensor | None = None,
                  out: QuantAct | torch.Tensor | None = None) -> ResidualNorm:
    """y = x + scale * gate * post(h), then n = y / rms(y) * w_pre, the input of the next linear.

    x, h [rows, cols] BF16; post is the RMS norm with weight w_post, or nothing.  Without h, y is x and only the
    norm is taken.  gate is [rows, 1], [1, cols] or [rows, cols].  The stored (BF16) y is what the norm sees.
    `y` may be x itself (the sum is then taken in place)."""
    _require(x, torch.bfloat16, "x")
    shape = x.shape
    rows, cols = shape
    flag = _layout_flag(layout)
    _branch(h, w_post, gate)
    if not eps > 0:
        raise ValueError("eps must be positive")
    w_pre_p = _weight(w_pre, cols, "w_pre")
    w_f32 = _same_type(w_pre, w_post)
    dev = x.device
    h_p = y_p = w_post_p = None
    ld_h = ld_y = 0
    if h is not None:
        h_p, ld_h = _bf16(h, shape, "h")
        if y is None:
            y = torch.empty(shape, dtype=torch.bfloat16, device=dev)
        y_p, ld_y = _bf16(y, shape, "y")
        if w_post is not None:
            w_post_p = _weight(w_post, cols, "w_post")
    elif y is not None:
        raise ValueError("y is only written with a block output h")
    kind, g_f32, ld_gate = _gate(gate, rows, cols)
    res, res_args = _result(out, rows, cols, flag, dev)
    rstd = torch.empty(rows, dtype=torch.float32, device=dev)
    rstd_post = torch.empty(rows, dtype=torch.float32, device=dev) if w_post is not None else None
    need = _norm_workspace(rows, cols, flag, 0)
    ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    st = _lib.puro_fp8_residual_norm(
        x.data_ptr(), x.stride(0), h_p, ld_h, w_pre_p, w_post_p, w_f32, _ptr(gate), ld_gate, kind, g_f32, scale, eps,
        rows, cols, y_p, ld_y, rstd.data_ptr(), _ptr(rstd_post), flag, *res_args, _ptr(ws), _stream())
    if st:
        _check(st, "puro_fp8_residual_norm")
    return ResidualNorm(x if h is None else y, res, rstd, rstd_post)


@_on_operand_device
def residual_norm_backward(dn: torch.Tensor, y: torch.Tensor, rstd: torch.Tensor, w_pre: torch.Tensor,
                           h: torch.Tensor | None = None, *, dy: torch.Tensor | None = None,
                           w_post: torch.Tensor | None = None, rstd_post: torch.Tensor | None = None,
                           gate: torch.Tensor | None = None, scale: float = 1.0, layout: str = "both",
                           dx: torch.Tensor | None = None, out: QuantAct | torch.Tensor | None = None,
                           dw_pre: torch.Tensor | None = None, dw_post: torch.Tensor | None = None,
                           dgate: torch.Tensor | None = None, accumulate: bool = False) -> ResidualNormGrad:
    """Gradients of residual_norm from dn (of n) and dy (of y, from further on; None: no such gradient).

    y, rstd, rstd_post: what residual_norm returned; h, the weights, gate and scale: what it was given.  dh comes
    back in `layout`, as the dY of the linear that made h.  dw_pre, dw_post and dgate may be given; with
    accumulate=True the weights' gradients, and the gradient of a gate [1, cols], are added into the given FP32
    buffers."""
    _require(dn, torch.bfloat16, "dn")
    shape = dn.shape
    rows, cols = shape
    flag = _layout_flag(layout)
    _branch(h, w_post, gate)
    y_p, ld_y = _bf16(y, shape, "y")
    rstd_p = _vector(rstd, rows, "rstd")
    w_pre_p = _weight(w_pre, cols, "w_pre")
    w_f32 = _same_type(w_pre, w_post)
    dev = dn.device
    dy_p = h_p = w_post_p = rstd_post_p = dw_post_p = None
    ld_dy = ld_h = 0
    if dy is not None:
        dy_p, ld_dy = _bf16(dy, shape, "dy")
    if h is not None:
        h_p, ld_h = _bf16(h, shape, "h")
    if w_post is not None:
        w_post_p = _weight(w_post, cols, "w_post")
        rstd_post_p = _vector(_need(rstd_post, "w_post needs the rstd_post of the forward pass"), rows, "rstd_post")
    kind, g_f32, ld_gate = _gate(gate, rows, cols)
    if dx is None:
        dx = torch.empty(shape, dtype=torch.bfloat16, device=dev)
    dx_p, ld_dx = _bf16(dx, shape, "dx")
    if h is None and out is not None:
        raise ValueError("out holds the gradient of h, which is missing")
    if (w_post is None and dw_post is not None) or (gate is None and dgate is not None):
        raise ValueError("dw_post and dgate need w_post and gate")
    if accumulate and (dw_pre is None or (w_post is not None and dw_post is None)
                       or (kind == _lib.PURO_GATE_CHANNEL and dgate is None)):
        raise ValueError("accumulate=True needs the FP32 buffers to add into")
    if dw_pre is None:
        dw_pre = torch.empty(cols, dtype=torch.float32, device=dev)
    dw_pre_p = _vector(dw_pre, cols, "dw_pre")
    if w_post is not None:
        if dw_post is None:
            dw_post = torch.empty(cols, dtype=torch.float32, device=dev)
        dw_post_p = _vector(dw_post, cols, "dw_post")
    if gate is not None:
        gtype = torch.bfloat16 if kind == _lib.PURO_GATE_FULL else torch.float32
        if dgate is None:
            dgate = torch.empty(gate.shape, dtype=gtype, device=dev)
        _check_tensor(dgate, gate.shape, (gtype,), "dgate")
        if kind == _lib.PURO_GATE_TOKEN and not dgate.is_contiguous():
            raise ValueError("dgate must be contiguous")
    res, res_args = _result(out, rows, cols, flag, dev) if h is not None else (None, _NO_RESULT)
    ws = torch.empty(_norm_workspace(rows, cols, flag if h is not None else 0, 1), dtype=torch.uint8, device=dev)
    st = _lib.puro_fp8_residual_norm_backward(
        dn.data_ptr(), dn.stride(0), dy_p, ld_dy, y_p, ld_y, rstd_p, h_p, ld_h, rstd_post_p, w_pre_p, w_post_p, w_f32,
        _ptr(gate), ld_gate, kind, g_f32, scale, rows, cols, dx_p, ld_dx, dw_pre_p, dw_post_p, _ptr(dgate), _ld(dgate),
        1 if accumulate else 0, flag, *res_args, ws.data_ptr(), _stream())
    if st:
        _check(st, "puro_fp8_residual_norm_backward")
    return ResidualNormGrad(dx, dw_pre, res, dw_post, dgate)


@_on_operand_device
def swiglu(gu: torch.Tensor, layout: str = "both", out: QuantAct | torch.Tensor | None = None):
    """silu(g) * u of gu = [g | u] [rows, 2f] BF16, the fused gate+up projection's output, as the QuantAct (or, with
    layout="bf16", the BF16 tensor) that the down projection takes."""
    _require(gu, torch.bfloat16, "gu")
    rows, f2 = gu.shape
    flag = _layout_flag(layout)
    if f2 % 2:
        raise ValueError("gu must hold two halves of equal width, got %d columns" % f2)
    res, res_args = _result(out, rows, f2 // 2, flag, gu.device)
    st = _lib.puro_fp8_swiglu(gu.data_ptr(), gu.stride(0), rows, f2 // 2, flag, *res_args, _stream())
    if st:
        _check(st, "puro_fp8_swiglu")
    return res


@_on_operand_device
def swiglu_backward(da: torch.Tensor, gu: torch.Tensor, layout: str = "both",
                    out: QuantAct | torch.Tensor | None = None):
    """[dg | du] of swiglu from da [rows, f] BF16, as the dY of the gate+up projection (QuantAct, or BF16 with
    layout="bf16")."""
    _require(da, torch.bfloat16, "da")
    rows, f = da.shape
    flag = _layout_flag(layout)
    gu_p, ld_gu = _bf16(gu, (rows, 2 * f), "gu")
    res, res_args = _result(out, rows, 2 * f, flag, gu.device)
    st = _lib.puro_fp8_swiglu_backward(da.data_ptr(), da.stride(0), gu_p, ld_gu, rows, f, flag, *res_args, _stream())
    if st:
        _check(st, "puro_fp8_swiglu_backward")
    return res
