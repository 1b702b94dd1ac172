"""Torch-facing wrappers of what stands between the FP8 linear layers of a
transformer block: the norms with gate and residual sum, and the gated
activation, forward and backward.  Each one leaves its result as the QuantAct
that linear_forward / linear_backward take, in the bytes quant_act would make
of the BF16 tensor, or as that BF16 tensor (layout="bf16").

As in linear.py: outputs are allocated with torch unless given, the call runs
on its operands' device and that device's current stream, arguments are refused
with ValueError before any launch, and a non-zero status is raised.  The checks
and allocations are compiled (csrc/binding.cpp): these calls are short on the
GPU.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import _lib
from .linear import QuantAct, _LAYOUTS, _check

_OUT_LAYOUTS = {**_LAYOUTS, "bf16": _lib.PURO_BF16}
_native = None


def _load():
    global _native
    try:
        from . import _binding
    except ImportError as e:
        raise RuntimeError("the compiled wrappers are missing (%s); build them with "
                           "`python -c 'import __graft_entry__ as g; g.build()'`" % e) from e
    _native = _binding
    return _binding


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


def _layout_flag(layout):
    flag = _OUT_LAYOUTS.get(layout) if isinstance(layout, str) else None
    if flag is None:
        raise ValueError("layout must be one of %s, got %r" % (", ".join(_OUT_LAYOUTS), layout))
    return flag


def _result(flag, rows, cols, new):
    """New q, s, qt, st, BF16 tensors as the result they are."""
    if flag == _lib.PURO_BF16:
        return new[4]
    return QuantAct(rows, cols, q=new[0], s=new[1], qt=new[2], st=new[3])


def residual_norm(x: torch.Tensor, w_pre: torch.Tensor, h: torch.Tensor | None = None, *,
                  w_post: torch.Tensor | None = None, gate: torch.Tensor | None = None, scale: float = 1.0,
                  eps: float = 1e-6, layout: str = "both", y: torch.Tensor | None = None,
                  out: QuantAct | torch.Tensor | None = None) -> ResidualNorm:
    """y = x + scale * gate * post(h), then n = y / rms(y) * w_pre, the input of the next linear.

    x, h [rows, cols] BF16; post is the RMS norm with weight w_post, or nothing.  Without h, y is x and only the
    norm is taken.  gate is [rows, 1], [1, cols] or [rows, cols] (with one row, [1, cols] is a gate per channel).  The
    stored (BF16) y is what the norm sees; it equals x.float() + scale * ((hh * w_post) * gate) in separate FP32
    operations, rounded.  `y` may be x or h itself (the sum is then taken in place); results must not overlap inputs
    or one another otherwise."""
    flag = _layout_flag(layout)
    r = (_native or _load()).residual_norm(x, w_pre, h, w_post, gate, scale, eps, flag, y, out)
    if r[0]:
        _check(r[0], "puro_fp8_residual_norm")
    n = out if out is not None else _result(flag, x.shape[0], x.shape[1], r[4:])
    return ResidualNorm(x if h is None else y if y is not None else r[1], n, r[2], r[3])


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
    buffers.  `dx` may be dn, y or dy itself; results must not overlap inputs or one another otherwise."""
    flag = _layout_flag(layout)
    r = (_native or _load()).residual_norm_backward(dn, y, rstd, w_pre, h, dy, w_post, rstd_post, gate, scale, flag, dx,
                                                    out, dw_pre, dw_post, dgate, accumulate)
    if r[0]:
        _check(r[0], "puro_fp8_residual_norm_backward")
    dh = None
    if h is not None:
        dh = out if out is not None else _result(flag, dn.shape[0], dn.shape[1], r[5:])
    return ResidualNormGrad(r[1] if dx is None else dx, r[2] if dw_pre is None else dw_pre, dh,
                            r[3] if dw_post is None else dw_post, r[4] if dgate is None else dgate)


def swiglu(gu: torch.Tensor, layout: str = "both", out: QuantAct | torch.Tensor | None = None):
    """silu(g) * u of gu = [g | u] [rows, 2f] BF16, the fused gate+up projection's output, as the QuantAct (or, with
    layout="bf16", the BF16 tensor) that the down projection takes.  `out` must not overlap gu."""
    flag = _layout_flag(layout)
    r = (_native or _load()).swiglu(gu, flag, out)
    if r[0]:
        _check(r[0], "puro_fp8_swiglu")
    return out if out is not None else _result(flag, gu.shape[0], gu.shape[1] // 2, r[1:])


def swiglu_backward(da: torch.Tensor, gu: torch.Tensor, layout: str = "both",
                    out: QuantAct | torch.Tensor | None = None):
    """[dg | du] of swiglu from da [rows, f] BF16, as the dY of the gate+up projection (QuantAct, or BF16 with
    layout="bf16").  `out` must not overlap da or gu."""
    flag = _layout_flag(layout)
    r = (_native or _load()).swiglu_backward(da, gu, flag, out)
    if r[0]:
        _check(r[0], "puro_fp8_swiglu_backward")
    return out if out is not None else _result(flag, gu.shape[0], gu.shape[1], r[1:])
