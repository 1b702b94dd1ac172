"""Torch-facing wrapper of the orthogonalised weight update (the Newton-Schulz
products of the Muon optimiser), for the FP32 main gradients that the
weight-gradient GEMM accumulates (dp.MainGrads), or for BF16 ones.
"""
from __future__ import annotations

import torch

from . import _lib
from .linear import _check, _on_operand_device, _stream


def _span(t: torch.Tensor):
    """[first, end) byte addresses that a row-major 2-D tensor covers."""
    if t.numel() == 0:
        return 0, 0
    start = t.data_ptr()
    return start, start + ((t.shape[0] - 1) * t.stride(0) + t.shape[1]) * t.element_size()


def _matrix(t: torch.Tensor, dtypes, name: str):
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.dtype not in dtypes:
        raise ValueError("%s must be %s, got %s" % (name, " or ".join(map(str, dtypes)), t.dtype))
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1) or (t.shape[0] > 1 and t.stride(0) < t.shape[1]):
        raise ValueError("%s must be a row-major 2-D tensor" % name)


def _row_stride(t: torch.Tensor) -> int:
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1])


@_on_operand_device
def orthogonalize(g: torch.Tensor, *, steps: int = 5, coefficients=(3.4445, -4.7750, 2.0315), eps: float = 1e-7,
                  out: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """The nearly orthogonal matrix of g [n, k] (FP32 or BF16, n, k <= 65536) that `steps` Newton-Schulz steps with the
    odd quintic a x + b x^3 + c x^5 reach from g / (|g| + eps), as BF16 [n, k].

    The coefficients must keep singular values that start in [0, 1] below 2, as Muon's do.  |g| is summed in FP32: it
    has to stay below 1e18, and eps should be small beside it (a g / eps below 1e-4 loses digits).
    `workspace`: a contiguous CUDA uint8 tensor of puro_fp8_orthogonalize_workspace_bytes(n, k) bytes to use instead
    of allocating it; calls that may run at the same time need distinct ones."""
    _matrix(g, (torch.float32, torch.bfloat16), "g")
    n, k = g.shape
    if n > 65536 or k > 65536:
        raise ValueError("g must be at most [65536, 65536], got [%d, %d]" % (n, k))
    if not 1 <= steps <= 64:
        raise ValueError("steps must be 1 to 64, got %r" % (steps,))
    if not eps >= 0:
        raise ValueError("eps must not be negative")
    a, b, c = coefficients
    if out is None:
        out = torch.empty((n, k), dtype=torch.bfloat16, device=g.device)
    _matrix(out, (torch.bfloat16,), "out")
    if tuple(out.shape) != (n, k):
        raise ValueError("out must be [%d, %d], got %s" % (n, k, tuple(out.shape)))
    (g0, g1), (o0, o1) = _span(g), _span(out)
    if g0 < o1 and o0 < g1:
        raise ValueError("out must not overlap g")
    need = _lib.puro_fp8_orthogonalize_workspace_bytes(n, k)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=g.device)
    elif (not workspace.is_cuda or workspace.dtype != torch.uint8 or not workspace.is_contiguous()
          or workspace.numel() < need):
        raise ValueError("workspace must be a contiguous CUDA uint8 tensor of at least %d bytes" % need)
    st = _lib.puro_fp8_orthogonalize(g.data_ptr(), _row_stride(g), int(g.dtype == torch.float32), n, k, steps, a, b, c,
                                     eps, out.data_ptr(), _row_stride(out), workspace.data_ptr(), _stream())
    if st == _lib.PURO_ERR_SHAPE:
        raise ValueError("the coefficients %r lead singular values out of range in %d steps" % (coefficients, steps))
    _check(st, "puro_fp8_orthogonalize")
    return out
