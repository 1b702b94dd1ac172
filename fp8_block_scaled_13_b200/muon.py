"""Torch-facing wrapper of the orthogonalised weight update (the Newton-Schulz
products of the Muon optimiser), for the FP32 main gradients that the
weight-gradient GEMM accumulates (dp.MainGrads), or for BF16 ones.
"""
from __future__ import annotations

import torch

from . import _lib, block
from .linear import _check


def orthogonalize_workspace_bytes(n: int, k: int) -> int:
    """Bytes of the workspace that orthogonalize takes for an [n, k] gradient (0 for sizes that it does not take)."""
    return _lib.puro_fp8_orthogonalize_workspace_bytes(n, k)


def orthogonalize(g: torch.Tensor, *, steps: int = 5, coefficients=(3.4445, -4.7750, 2.0315), eps: float = 1e-7,
                  out: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """The nearly orthogonal matrix of g [n, k] (FP32 or BF16, n, k <= 65536) that `steps` Newton-Schulz steps with the
    odd quintic a x + b x^3 + c x^5 reach from g / (|g| + eps), as BF16 [n, k].

    The coefficients must keep singular values that start in [0, 1] below 2, as Muon's do.  |g| is summed in FP32: it
    has to stay between 1e-18 and 1e18, and eps should be small beside it (a g / eps below 1e-4 loses digits).  The same
    g gives the same result.  A large g takes a cooperative launch, which waits until it fits on the device beside what
    runs on other streams.
    `workspace`: a contiguous CUDA uint8 tensor of at least orthogonalize_workspace_bytes(n, k) bytes, on a 256-byte
    boundary (as torch allocates), to use instead of allocating it; calls that may run at the same time need distinct
    ones.  Neither it nor `out` may overlap another of the call's tensors."""
    a, b, c = coefficients
    st, new = (block._native or block._load()).orthogonalize(g, steps, a, b, c, eps, out, workspace)
    if st == _lib.PURO_ERR_SHAPE:
        raise ValueError("the coefficients %r lead singular values out of range in %d steps" % (coefficients, steps))
    _check(st, "puro_fp8_orthogonalize")
    return new if out is None else out
