"""Newton-Schulz orthogonalisation without a GPU: the iteration's definition, the refusals of the C ABI and of the
wrapper, and the sizes of workspaces."""
import pytest
import torch

import fp8_block_scaled_13_b200 as fp8

A = 1 << 20  # an aligned fake device address; never dereferenced


@pytest.fixture(scope="module")
def lib():
    from fp8_block_scaled_13_b200 import _lib, build
    build.build()
    return _lib


def _call(lib, **over):
    a = dict(g=A, ld_g=64, g_f32=1, n=32, k=64, steps=5, a=3.4445, b=-4.7750, c=2.0315, eps=1e-7, out=A, ld_out=64,
             workspace=A)
    assert set(over) <= set(a)
    a.update(over)
    return lib.puro_fp8_orthogonalize(*a.values(), None)


@pytest.mark.parametrize("over,code", [
    (dict(g_f32=2), -4), (dict(n=-1), -3), (dict(k=-1), -3), (dict(n=65537), -3), (dict(k=65537), -3),
    (dict(steps=0), -3), (dict(steps=65), -3), (dict(eps=-1.0), -3), (dict(eps=float("nan")), -3),
    (dict(ld_g=63), -3), (dict(ld_out=63), -3),
    (dict(g=None), -1), (dict(out=None), -1), (dict(workspace=None), -1),
    (dict(g=A + 2), -2), (dict(g_f32=0, g=A + 1), -2), (dict(out=A + 1), -2), (dict(workspace=A + 128), -2),
    # coefficients that leave the range the FP16 form holds: they grow, or are no numbers
    (dict(a=4.0, b=0.0, c=0.0), -3), (dict(a=-4.0, b=0.0, c=0.0), -3), (dict(a=1.0, b=0.0, c=30.0), -3),
    (dict(a=float("nan")), -3), (dict(c=float("inf")), -3),
])
def test_argument_errors(lib, over, code):
    assert _call(lib, **over) == code


def test_empty_gradients_are_no_ops(lib):
    assert _call(lib, n=0, g=None, out=None, workspace=None) == 0
    assert _call(lib, k=0, g=None, out=None, workspace=None) == 0


def test_workspace_sizes(lib):
    size = lib.puro_fp8_orthogonalize_workspace_bytes
    assert size(0, 5) == size(5, 0) == size(-1, 5) == size(65537, 5) == 0
    for n, k in ((1, 1), (200, 333), (333, 200), (2048, 2048), (12288, 2048), (65536, 65536)):
        m = min(n, k)
        matrices = 8 * n * ((k + 7) // 8 * 8) + 4 * m * ((m + 7) // 8 * 8)
        # four matrices of X, two of its Gram matrix, small vectors, and the partials of at most 74 split units
        assert matrices < size(n, k) <= matrices + 8 * m + 16384 + 74 * 262144 + 10 * 256
        assert size(n, k) % 256 == 0


def test_wrapper_refusals():
    g = torch.zeros(8, 8)
    with pytest.raises(ValueError, match="CUDA"):
        fp8.orthogonalize(g)
    with pytest.raises(ValueError, match="different devices"):
        fp8.orthogonalize(g, out=torch.zeros(8, 8, dtype=torch.bfloat16, device="meta"))


def test_definition_reaches_an_orthogonal_matrix():
    """The quintic with its usual coefficients brings singular values into 0.7 .. 1.2, on either side of the matrix."""
    torch.manual_seed(0)
    for shape in ((20, 33), (33, 20), (24, 24)):
        x = torch.randn(*shape, dtype=torch.float64)
        x = x / x.norm()
        for _ in range(8):
            m = x @ x.T
            x = 3.4445 * x + (-4.7750 * m + 2.0315 * m @ m) @ x
        s = torch.linalg.svdvals(x)
        assert s.max() < 1.21 and s.min() > 0.66
