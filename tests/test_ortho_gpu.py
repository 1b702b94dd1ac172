"""Newton-Schulz orthogonalisation on the GPU against the iteration in 64 bits.

Errors are relative to the norm of the result.  Its one rounding to BF16 is off
by at most half a step: between 2^-9 and 2^-8 of a value, evenly spread, so at
most 2^-8 / sqrt(3) = 2.26e-3 in the mean square.  Between, X is
exact to 22 bits and what enters a product is rounded to FP16 off the diagonal:
a relative error of at most 2^-11 / sqrt(3) = 2.8e-4 in the mean square.  Five
steps take three products of two operands each, so 30 independent roundings,
sqrt(30) * 2.8e-4 = 1.6e-3.  (A step changes the relative error of a direction
by the factor x p'(x) / p(x), which is 1 for small x and, where x has grown to
0.7 or more, between -1.7 and 1: later steps do not let earlier errors grow.)
The bound is the plain sum, 2.26e-3 + 1.6e-3 = 3.9e-3.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

NS = (3.4445, -4.7750, 2.0315)
BOUND = 3.9e-3


@pytest.fixture(scope="module")
def fp8():
    import fp8_block_scaled_13_b200 as m
    from fp8_block_scaled_13_b200 import build
    build.build()
    return m


def _gradient(n, k, seed, dtype, size=1e-3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = max(1, min(n, k) // 8)
    v = torch.randn(n, r, generator=g, device="cuda") @ torch.randn(r, k, generator=g, device="cuda") / r ** 0.5
    return ((v + torch.randn(n, k, generator=g, device="cuda")) * size).to(dtype)


def _reference(g, steps=5, eps=1e-7, coefficients=NS):
    a, b, c = coefficients
    x = g.double()
    x = x / (x.norm() + eps)
    for _ in range(steps):
        m = x @ x.mT if x.shape[0] <= x.shape[1] else x.mT @ x
        p = b * m + c * m @ m
        x = a * x + (p @ x if x.shape[0] <= x.shape[1] else x @ p)
    return x


def _error(got, want):
    return ((got.double() - want).norm() / want.norm()).item()


@pytest.mark.parametrize("n,k", [(1, 1), (1, 40), (40, 1), (2, 3), (16, 16), (64, 64), (65, 63), (128, 128), (128, 640),
                                 (640, 128), (129, 257), (200, 333), (333, 200), (256, 512), (300, 1000), (1000, 300),
                                 (520, 520), (768, 2048), (2048, 768), (1100, 1537)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_orthogonalize(fp8, n, k, dtype):
    g = _gradient(n, k, n * 3 + k, dtype)
    got = fp8.orthogonalize(g)
    assert fp8.device_status() == 0
    assert got.dtype == torch.bfloat16 and _error(got, _reference(g)) <= BOUND


@pytest.mark.parametrize("n,k", [(257, 300), (300, 257), (640, 512), (1280, 2300), (2300, 1280)])
def test_any_strides_and_alignment(fp8, n, k):
    """Views that start and step off 16-byte boundaries give what aligned copies give, and nothing beside them is written."""
    for dtype in (torch.float32, torch.bfloat16):
        g = _gradient(n, k, n + k, dtype)
        want = fp8.orthogonalize(g)
        for shift, pad in ((0, 8), (1, 3), (3, 5)):
            wide = torch.full((n, k + shift + pad), float("nan"), dtype=dtype, device="cuda")
            wide[:, shift:shift + k] = g
            out = torch.full((n, k + shift + pad), -7.0, dtype=torch.bfloat16, device="cuda")
            got = fp8.orthogonalize(wide[:, shift:shift + k], out=out[:, shift:shift + k])
            assert torch.equal(got, want)
            assert (out[:, :shift] == -7).all() and (out[:, shift + k:] == -7).all()


# the kernel of one cluster: every size of cluster, an empty slice, slices and sides that end inside a tile
@pytest.mark.parametrize("n,k", [(128, 129), (129, 128), (3, 257), (128, 384), (511, 77), (100, 1025), (1, 2048), (2048, 128),
                                 (17, 1999), (2047, 33), (127, 1153)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_small_sides(fp8, n, k, dtype):
    g = _gradient(n, k, n + 2 * k, dtype)
    got = fp8.orthogonalize(g)
    assert _error(got, _reference(g)) <= BOUND
    assert torch.equal(fp8.orthogonalize(g), got)
    wide = torch.full((n, k + 9), float("nan"), dtype=dtype, device="cuda")
    wide[:, 1:k + 1] = g
    out = torch.full((n, k + 11), 5.0, dtype=torch.bfloat16, device="cuda")
    assert torch.equal(fp8.orthogonalize(wide[:, 1:k + 1], out=out[:, 3:k + 3]), got)
    assert (out[:, :3] == 5).all() and (out[:, k + 3:] == 5).all()
    assert fp8.device_status() == 0


# every way a product is cut: one tile; rounds of whole tiles; the rest split; three products or one for X X^T
@pytest.mark.parametrize("n,k", [(256, 256), (512, 2048), (1536, 1536), (2048, 1024), (2560, 2048), (300, 5000), (5000, 300),
                                 (4100, 2050)])
def test_tile_schedules_and_repeatability(fp8, n, k):
    g = _gradient(n, k, 5, torch.float32)
    got = fp8.orthogonalize(g)
    assert _error(got, _reference(g)) <= BOUND
    for _ in range(3):
        assert torch.equal(fp8.orthogonalize(g), got)
    assert fp8.device_status() == 0


def test_spectra(fp8):
    """Low rank over a floor, a power law, a geometric fall over two decades, one strong direction: a floor or a
    smallest value of 1 / 100 of the strongest direction, five times less than the bound's inputs; the roundings of
    X X^T then enter five times more, 2.26e-3 + 5 * 1.6e-3."""
    t = torch.Generator(device="cuda").manual_seed(3)
    n, k = 256, 768
    q1, _ = torch.linalg.qr(torch.randn(n, n, generator=t, device="cuda", dtype=torch.float64))
    q2, _ = torch.linalg.qr(torch.randn(k, n, generator=t, device="cuda", dtype=torch.float64))
    i = torch.arange(n, device="cuda", dtype=torch.float64)
    for s in (1 / (1 + i) + 0.01, 10 ** (-2 * i / n), (i < 16) + 0.05, (i < 1) + 0.02):
        g = (q1 * s) @ q2.T
        assert _error(fp8.orthogonalize(g.float()), _reference(g.float())) <= 2.26e-3 + 5 * 1.6e-3


@pytest.mark.parametrize("steps", [1, 2, 10])
def test_steps_and_coefficients(fp8, steps):
    for coefficients in (NS, (2.0, -1.5, 0.5), (1.875, -1.25, 0.375)):
        g = _gradient(200, 520, steps, torch.float32)
        got = fp8.orthogonalize(g, steps=steps, coefficients=coefficients)
        # six roundings of 2.8e-4 a step
        bound = 2.26e-3 + (6 * steps) ** 0.5 * 2.8e-4 * 2
        assert _error(got, _reference(g, steps, 1e-7, coefficients)) <= bound


def test_size_of_the_gradient(fp8):
    """The result does not depend on the gradient's size (eps is far below it), and a zero gradient gives zero."""
    g = _gradient(320, 512, 1, torch.float32, size=1.0)
    want = _reference(g)
    for size in (1e-12, 1e-3, 1e6, 1e15):
        assert _error(fp8.orthogonalize(g * size, eps=0.0 if size < 1e-6 else 1e-7), want) <= BOUND
    assert not fp8.orthogonalize(torch.zeros(320, 512, device="cuda")).any()
    # a gradient below eps: X0 is small, and five steps lift it by at most 3.4445 each
    small = g / g.norm() * 1e-5
    assert _error(fp8.orthogonalize(small, eps=1e-3), _reference(small, eps=1e-3)) <= BOUND
    for shape in ((0, 5), (5, 0)):
        assert fp8.orthogonalize(torch.empty(shape, device="cuda")).shape == shape

def test_mixed_sizes_on_several_streams(fp8):
    # the small kernel, one cluster and the cooperative grid side by side: the same bits as one at a time
    gs = [_gradient(n, k, i, torch.float32) for i, (n, k) in
          enumerate([(200, 333), (512, 512), (1024, 700), (100, 90), (900, 900), (333, 200)])]
    want = [fp8.orthogonalize(g) for g in gs]
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for turn in range(10):
        for i, g in enumerate(gs):
            with torch.cuda.stream(streams[(i + turn) % 3]):
                got.append((i, fp8.orthogonalize(g)))
    torch.cuda.synchronize()
    assert fp8.device_status() == 0
    assert all(torch.equal(out, want[i]) for i, out in got)


@pytest.mark.parametrize("n,k", [(600, 1100), (8, 2000), (150, 200)])
def test_streams_workspaces_and_graphs(fp8, n, k):
    from fp8_block_scaled_13_b200 import _lib
    gs = [_gradient(n + 40 * i, k, i, torch.float32) for i in range(4)]
    want = [fp8.orthogonalize(g) for g in gs]
    streams = [torch.cuda.Stream() for _ in gs]
    torch.cuda.synchronize()
    got = [None] * 4
    for _ in range(3):   # calls that may run at the same time
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = fp8.orthogonalize(gs[i])
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    # two captured calls on one workspace, whatever it held before, and inputs that change between replays
    ws = torch.full((max(_lib.puro_fp8_orthogonalize_workspace_bytes(*g.shape) for g in gs),), 255, dtype=torch.uint8,
                    device="cuda")
    g, out = [x.clone() for x in gs[:2]], [torch.empty_like(w) for w in want[:2]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i in range(2):
            fp8.orthogonalize(g[i], out=out[i], workspace=ws)
    for flip in (1.0, -1.0):
        for i in range(2):
            g[i].copy_(gs[i] * flip)
        ws.fill_(77)
        graph.replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(out[i], want[i] * flip)
    assert fp8.device_status() == 0


def test_refusals(fp8):
    g = _gradient(64, 96, 1, torch.float32)
    ws = torch.empty(255, dtype=torch.uint8, device="cuda")  # the smallest workspace is 256 bytes
    bad = [dict(steps=0), dict(steps=65), dict(eps=-1.0), dict(coefficients=(4.0, 0.0, 0.0)),
           dict(coefficients=(float("nan"), 0.0, 0.0)), dict(out=torch.empty(64, 95, dtype=torch.bfloat16, device="cuda")),
           dict(out=torch.empty(64, 96, device="cuda")), dict(out=torch.empty(64, 96, dtype=torch.bfloat16)),
           dict(out=torch.empty(96, 64, dtype=torch.bfloat16, device="cuda").T), dict(workspace=ws),
           dict(workspace=ws.cpu()), dict(workspace=ws.float())]
    for kw in bad:
        with pytest.raises(ValueError):
            fp8.orthogonalize(g, **kw)
    half = g.to(torch.bfloat16)
    for wrong in (g.half(), g.double(), g.T, g[0], g.reshape(2, 32, 96)):
        with pytest.raises(ValueError):
            fp8.orthogonalize(wrong)
    with pytest.raises(ValueError, match="overlap"):
        fp8.orthogonalize(half, out=half)
    wide = torch.empty(2, 65537, device="cuda")
    with pytest.raises(ValueError, match="65536"):
        fp8.orthogonalize(wide)
    assert fp8.device_status() == 0
