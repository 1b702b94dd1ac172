"""A caller's workspace of the orthogonalisation: its size from the package, and the refusal of one that the kernels
could not use or that lies in another of the call's tensors (all before any launch)."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fp8():
    import fp8_block_scaled_13_b200 as m
    from fp8_block_scaled_13_b200 import build
    build.build()
    return m


@pytest.mark.parametrize("n,k", [(40, 60), (200, 333), (600, 700)])
def test_a_workspace_of_just_the_size(fp8, n, k):
    g = torch.randn(n, k, generator=torch.Generator(device="cuda").manual_seed(n), device="cuda")
    size = fp8.orthogonalize_workspace_bytes(n, k)
    assert size >= 256
    buf = torch.full((size + 512,), 7, dtype=torch.uint8, device="cuda")
    want = fp8.orthogonalize(g)
    assert torch.equal(fp8.orthogonalize(g, workspace=buf[256:256 + size]), want)
    assert (buf[:256] == 7).all() and (buf[256 + size:] == 7).all()
    with pytest.raises(ValueError, match="workspace"):
        fp8.orthogonalize(g, workspace=buf[256:255 + size])
    for off in (16, 128):
        with pytest.raises(ValueError, match="256"):
            fp8.orthogonalize(g, workspace=buf[off:off + size])
    assert fp8.device_status() == 0


def test_a_workspace_inside_another_tensor(fp8):
    n, k = 200, 333
    size = fp8.orthogonalize_workspace_bytes(n, k)
    g = torch.randn(n, k, device="cuda")
    memory = torch.zeros(2 << 20, dtype=torch.uint8, device="cuda")
    inside = memory[:4 * n * k].view(torch.float32).view(n, k)
    inside.copy_(g)
    out = memory[-2 * n * k:].view(torch.bfloat16).view(n, k)
    start = (4 * n * k - 8) // 256 * 256   # the last bytes of g
    with pytest.raises(ValueError, match="overlap g"):
        fp8.orthogonalize(inside, workspace=memory[start:start + size])
    start = (memory.numel() - 2 * n * k + 8 - size) // 256 * 256 + 256   # ends in out's first bytes
    with pytest.raises(ValueError, match="overlap out"):
        fp8.orthogonalize(g, out=out, workspace=memory[start:start + size])
    # beside both
    start = (4 * n * k + 255) // 256 * 256
    assert torch.equal(fp8.orthogonalize(inside, out=out, workspace=memory[start:start + size]), fp8.orthogonalize(g))
    assert fp8.device_status() == 0
