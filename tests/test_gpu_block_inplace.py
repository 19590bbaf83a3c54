"""Norms whose outputs are their inputs: the same bits as with buffers of their own."""
import pytest
import torch

from test_gpu_block import BF, kda  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("V", [7, 64, 128, 200, 257, 1000, 4096])
@pytest.mark.parametrize("which", ["x", "gate"])
def test_gated_norm(kda, dtype, V, which):  # noqa: F811
    g = torch.Generator(device="cuda").manual_seed(V)
    x, z = (torch.randn(37, 5, V, generator=g, device="cuda").to(dtype) for _ in range(2))
    w = torch.rand(V, generator=g, device="cuda")
    want = kda.kda_gated_norm_fwd(x, z, w)
    assert torch.equal(kda.kda_gated_norm_fwd(x, z, w, out=x if which == "x" else z), want)


@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("rows,D", [(5, 24), (5, 1001), (9, 4096), (1500, 8192), (5, 12288), (3, 20000)])
@pytest.mark.parametrize("gate", [False, True])
def test_block_norm(kda, dtype, rows, D, gate):  # noqa: F811
    """h on the stream."""
    g = torch.Generator(device="cuda").manual_seed(D)
    x, r, z = (torch.randn(rows, D, generator=g, device="cuda").to(dtype) for _ in range(3))
    wp, wn = (torch.rand(D, generator=g, device="cuda") for _ in range(2))
    args = dict(post_weight=wp, gate=z if gate else None, pre_weight=wn, scale=0.7)
    h, y = kda.kda_block_norm_fwd(x, r, **args)
    h2, y2 = kda.kda_block_norm_fwd(x, r, residual_out=r, **args)
    assert h2 is r and torch.equal(h2, h) and torch.equal(y2, y)
