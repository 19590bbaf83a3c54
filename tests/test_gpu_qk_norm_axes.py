"""The axes of a rotation's pairs, however the caller holds them: the list's results."""
import numpy
import pytest
import torch

from test_gpu_qk_norm import DEV, freq, kda

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("R", [2, 6, 64])
def test_axes_of_pairs(R):
    gen = torch.Generator().manual_seed(R)
    x = torch.randn(2, 5, 3, 64, generator=gen).to(DEV)
    pos = torch.randint(1000, (3, 2, 5), generator=gen, dtype=torch.int32).to(DEV)
    axes = [(i + 1) % 3 for i in range(R // 2)]
    turn = lambda a: kda.kda_qk_norm_rope_fwd(x, positions=pos, inv_freq=freq(R).to(DEV), pair_axes=a)[0]  # noqa: E731
    want = turn(axes)
    plain = kda.kda_qk_norm_rope_fwd(x, positions=pos, inv_freq=freq(R).to(DEV))[0]
    assert not torch.equal(want, plain)
    for held in (tuple(axes), bytes(axes), numpy.array(axes), numpy.array(axes, dtype=numpy.int32), torch.tensor(axes)):
        assert torch.equal(turn(held), want)
    for bad in (numpy.array(axes) + 2, torch.tensor(axes) - 2, [0.5] * (R // 2)):
        with pytest.raises((ValueError, TypeError)):
            turn(bad)
