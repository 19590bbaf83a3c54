"""Waits of the gated delta rule's single tokens that give up: reported, and nothing is stored, so that a state that is
updated in place is still there."""
import pytest
import torch

from test_gpu_delta import call, kda, make

pytestmark = pytest.mark.gpu


@pytest.fixture
def hooks():
    yield kda.kda_test_hooks
    kda.kda_test_hooks()


@pytest.mark.parametrize("dtype,T,K,V", [(torch.bfloat16, 1, 128, 128), (torch.bfloat16, 4, 64, 64), (torch.float32, 3, 128, 256),
                                         (torch.float32, 2, 100, 77), (torch.bfloat16, 2, 128, 126)])
@pytest.mark.parametrize("form", ["chunk", "recurrent"])
def test_a_state_that_does_not_come(hooks, form, dtype, T, K, V):
    fn = kda.kda_delta_chunk_fwd if form == "chunk" else kda.kda_delta_recurrent_fwd
    x = make(2, T, 3, K, V, dtype, seed=91)
    want = call(fn, x)
    kda.kda_fused_wait_timeouts(reset=True)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    S, o = x["S0"].to("cuda"), torch.full_like(want[0], 7.0)
    kw = dict(initial_state=S, final_state=S, o=o) | (dict(status=status) if form == "chunk" else {})
    hooks(wait_timeout_chunk=0)
    call(fn, x, **kw)
    assert kda.kda_fused_wait_timeouts(reset=True) >= 6
    assert int(status) == (1 if form == "chunk" else 0)
    assert (o == 7).all() and torch.equal(S.cpu(), x["S0"])
    hooks()
    status.zero_()
    call(fn, x, **kw)
    assert int(status) == 0 and kda.kda_fused_wait_timeouts() == 0
    assert torch.equal(o, want[0]) and torch.equal(S, want[1])
