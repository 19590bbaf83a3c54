"""Single tokens and short sequences of the gated delta rule with states above what a block's shared memory holds whole and
rows that are not whole vectors: rows and columns behind the last masked, against float64, in place and packed."""
import pytest
import torch

from test_gpu_delta import call, check, kda, make, reference

pytestmark = pytest.mark.gpu

SIZES = [(236, 253), (213, 255), (251, 254), (255, 213), (256, 253), (218, 249)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("K,V", SIZES)
@pytest.mark.parametrize("raw", [False, True])
def test_large_odd_states(dtype, K, V, raw):
    assert K * V > 54000 and V % 4 != 0
    for B, T, H, Hk in ((3, 1, 4, 2), (2, 5, 3, 3)):
        x = make(B, T, H, K, V, dtype, Hk=Hk, raw=raw, seed=K + V + T)
        got = call(kda.kda_delta_recurrent_fwd, x, raw=raw)
        check(got, reference(x, raw=raw), dtype, K)
        S = x["S0"].to("cuda")
        o, S1 = call(kda.kda_delta_recurrent_fwd, x, raw=raw, initial_state=S, final_state=S)
        assert S1 is S and torch.equal(S, got[1]) and torch.equal(o, got[0])


@pytest.mark.parametrize("K,V", SIZES[:2])
def test_large_odd_states_of_packed_tokens(K, V):
    edges = [0, 0, 2, 3, 3, 6]
    x = make(1, 9, 2, K, V, torch.bfloat16, edges=edges, seed=3)
    want = reference(x, edges=edges)
    for name in "qkv":
        x[name][:, 6:] = float("nan")
    n = x["S0"].numel()
    guard = torch.full((n + 128,), 5.0, device="cuda")  # floats in front of and behind the call's own states
    S = guard[64:64 + n].view(x["S0"].shape)
    S.copy_(x["S0"])
    o = torch.full((1, 9, 2, V), 7.0, dtype=torch.bfloat16, device="cuda")
    got = call(kda.kda_delta_recurrent_fwd, x, edges=edges, o=o, initial_state=S, final_state=S)
    check(got, want, torch.bfloat16, K, rows=6)
    assert (o[:, 6:] == 7).all() and (guard[:64] == 5).all() and (guard[64 + n:] == 5).all()
    for n in (0, 3):
        assert torch.equal(got[1][n].cpu(), x["S0"][n])
