"""The gated delta rule with the rows' norms asked for, and rows whose sum of squares overflows float32: they are none."""
import pytest
import torch

from test_gpu_delta import call, kda, make

pytestmark = pytest.mark.gpu
FORMS = {"chunk": kda.kda_delta_chunk_fwd, "recurrent": kda.kda_delta_recurrent_fwd}
CASES = [("chunk", torch.bfloat16, 150, 128, 128), ("chunk", torch.bfloat16, 150, 64, 40), ("chunk", torch.float32, 150, 128, 128),
         ("chunk", torch.bfloat16, 150, 256, 64), ("chunk", torch.bfloat16, 4, 128, 128), ("recurrent", torch.float32, 9, 128, 128),
         ("recurrent", torch.bfloat16, 9, 100, 77), ("recurrent", torch.bfloat16, 9, 236, 253)]


@pytest.mark.parametrize("form,dtype,T,K,V", CASES)
def test_a_key_whose_squares_overflow(form, dtype, T, K, V):
    """Its head's outputs from its token on, and its state, are no numbers."""
    x = make(1, T, 2, K, V, dtype, raw=True, seed=81)
    clean = call(FORMS[form], x, raw=True)
    for t in (T // 2, T - 1, 0, T // 65 * 64):  # in the middle, last, first, and the first of a chunk
        y = x | {"k": x["k"].clone()}
        y["k"][0, t, 1, :2] = 1.5e19  # their squares' sum is 4.5e38
        o, S = call(FORMS[form], y, raw=True)
        assert torch.equal(o[:, :, 0], clean[0][:, :, 0]) and torch.equal(S[:, 0], clean[1][:, 0])
        assert torch.equal(o[:, :t], clean[0][:, :t])
        assert o[0, t:, 1].isnan().all() and S[0, 1].isnan().all()


@pytest.mark.parametrize("form,dtype,T,K,V", CASES)
def test_a_query_whose_squares_overflow(form, dtype, T, K, V):
    """Its own row of its head is no numbers."""
    x = make(1, T, 2, K, V, dtype, raw=True, seed=82)
    clean = call(FORMS[form], x, raw=True)
    for t in (T // 2, T - 1, 0, T // 65 * 64):
        y = x | {"q": x["q"].clone()}
        y["q"][0, t, 1, :2] = 1.5e19
        o, S = call(FORMS[form], y, raw=True)
        assert torch.equal(S, clean[1]) and o[0, t, 1].isnan().all()
        o[0, t, 1] = clean[0][0, t, 1]
        assert torch.equal(o, clean[0])


@pytest.mark.parametrize("V", [128, 72])
@pytest.mark.parametrize("beta,v,back", [(1.0, 3.3895e38, 9e35), (2.0, 1.694e38, 5.2e35), (4.0, 3e38, 0.0)])
def test_corrections_at_the_end_of_the_range(V, beta, v, back):
    """v - S^T k, beta times it, or neither, beyond the largest bf16 number or float32's: nothing of it reaches back, nor
    another channel."""
    t = 70
    x = make(1, 150, 2, 128, V, torch.bfloat16, seed=83)
    x["g"][:] = 0
    x["beta"] = x["beta"].float()
    x["beta"][0, :t, 1] = 0  # the state is the incoming one up to the token
    x["beta"][0, t, 1] = beta
    k = x["k"][0, t, 1].double()
    x["S0"][0, 1, :, 3] = (-back * k / (k * k).sum()).float()
    x["v"][0, t, 1, 3] = 0
    clean = call(kda.kda_delta_chunk_fwd, x)
    assert torch.isfinite(clean[0]).all()
    x["v"][0, t, 1, 3] = v
    r = float(x["v"][0, t, 1, 3]) + back
    assert r < 3.4028e38 and (back == 0 or 3.3953e38 < r * beta < 3.4028e38)
    o, S = call(kda.kda_delta_chunk_fwd, x)
    keep = torch.ones_like(o, dtype=torch.bool)
    keep[0, t:, 1, 3] = False
    assert torch.equal(o[keep], clean[0][keep])
    keep = torch.ones_like(S, dtype=torch.bool)
    keep[0, 1, :, 3] = False
    assert torch.equal(S[keep], clean[1][keep])
    if back == 0:
        assert not torch.isfinite(o[0, t:, 1, 3]).any() and not torch.isfinite(S[0, 1, :, 3]).any()
