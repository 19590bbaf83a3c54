"""Packed sequences of the gated delta rule straight from the projections (raw gates, logits, rows without a norm): nothing
of the rows behind a sequence reaches it, whatever they hold.  Against float64, tolerances of the other shapes."""
import pytest
import torch

from test_gpu_delta import DEV, call, check, kda, make, reference

pytestmark = pytest.mark.gpu
FORMS = {"chunk": kda.kda_delta_chunk_fwd, "recurrent": kda.kda_delta_recurrent_fwd}


@pytest.mark.parametrize("form,dtype,K,V", [
    ("chunk", torch.bfloat16, 128, 128), ("chunk", torch.bfloat16, 64, 200), ("chunk", torch.float32, 128, 128),
    ("chunk", torch.bfloat16, 100, 100), ("recurrent", torch.bfloat16, 128, 128), ("recurrent", torch.float32, 99, 77)])
@pytest.mark.parametrize("behind", [float("nan"), float("inf"), 3e38])
def test_packed_raw_rows_with_anything_behind_them(form, dtype, K, V, behind):
    edges = [0, 0, 1, 66, 66, 130, 194, 323, 323]
    x = make(1, 340, 4, K, V, dtype, Hk=2, raw=True, edges=edges, seed=83)
    want = reference(x, raw=True, edges=edges)
    for name in ("q", "k", "v", "g", "beta"):
        x[name][:, 323:] = behind
    o = torch.full((1, 340, 4, V), 7.0, dtype=dtype, device=DEV)
    got = call(FORMS[form], x, raw=True, edges=edges, o=o)
    check(got, want, dtype, K, rows=323)
    assert (o[:, 323:] == 7).all()
    for n in (0, 3, 7):
        assert torch.equal(got[1][n].cpu(), x["S0"][n])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_packed_raw_rows_beside_sequences_that_are_none(dtype):
    """A sequence's rows with nothing finite in them reach no other sequence, though their tiles overlap."""
    edges = [0, 70, 75, 200, 203]
    x = make(1, 203, 2, 128, 128, dtype, raw=True, edges=edges, seed=85)
    clean = call(kda.kda_delta_chunk_fwd, x, raw=True, edges=edges)
    for name in ("q", "k", "v", "g", "beta"):
        x[name][:, 70:75] = float("nan")
        x[name][:, 200:] = float("inf")
    o, S = call(kda.kda_delta_chunk_fwd, x, raw=True, edges=edges)
    for n, (lo, hi) in ((0, (0, 70)), (2, (75, 200))):
        assert torch.equal(o[:, lo:hi], clean[0][:, lo:hi]) and torch.equal(S[n], clean[1][n])
    assert not torch.isfinite(o[:, 70:75]).any() and not torch.isfinite(S[1]).any()
