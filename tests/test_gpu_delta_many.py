"""The gated delta rule in FP32 chunks with as many heads as its wider column blocks want (two and four columns a thread),
against float64."""
import pytest
import torch

from test_gpu_delta import call, check, kda, make, reference

pytestmark = pytest.mark.gpu


def units(per_sm):
    return max(1, int(per_sm * torch.cuda.get_device_properties(0).multi_processor_count)) + 3


@pytest.mark.parametrize("dtype,o_dtype,K,V,per_sm,T", [
    (torch.float32, None, 128, 128, 1, 70), (torch.float32, None, 64, 33, 1, 130), (torch.float32, None, 200, 72, 1, 65),
    (torch.float32, None, 128, 64, 0.6, 70), (torch.float32, None, 33, 50, 0.6, 64),
    (torch.bfloat16, torch.float32, 128, 128, 1, 70), (torch.bfloat16, torch.float32, 128, 64, 0.6, 129),
    (torch.bfloat16, None, 256, 256, 1, 70), (torch.bfloat16, None, 250, 100, 0.6, 66), (torch.bfloat16, None, 60, 60, 1, 100),
])
def test_many_units(dtype, o_dtype, K, V, per_sm, T):
    n = units(per_sm)
    x = make(1, T, n, K, V, dtype, seed=K + V)
    want = reference(x)
    got = call(kda.kda_delta_chunk_fwd, x, o_dtype=o_dtype)
    check(got, want, dtype, K, o_dtype)
    # the output in v's place, the state in place
    if o_dtype is None or o_dtype == dtype:
        v, S = x["v"].to("cuda"), x["S0"].to("cuda")
        o, S1 = call(kda.kda_delta_chunk_fwd, x | {"v": v, "S0": S}, o=v, initial_state=S, final_state=S)
        assert o is v and S1 is S and torch.equal(o, got[0]) and torch.equal(S, got[1])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_many_packed_units(dtype):
    edges = [0, 0, 1, 66, 130, 194, 250, 250]
    n = units(1 / 7)
    x = make(1, 260, n, 96, 100, dtype, edges=edges, seed=2)
    want = reference(x, edges=edges)
    for name in "qkv":
        x[name][:, 250:] = float("nan")
    o = torch.full((1, 260, n, 100), 7.0, dtype=dtype, device="cuda")
    got = call(kda.kda_delta_chunk_fwd, x, edges=edges, o=o)
    check(got, want, dtype, 96, rows=250)
    assert (o[:, 250:] == 7).all()
    for s in (0, 6):
        assert torch.equal(got[1][s].cpu(), x["S0"][s])


def test_a_value_that_is_not_finite_stays_in_its_channel():
    x = make(1, 150, units(1), 128, 64, torch.float32, seed=6)
    clean = call(kda.kda_delta_chunk_fwd, x)[0]
    x["v"][0, 70, 1, 3] = float("inf")
    o, S = call(kda.kda_delta_chunk_fwd, x)
    keep = torch.ones_like(o, dtype=torch.bool)
    keep[:, 70:, 1, 3] = False
    assert torch.equal(o[keep], clean[keep]) and not torch.isfinite(o[0, 70, 1, 3])
    assert not torch.isfinite(S[0, 1, :, 3]).all() and torch.isfinite(S[0, 1, :, 4]).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", [1, 4, 5, 16, 17])
@pytest.mark.parametrize("K,V", [(128, 128), (64, 40), (100, 7)])
def test_few_tokens(dtype, T, K, V):
    for B, H in ((1, 3), (units(1) // 4 + 1, 4)):
        x = make(B, T, H, K, V, dtype, seed=T + B)
        check(call(kda.kda_delta_chunk_fwd, x), reference(x), dtype, K)
        o, S = call(kda.kda_delta_chunk_fwd, x, output_final_state=False)
        assert S is None and torch.equal(o, call(kda.kda_delta_chunk_fwd, x)[0])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_many_short_sequences(dtype):
    lengths = [7, 1, 0, 5, 16, 17, 3, 31, 33, 2] * 3
    edges = [0]
    for n in lengths:
        edges.append(edges[-1] + n)
    x = make(1, edges[-1], 8, 128, 72, dtype, edges=edges, seed=12)
    check(call(kda.kda_delta_chunk_fwd, x, edges=edges), reference(x, edges=edges), dtype, 128)
