"""The gated delta rule with the output in the values' place and the state in its own, in every kernel: the same as apart."""
import pytest
import torch

from test_gpu_delta import call, kda, make

pytestmark = pytest.mark.gpu


@pytest.fixture
def hooks():
    yield kda.kda_test_hooks
    kda.kda_test_hooks()


def same_in_place(fn, x, **kw):
    want = call(fn, x, **kw)
    for _ in range(3):
        v, S = x["v"].to("cuda"), x["S0"].to("cuda")
        o, S1 = call(fn, x | {"v": v, "S0": S}, o=v, initial_state=S, final_state=S, **kw)
        assert o is v and S1 is S and torch.equal(o, want[0]) and torch.equal(S, want[1])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("K,V", [(64, 64), (128, 128), (128, 256), (100, 77), (128, 126), (251, 254), (236, 253)])
@pytest.mark.parametrize("T", [1, 9])
def test_tokens(dtype, K, V, T):
    same_in_place(kda.kda_delta_recurrent_fwd, make(40, T, 8, K, V, dtype, Hk=4, seed=T + K))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", [1, 4, 15])
def test_a_few_tokens_of_the_chunked_form(dtype, T):
    same_in_place(kda.kda_delta_chunk_fwd, make(40, T, 8, 128, 128, dtype, seed=T))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("K,V", [(128, 128), (64, 200), (256, 64)])
def test_chunks(dtype, K, V):
    same_in_place(kda.kda_delta_chunk_fwd, make(2, 200, 6, K, V, dtype, Hk=3, seed=K))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_packed_chunks_that_end_inside_tiles(dtype):
    edges = [0, 1, 66, 66, 130, 194, 323]
    same_in_place(kda.kda_delta_chunk_fwd, make(1, 323, 6, 128, 128, dtype, edges=edges, seed=2), edges=edges)
    same_in_place(kda.kda_delta_recurrent_fwd, make(1, 323, 6, 128, 128, dtype, edges=edges, seed=2), edges=edges)


def test_cut_units(hooks):
    hooks(sm_count=3)
    assert kda.kda_delta_chunk_workspace_bytes(torch.bfloat16, 2, 400, 2, 128, 128) > 0
    same_in_place(kda.kda_delta_chunk_fwd, make(2, 400, 2, 128, 128, torch.bfloat16, seed=3))
