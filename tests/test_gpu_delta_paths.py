"""Schedules of the gated delta rule's tensor-core kernel: cut units, many units, long sequences, a wait that gives up."""
import pytest
import torch

from delta_reference import F32
from test_gpu_delta import DEV, call, check, make, reference

pytestmark = pytest.mark.gpu

kda = pytest.importorskip("chunked_kda_gb300")


@pytest.fixture
def hooks():
    yield kda.kda_test_hooks
    kda.kda_test_hooks()


@pytest.mark.parametrize("B,T,H,V,sms", [(2, 400, 2, 128, 3), (1, 1000, 3, 128, 2), (3, 330, 1, 256, 5), (1, 700, 7, 72, 5)])
def test_cut_units_are_bitwise_whole_ones(hooks, B, T, H, V, sms):
    x = make(B, T, H, 128, V, torch.bfloat16, seed=41)
    size = lambda: kda.kda_delta_chunk_workspace_bytes(torch.bfloat16, B, T, H, 128, V)  # noqa: E731
    assert size() == 0
    whole = call(kda.kda_delta_chunk_fwd, x)
    hooks(sm_count=sms)
    assert size() > 0
    ws = torch.randint(256, (size(),), dtype=torch.uint8, device=DEV)  # its contents do not matter
    cut = call(kda.kda_delta_chunk_fwd, x, workspace=ws)
    assert torch.equal(cut[0], whole[0]) and torch.equal(cut[1], whole[1])
    S = x["S0"].to(DEV)  # in place
    o, S1 = call(kda.kda_delta_chunk_fwd, x, initial_state=S, final_state=S)
    assert S1 is S and torch.equal(o, whole[0]) and torch.equal(S, whole[1])
    check(cut, reference(x), torch.bfloat16, 128)


def test_cut_units_replayed_from_a_graph(hooks):
    hooks(sm_count=3)
    x = make(2, 400, 2, 128, 128, torch.bfloat16, seed=43)
    want = call(kda.kda_delta_chunk_fwd, x)
    d = {n: t.to(DEV) for n, t in x.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, S = kda.kda_delta_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], initial_state=d["S0"], output_final_state=True)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want[0]) and torch.equal(S, want[1])


@pytest.mark.parametrize("raw", [False, True])
def test_many_units_over_many_chunks(raw):
    """More units than the device has multiprocessors, each over many chunks: every block's waits in every order that
    comes about, a few units against float64 and each against itself at once more."""
    B, T, H = 2, 1500, 100
    x = make(B, T, H, 128, 128, torch.bfloat16, Hk=50, raw=raw, seed=45)
    kda.kda_fused_wait_timeouts(reset=True)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    first = call(kda.kda_delta_chunk_fwd, x, raw=raw, status=status)
    for _ in range(4):
        again = call(kda.kda_delta_chunk_fwd, x, raw=raw)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    assert kda.kda_fused_wait_timeouts() == 0 and int(status) == 0
    for h in (0, 37, 99):
        part = {n: t for n, t in x.items()}
        part |= {n: x[n][:, :, h // 2:h // 2 + 1] for n in "qk"} | {n: x[n][:, :, h:h + 1] for n in ("v", "g", "beta")}
        part["S0"] = x["S0"][:, h:h + 1]
        if raw:
            part |= {n: x[n][h:h + 1] for n in ("A_log", "dt_bias")}
        check((first[0][:, :, h:h + 1], first[1][:, h:h + 1]), reference(part, raw=raw), torch.bfloat16, 128)


def test_a_long_sequence_with_hardly_any_decay():
    """6000 tokens (94 chunks): the state's error over many chunks stays float32's."""
    x = make(1, 6000, 1, 128, 128, torch.bfloat16, seed=47, slow=True)
    check(call(kda.kda_delta_chunk_fwd, x), reference(x), torch.bfloat16, 128)


def test_many_packed_sequences():
    """More sequences than the blocks rank by length."""
    lens = [(7 * i) % 70 for i in range(200)]
    edges = [0]
    for n in lens:
        edges.append(edges[-1] + n)
    x = make(1, edges[-1] + 3, 1, 64, 64, torch.bfloat16, edges=edges, seed=49)
    check(call(kda.kda_delta_chunk_fwd, x, edges=edges), reference(x, edges=edges), torch.bfloat16, 64, rows=edges[-1])


def test_a_wait_that_gives_up_is_reported(hooks):
    x = make(1, 300, 2, 128, 128, torch.bfloat16, seed=51)
    want = call(kda.kda_delta_chunk_fwd, x)
    kda.kda_fused_wait_timeouts(reset=True)
    hooks(wait_timeout_chunk=2)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    call(kda.kda_delta_chunk_fwd, x, status=status)
    assert int(status) == 1 and kda.kda_fused_wait_timeouts(reset=True) >= 2
    hooks()
    status.zero_()
    got = call(kda.kda_delta_chunk_fwd, x, status=status)
    assert int(status) == 0 and kda.kda_fused_wait_timeouts() == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
