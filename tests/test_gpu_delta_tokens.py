"""Single tokens and short sequences of the gated delta rule at the state sizes that its tiles are cut by: a whole state a
block (three sizes of block) and column blocks, the last one part empty.  Against float64; tolerances of the other sizes."""
import pytest
import torch

from test_gpu_delta import call, check, kda, make, reference

pytestmark = pytest.mark.gpu

SIZES = [  # K, V: bytes of a state up to 16 KB, 40 KB, 64 KB, and beyond: columns of a block
    (64, 64), (16, 256), (33, 124), (1, 4),  # 64 threads
    (65, 64), (100, 100), (40, 256), (256, 36),  # 128
    (101, 104), (64, 256), (256, 64), (80, 204),  # 256
    (128, 132), (234, 128), (256, 256), (251, 200), (65, 256), (256, 68),  # column blocks
    (128, 126), (256, 210), (4, 1), (100, 77), (212, 253),  # whole, two columns or one a thread
    (256, 254), (99, 77), (255, 3), (17, 6),  # by single loads
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("K,V", SIZES)
def test_sizes_of_a_state(dtype, K, V):
    for B, T, H, Hk in ((3, 1, 4, 2), (2, 5, 3, 3)):
        x = make(B, T, H, K, V, dtype, Hk=Hk, seed=K + V + T)
        want = reference(x)
        got = call(kda.kda_delta_recurrent_fwd, x)
        check(got, want, dtype, K)
        # the state in place, and none to begin with
        S = x["S0"].to("cuda")
        o, S1 = call(kda.kda_delta_recurrent_fwd, x | {"S0": None}, initial_state=S, final_state=S)
        assert S1 is S and torch.equal(S, got[1]) and torch.equal(o, got[0])
        none = x | {"S0": None}
        check(call(kda.kda_delta_recurrent_fwd, none), reference(x | {"S0": torch.zeros_like(x["S0"])}), dtype, K)


@pytest.mark.parametrize("K,V", [(64, 64), (234, 128), (256, 256)])
def test_packed_tokens_leave_what_is_not_theirs(K, V):
    edges = [0, 0, 2, 3, 3, 6]
    x = make(1, 9, 2, K, V, torch.bfloat16, edges=edges, seed=3)
    want = reference(x, edges=edges)
    for name in "qkv":
        x[name][:, 6:] = float("nan")
    o = torch.full((1, 9, 2, V), 7.0, dtype=torch.bfloat16, device="cuda")
    got = call(kda.kda_delta_recurrent_fwd, x, edges=edges, o=o)
    check(got, want, torch.bfloat16, K, rows=6)
    assert (o[:, 6:] == 7).all()
    for n in (0, 3):
        assert torch.equal(got[1][n].cpu(), x["S0"][n])


@pytest.mark.parametrize("K,V", [(128, 128), (128, 256), (100, 77), (64, 64)])
def test_tokens_captured_and_on_other_streams(K, V):
    xs = [make(2, 1, 3, K, V, torch.bfloat16, seed=s) for s in (61, 62)]
    want = [call(kda.kda_delta_recurrent_fwd, x) for x in xs]
    d = {n: t.to("cuda") for n, t in xs[0].items()}
    S = torch.empty_like(d["S0"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, _ = kda.kda_delta_recurrent_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], initial_state=d["S0"], final_state=S)
    for x, (wo, wS) in zip(xs, want):
        for n in d:
            d[n].copy_(x[n])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, wo) and torch.equal(S, wS)
    dev, got = [{n: t.to("cuda") for n, t in x.items()} for x in xs], []
    torch.cuda.synchronize()
    for y in dev:  # two calls at once
        got.append(kda.kda_delta_recurrent_fwd(y["q"], y["k"], y["v"], y["g"], y["beta"], initial_state=y["S0"],
                                               output_final_state=True, stream=torch.cuda.Stream()))
    torch.cuda.synchronize()
    for (o, S), (wo, wS) in zip(got, want):
        assert torch.equal(o, wo) and torch.equal(S, wS)
    assert kda.kda_fused_wait_timeouts() == 0
