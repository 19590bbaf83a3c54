"""The gated delta rule and the norm and rotation of its rows where offsets pass 32 bits: the last sequences' results are
those of a call with nothing in front of them."""
import pytest
import torch

from test_gpu_delta import DEV, kda

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def memory():
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GB")
    yield
    torch.cuda.empty_cache()


def inputs(gen, dtype, T, H, D):
    r = lambda *s: torch.randn(*s, generator=gen, device=DEV, dtype=dtype)  # noqa: E731
    q, k, v = r(1, T, H, D).mul_(D ** -0.5), r(1, T, H, D).mul_(D ** -0.5), r(1, T, H, D)
    g = -torch.rand(1, T, H, generator=gen, device=DEV)
    return q, k, v, g, torch.rand(1, T, H, generator=gen, device=DEV).to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_chunks(dtype):
    T, H, D, last = (1 << 18) + 300, 64, 128, 190
    assert (T - last) * H * D > 1 << 31
    x = inputs(torch.Generator(device=DEV).manual_seed(1), dtype, T, H, D)
    S0 = torch.full((2, H, D, D), 0.1, device=DEV)
    cu = torch.tensor([0, T - last, T], device=DEV, dtype=torch.int32)
    o, S = kda.kda_delta_chunk_fwd(*x, initial_state=S0, output_final_state=True, cu_seqlens=cu)
    assert torch.isfinite(S).all()
    alone = torch.tensor([0, last], device=DEV, dtype=torch.int32)
    want = kda.kda_delta_chunk_fwd(*(t[:, T - last:].clone() for t in x), initial_state=S0[1:].clone(), output_final_state=True,
                                   cu_seqlens=alone)
    assert torch.equal(o[:, T - last:], want[0]) and torch.equal(S[1:], want[1])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("K,V", [(128, 128), (128, 256), (128, 126), (236, 253)])
def test_states_of_single_tokens(dtype, K, V):
    H = 64
    N = (1 << 31) // (H * K * V) + 3
    gen = torch.Generator(device=DEV).manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    q, k, v = (r(N, 1, H, K) * K ** -0.5).to(dtype), (r(N, 1, H, K) * K ** -0.5).to(dtype), r(N, 1, H, V).to(dtype)
    g, beta, S = -r(N, 1, H).abs(), torch.sigmoid(r(N, 1, H)).to(dtype), torch.full((N, H, K, V), 0.1, device=DEV)
    want = kda.kda_delta_recurrent_fwd(*(t[-2:].clone() for t in (q, k, v, g, beta)), initial_state=S[-2:].clone(), output_final_state=True)
    o, _ = kda.kda_delta_recurrent_fwd(q, k, v, g, beta, initial_state=S, final_state=S)
    assert torch.equal(o[-2:], want[0]) and torch.equal(S[-2:], want[1])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R", [128, 104, 34])
def test_rows_of_queries_and_keys(dtype, R):
    T, Hq, Hk, D, last = (1 << 18) + 77, 48, 8, 128, 60
    rows = torch.randn(1, T, Hq + 2 * Hk, D, generator=torch.Generator(device=DEV).manual_seed(3), device=DEV, dtype=dtype)
    assert (T - last) * (Hq + 2 * Hk) * D > 1 << 31
    pos = torch.arange(T, device=DEV, dtype=torch.int32)[None] * 1000
    f = (1e4 ** (-torch.arange(0, R, 2) / R)).float().to(DEV)
    w = torch.linspace(0.5, 1.5, D, device=DEV)
    part = rows[:, T - last:].clone()
    want = kda.kda_qk_norm_rope_fwd(part[:, :, :Hq], part[:, :, Hq:Hq + Hk], w, w, positions=pos[:, T - last:].contiguous(), inv_freq=f)
    q, k = rows[:, :, :Hq], rows[:, :, Hq:Hq + Hk]
    kda.kda_qk_norm_rope_fwd(q, k, w, w, positions=pos, inv_freq=f, q_out=q, k_out=k)
    half = 2.0 ** (-23 if dtype == torch.float32 else -7)  # the two calls may take different kernels: a step of an output
    for got, x in ((q, want[0]), (k, want[1])):
        got, x = got[:, T - last:].double(), x.double()
        assert ((got - x).abs() <= 4e-6 * x.norm(dim=-1, keepdim=True) + half * x.abs()).all()
    assert torch.equal(rows[:, T - last:, Hq + Hk:], part[:, :, Hq + Hk:])
