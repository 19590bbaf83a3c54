"""Calls of the gated delta rule side by side on several streams: units cut between multiprocessors (whose second parts wait for
the first ones), whole ones, FP32 chunks, single tokens, and a graph that is replayed meanwhile.  Each has its own results."""
import torch
import pytest

from test_gpu_delta import DEV, kda

pytestmark = pytest.mark.gpu


def prepared(fn, dtype, B, T, H, K, V, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    q, k = (torch.nn.functional.normalize(r(B, T, H, K), dim=-1).to(dtype) for _ in range(2))
    x = (q, k, r(B, T, H, V).to(dtype), -r(B, T, H).abs(), torch.sigmoid(r(B, T, H)).to(dtype))
    S = 0.1 * r(B, H, K, V)
    return lambda **kw: fn(*x, initial_state=S, output_final_state=True, **kw)


def test_side_by_side():
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    chunk, token = kda.kda_delta_chunk_fwd, kda.kda_delta_recurrent_fwd
    H = sms // 4 + 7  # four sequences: a part more units than multiprocessors
    assert kda.kda_delta_chunk_workspace_bytes(torch.bfloat16, 4, 512, H, 128, 128) > 0
    calls = [prepared(chunk, torch.bfloat16, 4, 512, H, 128, 128, 1), prepared(chunk, torch.bfloat16, 4, 512, H, 128, 128, 2),
             prepared(chunk, torch.bfloat16, 1, 700, 40, 64, 136, 3), prepared(chunk, torch.float32, 2, 200, 20, 128, 128, 4),
             prepared(token, torch.bfloat16, 64, 1, 32, 128, 256, 5), prepared(token, torch.float32, 30, 3, 8, 100, 77, 6)]
    want = [c() for c in calls]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = calls[0]()
    torch.cuda.synchronize()
    kda.kda_fused_wait_timeouts(reset=True)
    streams, side, got = [torch.cuda.Stream() for _ in calls], torch.cuda.Stream(), []
    for _ in range(10):
        with torch.cuda.stream(side):
            graph.replay()
        got.append([c(stream=s) for c, s in zip(calls, streams)])
    torch.cuda.synchronize()
    assert kda.kda_fused_wait_timeouts() == 0
    for outs in got + [[captured]]:
        for (o, S), (wo, wS) in zip(outs, want):
            assert torch.equal(o, wo) and torch.equal(S, wS)
