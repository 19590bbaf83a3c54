"""Calls of one operator from several host threads at once, whose sizes ask for different amounts of shared memory of the same
kernel: none is refused, and each has its own results.  The library's functions are called as they are: the binding's own work
between two calls would keep them from meeting."""
import threading

import pytest
import torch

from test_gpu_delta import kda, make

pytestmark = pytest.mark.gpu
DEV = "cuda"


def side_by_side(*calls, times=4000):
    """calls: (function of the library, arguments before the stream, outputs).  Each again and again in a thread of its own;
    its outputs are those of the call by itself."""
    def once(fn, args):
        return fn(*args, torch.cuda.current_stream().cuda_stream)

    assert [once(fn, args) for fn, args, _ in calls] == [0] * len(calls)
    torch.cuda.synchronize()
    want = [[t.clone() for t in outs] for _, _, outs in calls]
    start, codes, streams = threading.Barrier(len(calls)), [None] * len(calls), [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()

    def work(i):
        fn, args, _ = calls[i]
        stream, bad = streams[i].cuda_stream, 0
        start.wait(60)
        for _ in range(times):
            bad += fn(*args, stream) != 0
        codes[i] = bad

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert codes == [0] * len(calls)  # calls that were refused
    for (_, _, outs), w in zip(calls, want):
        assert all(torch.equal(a, b) for a, b in zip(outs, w))


def p(t):
    return None if t is None else t.data_ptr()


def tokens(K, V):
    x = {n: None if t is None else t.to(DEV) for n, t in make(1, 1, 1, K, V, torch.bfloat16, seed=K).items()}
    x["o"], x["S1"] = torch.empty_like(x["v"]), torch.empty_like(x["S0"])
    args = (p(x["q"]), p(x["k"]), p(x["v"]), 1, p(x["g"]), 0, None, None, 0, p(x["beta"]), 1, p(x["S0"]), p(x["S1"]), None, 0, 1, 1, 1, 1,
            K, V, p(x["o"]), 1, 0)
    return kda.load_library().kda_delta_recurrent_fwd, args, list(x.values())  # (the inputs live as long as the call)


@pytest.mark.parametrize("sizes", [[(128, 128), (128, 104), (256, 256), (200, 80)], [(128, 126), (256, 210), (200, 100), (160, 90)],
                                   [(140, 77), (212, 253), (230, 99), (250, 201)]])
def test_single_tokens(sizes):
    side_by_side(*(tokens(K, V) for K, V in sizes))


def test_norm_and_rotation():
    def rope(R):
        tokens, heads, D = 2600, 64, 128
        x = torch.randn(tokens, heads, D, device=DEV).bfloat16()
        y, pos, f = torch.empty_like(x), torch.arange(tokens, device=DEV, dtype=torch.int32), torch.full((R // 2,), 0.1, device=DEV)
        n = heads * D
        args = (p(x), n, None, 0, 1, None, None, 1, 1e-6, p(pos), 1, p(f), None, R, 0, 1.0, tokens, heads, 0, D, p(y), n, None, 0)
        return kda.load_library().kda_qk_norm_rope_fwd, args, [y, x, pos, f]

    side_by_side(*(rope(R) for R in (16, 128, 32, 64)))


def test_norm_of_long_rows():
    w = torch.ones(4608, device=DEV)

    def norm(gated):
        x = torch.randn(1300, 4608, device=DEV).bfloat16()
        h, y = torch.empty_like(x), torch.empty_like(x)
        args = (p(x), 1, None, 1, None, p(x) if gated else None, 1, 1.0, None, p(w), 1e-6, 1300, 4608, p(h), p(y))
        return kda.load_library().kda_block_norm_fwd, args, [h, y, x, w]

    side_by_side(norm(False), norm(True), norm(False), norm(True))


def test_decayed_attention_in_float32():
    def decay(K):
        q, k, v = (torch.randn(1, 64, 1, K, device=DEV) for _ in range(3))
        a, o = -torch.rand(1, 64, 1, device=DEV), torch.empty(1, 64, 1, K, device=DEV)
        ws = torch.empty(max(256, kda.kda_decay_chunk_workspace_bytes(torch.float32, 1, 64, 1, K, K)), device=DEV, dtype=torch.uint8)
        args = (p(q), p(k), p(v), 0, p(a), 1, None, None, None, 0, 1, 64, 1, 1, K, K, p(o), 0, p(ws), ws.numel(), None)
        return kda.load_library().kda_decay_chunk_fwd, args, [o, q, k, v, a, ws]

    side_by_side(*(decay(K) for K in (40, 250, 100, 180)))
