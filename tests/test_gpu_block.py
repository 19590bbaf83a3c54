"""The operators around the recurrence on the GPU, against float64.

Bounds, with u = 2^-24 (half a float32 step) and w = 2^-8 (half a bf16 step), element by element:
  rounding to the output's type adds its half step times the value;
  a float32 sum of n products is off by at most (n + 2) u times the sum of the absolute values, and
  a root, a quotient or an exponential by a few u;
  the chunked bf16 form rounds the scores and the state once to bf16 as operands of products, which
  adds at most w times the sum of the absolute values of the terms (block_reference).
"""
import pytest
import torch

import block_reference as ref
from block_reference import F32, HALF

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def kda():
    import __graft_entry__

    __graft_entry__.build()
    import chunked_kda_gb300

    return chunked_kda_gb300


def dev(x):
    return None if x is None else x.cuda()


def close(got, want, bound, what):
    d = (got.double().cpu() - want).abs()
    bad = ~(d <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((d / bound.clamp_min(1e-300)).max()):.3g} of its bound"


def inputs(seed, B, T, H, Hk, K, V, dtype, N, fixed=False, state=True, span=3.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    q, k = (torch.nn.functional.normalize(r(B, T, Hk, K), dim=-1).to(dtype) for _ in range(2))
    v = r(B, T, H, V).to(dtype)
    decay = -torch.rand(H, generator=g) * 0.3 if fixed else -span * torch.rand(B, T, H, generator=g) ** 3
    return q, k, v, decay, (r(N, H, K, V) * 0.3 if state else None)


def check(kda, fn, x, edges=None, o_dtype=None, inplace=False, chunked=True):
    q, k, v, decay, S0 = x
    o_ref, S_ref, oa, Sa = ref.decay_attention(q, k, v, decay, S0, edges)
    cu = None if edges is None else torch.tensor(edges, dtype=torch.int32, device="cuda")
    s0 = dev(S0)
    o, S = getattr(kda, fn)(dev(q), dev(k), dev(v), dev(decay), initial_state=s0, output_final_state=True,
                            cu_seqlens=cu, o_dtype=o_dtype, final_state=s0 if inplace else None)
    torch.cuda.synchronize()
    T = max([b - a for a, b in zip(edges, edges[1:])] or [0]) if edges is not None else q.shape[1]
    # float32 sums over the channels and tokens, the state's running sum (a chunk of 64 tokens in
    # twelve accumulations) and exponentials of sums of up to 64 decays
    f32 = (q.shape[3] + 128 + T) * F32
    operand = HALF[BF] * (1 + 2.0 ** -6) if chunked and q.dtype == BF else 0.0
    rows = slice(0, edges[-1]) if edges is not None else slice(None)
    close(o[:, rows], o_ref[:, rows], HALF[o.dtype] * o_ref.abs()[:, rows] + (operand + f32) * oa[:, rows] + 1e-30, "o")
    close(S, S_ref, f32 * Sa + 1e-30, "state")
    if o_ref[:, rows].numel() > 4096 and q.dtype == BF:  # random roundings: their 2-norm
        assert (o[:, rows].double().cpu() - o_ref[:, rows]).norm() <= HALF[BF] * o_ref[:, rows].norm()
    return o, S


SIZES = [(64, 64), (128, 128), (64, 128), (128, 64), (256, 256), (128, 256), (40, 72), (1, 1), (255, 3)]


@pytest.mark.parametrize("fn", ["kda_decay_chunk_fwd", "kda_decay_recurrent_fwd"])
@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("K,V", SIZES)
def test_head_sizes(kda, fn, dtype, K, V):
    check(kda, fn, inputs(K + V, 2, 150, 2, 1, K, V, dtype, 2), chunked="chunk" in fn)


@pytest.mark.parametrize("fn", ["kda_decay_chunk_fwd", "kda_decay_recurrent_fwd"])
@pytest.mark.parametrize("T", [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200, 321])
@pytest.mark.parametrize("fixed", [False, True])
def test_lengths(kda, fn, T, fixed):
    x = inputs(T, 1, T, 3, 3, 128, 128, BF, 1, fixed)
    o, S = check(kda, fn, x, chunked="chunk" in fn)
    if T == 0:
        assert torch.equal(S.cpu(), x[4])


@pytest.mark.parametrize("fn", ["kda_decay_chunk_fwd", "kda_decay_recurrent_fwd"])
@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("H,Hk", [(1, 1), (6, 2), (5, 5), (8, 1)])
def test_heads_that_share_queries(kda, fn, dtype, H, Hk):
    check(kda, fn, inputs(H, 2, 70, H, Hk, 64, 128, dtype, 2), chunked="chunk" in fn)


PACKED = [[0, 64, 128], [0, 0, 1, 1, 70, 200], [0, 5, 5, 5, 133], [0, 130, 130], [0, 0, 0], [0], [0, 1, 2, 3, 4, 5]]


@pytest.mark.parametrize("fn", ["kda_decay_chunk_fwd", "kda_decay_recurrent_fwd"])
@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("edges", PACKED)
@pytest.mark.parametrize("K", [128, 96])
def test_packed(kda, fn, dtype, edges, K):
    """Empty sequences pass their states through, and rows behind the last offset are NaN on the way
    in and untouched on the way out."""
    cap = edges[-1] + 37
    x = inputs(len(edges), 1, cap, 2, 2, K, 128, dtype, len(edges) - 1)
    q, k, v, decay, S0 = x
    want = ref.decay_attention(q, k, v, decay, S0, edges)
    for t in (q, k, v, decay):
        t[:, edges[-1]:] = float("nan")
    o = torch.full(v.shape, 7.0, dtype=dtype, device="cuda")
    s = dev(S0)
    cu = torch.tensor(edges, dtype=torch.int32, device="cuda")
    _, S = getattr(kda, fn)(dev(q), dev(k), dev(v), dev(decay), initial_state=s, final_state=s, cu_seqlens=cu, o=o)
    torch.cuda.synchronize()
    f32 = (K + 128 + cap) * F32
    operand = HALF[BF] * (1 + 2.0 ** -6) if "chunk" in fn and dtype == BF else 0.0
    n = edges[-1]
    close(o[:, :n], want[0][:, :n], HALF[dtype] * want[0][:, :n].abs() + (operand + f32) * want[2][:, :n] + 1e-30, "o")
    assert bool((o[:, n:] == 7.0).all())
    close(S, want[1], f32 * want[3] + 1e-30, "state")
    for i, (a, b) in enumerate(zip(edges, edges[1:])):
        if a == b:
            assert torch.equal(S[i].cpu(), S0[i])


@pytest.mark.parametrize("fn", ["kda_decay_chunk_fwd", "kda_decay_recurrent_fwd"])
@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("kind", ["none", "strong", "reset", "lowest", "mixed"])
def test_decays(kda, fn, dtype, kind):
    """No decay, decays whose products underflow, and decays of -inf or of the type's lowest value,
    which clear the state."""
    x = list(inputs(5, 1, 200, 2, 2, 128, 64, dtype, 1))
    g = torch.Generator().manual_seed(3)
    a = x[3]
    if kind == "none":
        a.zero_()
    elif kind == "strong":
        a.copy_(-20.0 * torch.rand(a.shape, generator=g))
    else:
        at = torch.rand(a.shape, generator=g) < 0.05
        a[at] = torch.finfo(torch.float32).min if kind == "lowest" else -float("inf")
        if kind == "mixed":
            a[torch.rand(a.shape, generator=g) < 0.2] = -1000.0
    check(kda, fn, x, chunked="chunk" in fn)


@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_chunked_float32_output_and_null_state(kda, dtype):
    x = inputs(8, 2, 190, 2, 2, 128, 128, dtype, 2, state=False)
    check(kda, "kda_decay_chunk_fwd", x, o_dtype=torch.float32)


@pytest.mark.parametrize("T,H,B", [(4096, 1, 1), (3001, 2, 1), (2048, 3, 2)])
def test_long_prompts_with_few_heads(kda, T, H, B):
    check(kda, "kda_decay_chunk_fwd", inputs(T, B, T, H, H, 128, 128, BF, B, fixed=H == 2))


@pytest.mark.parametrize("sms,B,T,H,K,V", [(3, 2, 1270, 2, 128, 128), (2, 1, 1500, 5, 64, 128), (7, 3, 1536, 3, 128, 64), (3, 1, 1601, 2, 128, 256), (3, 1, 1601, 2, 256, 256)])
@pytest.mark.parametrize("inplace", [False, True])
def test_units_cut_between_processors(kda, sms, B, T, H, K, V, inplace):
    """More units than multiprocessors and a last wave part-empty: some are cut and joined by their state."""
    x = inputs(T, B, T, H, H, K, V, BF, B)
    before = kda.kda_fused_wait_timeouts()
    try:
        kda.kda_test_hooks(sm_count=sms)
        o, S = check(kda, "kda_decay_chunk_fwd", x, inplace=inplace)
        again = kda.kda_decay_chunk_fwd(*(dev(t) for t in x[:4]), initial_state=dev(x[4]), output_final_state=True)
        assert torch.equal(again[0], o) and torch.equal(again[1], S)
        check(kda, "kda_decay_chunk_fwd", (*x[:4], None))
    finally:
        kda.kda_test_hooks()
    assert kda.kda_fused_wait_timeouts() == before


def test_cut_units_replayed_from_a_graph(kda):
    """Each replay clears the counters that the pieces of a unit meet at."""
    x = [dev(t) for t in inputs(7, 2, 1400, 2, 2, 128, 128, BF, 2)]
    before = kda.kda_fused_wait_timeouts()
    try:
        kda.kda_test_hooks(sm_count=3)
        want = kda.kda_decay_chunk_fwd(*x[:4], initial_state=x[4], output_final_state=True)
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                o, S = kda.kda_decay_chunk_fwd(*x[:4], initial_state=x[4], output_final_state=True)
    finally:
        kda.kda_test_hooks()
    for _ in range(3):
        o.zero_()
        S.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want[0]) and torch.equal(S, want[1])
    assert kda.kda_fused_wait_timeouts() == before


def test_chunked_continues_in_single_tokens(kda):
    """A prompt in chunks and then token by token, in place, is the whole sequence at once."""
    q, k, v, a, _ = (dev(t) for t in inputs(1, 2, 100, 4, 2, 128, 128, BF, 2, state=False))
    whole, S = kda.kda_decay_chunk_fwd(q, k, v, a, output_final_state=True)
    cut = lambda t, lo, hi: t[:, lo:hi].contiguous()  # noqa: E731
    o, s = kda.kda_decay_chunk_fwd(*(cut(t, 0, 90) for t in (q, k, v, a)), output_final_state=True)
    parts = [o]
    for t in range(90, 100):
        o, s2 = kda.kda_decay_recurrent_fwd(*(cut(x, t, t + 1) for x in (q, k, v, a)), initial_state=s, final_state=s)
        assert s2 is s
        parts.append(o)
    got = torch.cat(parts, 1)
    assert (got - whole).double().norm() <= 2 * HALF[BF] * whole.double().norm()
    assert (s - S).double().norm() <= 256 * F32 * S.double().norm()


def test_graph_replay_and_side_stream(kda):
    q, k, v, a, S0 = (dev(t) for t in inputs(2, 1, 300, 4, 4, 128, 128, BF, 1))
    z, w = torch.randn_like(v), torch.rand(128, device="cuda")

    def block():
        o, S = kda.kda_decay_chunk_fwd(q, k, v, a, initial_state=S0, output_final_state=True)
        return kda.kda_gated_norm_fwd(o, z, w), S

    want = block()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = kda.kda_decay_chunk_fwd(q, k, v, a, initial_state=S0, output_final_state=True, stream=side)
    side.synchronize()
    assert torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block()
    q.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    again = block()
    torch.cuda.synchronize()
    assert torch.equal(out[0], again[0]) and torch.equal(out[1], again[1])


# ------------------------------------------------------------------ norms

@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("V", [1, 7, 16, 64, 72, 128, 200, 256, 257, 512, 1000, 4096])
@pytest.mark.parametrize("act", [0, 1, 2])
def test_gated_norm(kda, dtype, V, act):
    g = torch.Generator().manual_seed(V)
    x, z = torch.randn(3, 11, V, generator=g).to(dtype), (3 * torch.randn(3, 11, V, generator=g)).to(dtype)
    x[0, 0], x[0, 1] = 0, 1e-6
    w = torch.rand(V, generator=g) if V % 2 else None
    y = kda.kda_gated_norm_fwd(dev(x), dev(z), dev(w), eps=1e-5, act=act)
    want = ref.gated_norm(x, z, w, 1e-5, act)
    fast = 2.0 ** -18 if dtype == BF else 24 * F32  # the gate's exponential
    close(y, want, (HALF[dtype] + fast + (V // 8 + 16) * F32) * want.abs() + 1e-30, "y")
    again = kda.kda_gated_norm_fwd(xd := dev(x), dev(z), dev(w), eps=1e-5, act=act, out=xd)
    assert again is xd and torch.equal(again, y)


@pytest.mark.parametrize("dtype,res", [(BF, BF), (BF, torch.float32), (torch.float32, BF), (torch.float32, torch.float32)])
@pytest.mark.parametrize("D", [1, 24, 100, 128, 1000, 2048, 2500, 4096, 8192, 9001, 12288, 20000])
@pytest.mark.parametrize("parts", ["all", "residual", "post", "plain", "pre", "gate"])
def test_block_norm(kda, dtype, res, D, parts):
    g = torch.Generator().manual_seed(D)
    rows = 5
    x = (0.5 * torch.randn(rows, D, generator=g)).to(dtype)
    x[1] = 0
    every = parts == "all"
    r = torch.randn(rows, D, generator=g).to(res) if every or parts in ("residual", "post") else None
    wp = torch.rand(D, generator=g) + 0.5 if every or parts == "post" else None
    z = torch.randn(rows, D, generator=g).to(dtype) if every or parts == "gate" else None
    c = torch.rand(D, generator=g) if every else None
    wn = torch.rand(D, generator=g) + 0.5 if every or parts in ("pre", "residual") else None
    rd = dev(r)
    into = rd if every else None
    h, y = kda.kda_block_norm_fwd(dev(x), rd, dev(wp), dev(z), dev(wn), scale=0.7, channel_scale=dev(c), eps=1e-6,
                                  act=2, residual_out=into)
    assert h.dtype == (res if r is not None else dtype) and y.dtype == dtype
    wh, wy = ref.block_norm(x, r, wp, z, 2, 0.7, c, wn, 1e-6)
    n = (D // 8 + 24) * F32 + (2.0 ** -18 if dtype == BF and z is not None else 24 * F32)
    size = wh.abs() + (0 if r is None else 2 * r.double().abs())  # h is a difference where signs differ
    close(h, wh, HALF[h.dtype] * wh.abs() + n * size + 1e-30, "h")
    rel = size / wh.abs().clamp_min(1e-300)
    mean = (size.square().mean(-1, keepdim=True) / (wh.square().mean(-1, keepdim=True) + 1e-6)).sqrt()
    close(y, wy, (HALF[dtype] + n * (rel + mean)) * wy.abs() + 1e-30, "y")


@pytest.mark.parametrize("dtype,res", [(BF, torch.float32), (BF, BF), (BF, None), (torch.float32, torch.float32)])
@pytest.mark.parametrize("D", [4104, 6000, 8192])
@pytest.mark.parametrize("gate", [False, True])
def test_block_norm_of_many_long_rows(kda, dtype, res, D, gate):
    """More rows than the blocks that stay resident hold at once; h in place of the stream."""
    g = torch.Generator().manual_seed(D)
    rows = 1217 if D == 6000 else 1500
    x = (0.5 * torch.randn(rows, D, generator=g)).to(dtype)
    x[rows - 1] = 0
    r = None if res is None else torch.randn(rows, D, generator=g).to(res)
    z = torch.randn(rows, D, generator=g).to(dtype) if gate else None
    wp, wn = (torch.rand(D, generator=g) + 0.5 for _ in range(2))
    wh, wy = ref.block_norm(x, r, wp, z, 1, 0.7, None, wn, 1e-6)
    rd = dev(r)
    before = kda.kda_fused_wait_timeouts()
    h, y = kda.kda_block_norm_fwd(dev(x), rd, dev(wp), dev(z), dev(wn), scale=0.7, act=1, residual_out=rd)
    assert r is None or h is rd
    n = (D // 8 + 24) * F32 + (2.0 ** -18 if dtype == BF and gate else 24 * F32)
    size = wh.abs() + (0 if r is None else 2 * r.double().abs())
    close(h, wh, HALF[h.dtype] * wh.abs() + n * size + 1e-30, "h")
    rel = size / wh.abs().clamp_min(1e-300)
    mean = (size.square().mean(-1, keepdim=True) / (wh.square().mean(-1, keepdim=True) + 1e-6)).sqrt()
    close(y, wy, (HALF[dtype] + n * (rel + mean)) * wy.abs() + 1e-30, "y")
    assert kda.kda_fused_wait_timeouts() == before


def test_block_norm_without_one_output(kda):
    x, w = torch.randn(3, 256, device="cuda"), torch.rand(256, device="cuda")
    import ctypes

    lib = kda.load_library()
    h, y = kda.kda_block_norm_fwd(x, pre_weight=w)
    h2, y2 = torch.full_like(x, 7.0), torch.full_like(x, 7.0)
    p = lambda t: None if t is None else ctypes.c_void_p(t.data_ptr())  # noqa: E731
    torch.cuda.synchronize()
    for a, b in ((h2, None), (None, y2)):
        assert lib.kda_block_norm_fwd(p(x), 0, None, 0, None, None, 1, 1.0, None, p(w), 1e-6, 3, 256, p(a), p(b), None) == 0
    torch.cuda.synchronize()
    assert torch.equal(h, h2) and torch.equal(y, y2)


# ------------------------------------------------------------------ convolution

def check_conv(kda, dtype, T, D, W, edges=None, B=1, act=2, bias=False, state=True, inplace=False):
    g = torch.Generator().manual_seed(T + D + W)
    N = B if edges is None else len(edges) - 1
    x = torch.randn(B, T, D, generator=g).to(dtype)
    w = torch.randn(D, W, generator=g)
    b = torch.randn(D, generator=g) if bias else None
    S0 = torch.randn(N, W - 1, D, generator=g).to(dtype) if state else None
    pre, want, last = ref.short_conv(x, w, b, act, S0, edges)
    n = T if edges is None else edges[-1]
    x[:, n:] = float("nan")
    cu = None if edges is None else torch.tensor(edges, dtype=torch.int32, device="cuda")
    s0, out = dev(S0), torch.full(x.shape, 7.0, dtype=dtype, device="cuda")
    y, S = kda.kda_short_conv_fwd(dev(x), dev(w), dev(b), act=act, initial_state=s0, output_final_state=True,
                                  cu_seqlens=cu, out=out, final_state=s0 if inplace else None)
    torch.cuda.synchronize()
    assert torch.equal(S.double().cpu(), last)
    assert bool((y[:, n:] == 7.0).all())
    # |d act / d z| <= 1.1; the terms' absolute values are at most their sum of W products of N(0, 1)
    terms = 1.1 * (W + 3) * F32 * (W + 1) * 25.0
    fast = 2.0 ** -17 if dtype == BF else 24 * F32
    close(y[:, :n], want[:, :n], (HALF[dtype] + fast) * want[:, :n].abs() + terms, "y")


@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("W", range(2, 9))
@pytest.mark.parametrize("D", [1, 12, 64, 1032])
def test_conv_dense(kda, dtype, W, D):
    check_conv(kda, dtype, 67, D, W, B=2, act=W % 3, bias=W % 2 == 0)


@pytest.mark.parametrize("T", [0, 1, 2, 3, 4, 5, 31, 32, 33, 64, 100])
@pytest.mark.parametrize("inplace", [False, True])
def test_conv_lengths(kda, T, inplace):
    check_conv(kda, BF, T, 256, 4, B=3, inplace=inplace)


@pytest.mark.parametrize("edges", PACKED + [[0, 2, 2, 5, 6, 100, 101], list(range(0, 200))])
@pytest.mark.parametrize("inplace", [False, True])
def test_conv_packed(kda, edges, inplace):
    if len(edges) == 1:
        pytest.skip("no sequence")
    check_conv(kda, BF, edges[-1] + 9, 136, 4, edges=edges, inplace=inplace)


def test_conv_without_state(kda):
    check_conv(kda, BF, 10, 128, 4, state=False)
    check_conv(kda, BF, 40, 128, 4, edges=[0, 2, 2, 38], state=False)


# ------------------------------------------------------------------ the binding's checks

def test_the_binding_refuses_what_it_can_see(kda):
    z = lambda *s, **k: torch.zeros(*s, device="cuda", **k)  # noqa: E731
    q, v, a = z(1, 8, 2, 64), z(1, 8, 4, 64), z(1, 8, 4)
    bad = [
        (ValueError, "heads", lambda: kda.kda_decay_recurrent_fwd(z(1, 8, 3, 64), z(1, 8, 3, 64), v, a)),
        (ValueError, "four dimensions", lambda: kda.kda_decay_chunk_fwd(q[0], q[0], v[0], a)),
        (ValueError, "decay must have shape", lambda: kda.kda_decay_chunk_fwd(q, q, v, z(1, 8, 2))),
        (TypeError, "decay", lambda: kda.kda_decay_chunk_fwd(q, q, v, a.bfloat16())),
        (TypeError, "v must be", lambda: kda.kda_decay_chunk_fwd(q, q, v.bfloat16(), a)),
        (ValueError, "contiguous", lambda: kda.kda_decay_chunk_fwd(q, z(1, 2, 8, 64).transpose(1, 2), v, a)),
        (ValueError, "initial_state", lambda: kda.kda_decay_chunk_fwd(q, q, v, a, initial_state=z(1, 4, 64, 32))),
        (ValueError, "CUDA", lambda: kda.kda_decay_chunk_fwd(q, q, v, a.cpu())),
        (ValueError, "requires grad", lambda: kda.kda_decay_chunk_fwd(q, q, v.clone().requires_grad_(), a)),
        (ValueError, "B == 1", lambda: kda.kda_decay_chunk_fwd(z(2, 8, 2, 64), z(2, 8, 2, 64), z(2, 8, 4, 64), z(2, 8, 4),
                                                               cu_seqlens=z(2, dtype=torch.int32))),
        (TypeError, "cu_seqlens", lambda: kda.kda_decay_chunk_fwd(q, q, v, a, cu_seqlens=z(2, dtype=torch.int64))),
        (TypeError, "float16", lambda: kda.kda_gated_norm_fwd(v.half(), v.half())),
        (ValueError, "gate must have shape", lambda: kda.kda_gated_norm_fwd(v, q)),
        (TypeError, "weight", lambda: kda.kda_gated_norm_fwd(v, v, z(64, dtype=torch.bfloat16))),
        (TypeError, "float64", lambda: kda.kda_block_norm_fwd(v.double())),
        (ValueError, "residual must have shape", lambda: kda.kda_block_norm_fwd(v, residual=q)),
        (ValueError, r"\[B, T, D\]", lambda: kda.kda_short_conv_fwd(q, z(64, 4))),
        (ValueError, "weight must have shape", lambda: kda.kda_short_conv_fwd(v[0], z(63, 4))),
        (ValueError, "initial_state must have shape", lambda: kda.kda_short_conv_fwd(v[0], z(64, 4), initial_state=z(8, 4, 64))),
    ]
    for kind, words, call in bad:
        with pytest.raises(kind, match=words):
            call()
    with pytest.raises(kda.KdaError, match="W must be"):
        kda.kda_short_conv_fwd(v[0], z(64, 9))
    with pytest.raises(kda.KdaError, match="aligned"):
        kda.kda_gated_norm_fwd(z(129)[1:].view(1, 128), z(1, 128))
    with pytest.raises(kda.KdaError, match="workspace"):
        big = z(1, 4096, 1, 128, dtype=torch.bfloat16)
        kda.kda_decay_chunk_fwd(big, big, big, z(1, 4096, 1), workspace=z(256, dtype=torch.uint8))


def test_a_wait_that_gives_up_is_reported(kda):
    """The tensor-core kernel's waits are bounded: a forced give-up sets the status word, is counted,
    and leaves the context usable."""
    x = [dev(t) for t in inputs(3, 1, 700, 4, 4, 128, 128, BF, 1)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kda.kda_fused_wait_timeouts(reset=True)
    try:
        for chunk in (0, 1, 3):  # (a segment here has four)
            kda.kda_test_hooks(wait_timeout_chunk=chunk)
            status.zero_()
            kda.kda_decay_chunk_fwd(*x[:4], initial_state=x[4], output_final_state=True, status=status)
            torch.cuda.synchronize()
            assert int(status) == 1
            assert kda.kda_fused_wait_timeouts(reset=True) > 0
    finally:
        kda.kda_test_hooks()
    status.zero_()
    check(kda, "kda_decay_chunk_fwd", inputs(3, 1, 700, 4, 4, 128, 128, BF, 1))
    assert int(status) == 0 and kda.kda_fused_wait_timeouts() == 0
