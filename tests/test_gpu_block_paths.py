"""Schedules of decayed attention that small calls do not take, against float64: packed sequences in time
segments, more sequences than are ranked by length, heads of 256 in two halves, and the precision of a state
over one and many chunks.  Bounds as in test_gpu_block."""
import functools

import pytest
import torch

import block_reference as ref
from block_reference import F32, HALF
from test_gpu_block import BF, check, close, dev, inputs, kda  # noqa: F401

pytestmark = pytest.mark.gpu

EDGES = {
    "long": [0, 0, 1500, 1500, 1501, 4000],  # segments; empty sequences first and between, one of one token
    "ends": [0, 1024, 1024, 2048, 2049, 3000, 3000],  # sequences that end with a segment, an empty one last
    "many": sorted([0, 900] + [(37 * i) % 900 for i in range(199)] + [450] * 3),  # 203 sequences, some empty
}


@functools.lru_cache(maxsize=None)
def case(name, K, V, H, Hk, dtype, T=None):
    edges = EDGES[name]
    x = inputs(K + V, 1, edges[-1] + 37, H, Hk, K, V, dtype, len(edges) - 1, span=0.3)
    return edges, x, ref.decay_attention(*x, edges)


@pytest.mark.parametrize("name,H,Hk", [("long", 2, 2), ("ends", 2, 1), ("many", 3, 3)])
@pytest.mark.parametrize("K,V", [(128, 128), (64, 64), (256, 128), (128, 256), (256, 256), (96, 40)])
@pytest.mark.parametrize("o_dtype", [BF, torch.float32])
@pytest.mark.parametrize("inplace", [False, True])
def test_packed(kda, name, H, Hk, K, V, o_dtype, inplace):  # noqa: F811
    """Rows behind the last offset are NaN on the way in and untouched on the way out."""
    edges, x, (o_ref, S_ref, oa, Sa) = case(name, K, V, H, Hk, BF)
    n = edges[-1]
    q, k, v, decay = (t.clone() for t in x[:4])
    for t in (q, k, v, decay):
        t[:, n:] = float("nan")
    s = dev(x[4])
    o = torch.full(v.shape, 7.0, dtype=o_dtype, device="cuda")
    cu = torch.tensor(edges, dtype=torch.int32, device="cuda")
    before = kda.kda_fused_wait_timeouts()
    _, S = kda.kda_decay_chunk_fwd(dev(q), dev(k), dev(v), dev(decay), initial_state=s, output_final_state=True,
                                   final_state=s if inplace else None, cu_seqlens=cu, o=o)
    torch.cuda.synchronize()
    assert (S is s) == inplace and kda.kda_fused_wait_timeouts() == before
    longest = max(b - a for a, b in zip(edges, edges[1:]))
    f32 = (K + 128 + longest) * F32
    operand = HALF[BF] * (1 + 2.0 ** -6)
    close(o[:, :n], o_ref[:, :n], HALF[o_dtype] * o_ref.abs()[:, :n] + (operand + f32) * oa[:, :n] + 1e-30, "o")
    assert bool((o[:, n:] == 7.0).all())
    close(S, S_ref, f32 * Sa + 1e-30, "state")
    assert (o[:, :n].double().cpu() - o_ref[:, :n]).norm() <= HALF[BF] * o_ref[:, :n].norm()
    for i, (a, b) in enumerate(zip(edges, edges[1:])):
        if a == b:
            assert torch.equal(S[i].cpu(), x[4][i])


@pytest.mark.parametrize("edges", [[0, 0, 1, 1, 70, 200], [0, 130, 130], [0, 0, 0]])
@pytest.mark.parametrize("V", [64, 256])
@pytest.mark.parametrize("o_dtype", [None, torch.float32])
def test_heads_of_256_packed(kda, edges, V, o_dtype):  # noqa: F811
    x = inputs(V, 1, edges[-1], 2, 1, 256, V, BF, len(edges) - 1)
    check(kda, "kda_decay_chunk_fwd", x, edges, o_dtype=o_dtype, inplace=True)


@pytest.mark.parametrize("T", [0, 1, 64, 65, 1100])
@pytest.mark.parametrize("o_dtype", [None, torch.float32])
def test_heads_of_256_dense(kda, T, o_dtype):  # noqa: F811
    x = inputs(T, 1, T, 2, 2, 256, 256, BF, 1, span=0.3)
    o, S = check(kda, "kda_decay_chunk_fwd", x, o_dtype=o_dtype, inplace=True)
    if T == 0:
        assert torch.equal(S.cpu(), x[4])


@pytest.mark.parametrize("K,V", [(64, 64), (64, 128), (128, 64), (64, 256), (256, 64)])
@pytest.mark.parametrize("B,T", [(1, 1100), (2, 777)])
def test_segments_of_other_heads(kda, K, V, B, T):  # noqa: F811
    check(kda, "kda_decay_chunk_fwd", inputs(T, B, T, 2, 2, K, V, BF, B, fixed=True), inplace=True)


# A float32 state out of bf16 inputs.  Each of a chunk's twelve accumulations (four of 16 tokens for each of the three
# bf16 terms of a scaled value) cuts at most one unit of the last place, 2^-23 of the sum; the value's factor and
# its three terms are good to 8 u.  With inputs of one sign the sum of absolute values is the sum itself.
def state_bound(tokens):
    return 12 * -(-tokens // 64) * 2 * F32 + 8 * F32


@pytest.mark.parametrize("K", [64, 128, 256])
@pytest.mark.parametrize("T,rate", [(64, 0.01), (64, 0.3), (64, 0.0), (63, 0.05), (4096, 0.0), (4096, 0.002), (2500, 0.0)])
def test_a_state_of_one_sign(kda, K, T, rate):  # noqa: F811
    """Whole sequences (a pretended count of one multiprocessor): one chunk shows the values' 24 bits (without the
    third term a state would be off by 2^-17 in the mean), many chunks the accumulation's lean towards zero."""
    q, k, v, decay, _ = inputs(T, 1, T, 2, 2, K, 64, BF, 1, fixed=True, state=False)
    decay.copy_(torch.tensor([-rate, -1.1 * rate]))
    k, v = k.abs(), v.abs()
    S_ref = torch.zeros(1, 2, K, 64, dtype=torch.float64)
    for t in range(T):
        S_ref = decay.double().exp()[None, :, None, None] * S_ref + k[:, t].double()[..., None] * v[:, t].double()[:, :, None, :]
    try:
        kda.kda_test_hooks(sm_count=1)
        _, S = kda.kda_decay_chunk_fwd(dev(q), dev(k), dev(v), dev(decay), output_final_state=True)
    finally:
        kda.kda_test_hooks()
    memory = T if rate == 0 else min(T, 1 / rate + 64)  # (a cut fades as the state does)
    # expf of a decay and its sum's 2^-25 unit: a relative step for each token of the memory
    steps = memory * 2 * F32 if rate else 0.0
    close(S, S_ref, (state_bound(memory) + steps) * S_ref.abs() + 1e-30, "state")


@pytest.mark.parametrize("post,pre,scale,residual", [(False, True, False, True), (True, False, True, True),
                                                     (False, False, True, False), (True, True, True, False)])
@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_parts_of_the_block_norm_of_many_long_rows(kda, post, pre, scale, residual, dtype):  # noqa: F811
    g = torch.Generator().manual_seed(8)
    rows, D = 1500, 8192
    x = (0.5 * torch.randn(rows, D, generator=g)).to(dtype)
    r = torch.randn(rows, D, generator=g) if residual else None
    wp, wn, c = (torch.rand(D, generator=g) + 0.5 if on else None for on in (post, pre, scale))
    wh, wy = ref.block_norm(x, r, wp, None, 0, 0.7, c, wn, 1e-6)
    h, y = kda.kda_block_norm_fwd(dev(x), dev(r), dev(wp), None, dev(wn), scale=0.7, channel_scale=dev(c), eps=1e-6)
    n = (D // 8 + 24 + 24) * F32
    size = wh.abs() + (0 if r is None else 2 * r.double().abs())
    close(h, wh, HALF[h.dtype] * wh.abs() + n * size + 1e-30, "h")
    rel = size / wh.abs().clamp_min(1e-300)
    mean = (size.square().mean(-1, keepdim=True) / (wh.square().mean(-1, keepdim=True) + 1e-6)).sqrt()
    close(y, wy, (HALF[dtype] + n * (rel + mean)) * wy.abs() + 1e-30, "y")


@pytest.mark.parametrize("name,H,Hk", [("long", 2, 2), ("ends", 2, 1), ("many", 3, 3)])
@pytest.mark.parametrize("K,V", [(128, 128), (40, 72)])
@pytest.mark.parametrize("state", ["none", "given", "in place"])
def test_packed_float32(kda, name, H, Hk, K, V, state):  # noqa: F811
    """The FP32 chunks: first chunks read the initial state, last ones make the final state, also in its place."""
    edges, x, want = case(name, K, V, H, Hk, torch.float32)
    if state == "none":
        want = ref.decay_attention(*x[:4], None, edges)
    o_ref, S_ref, oa, Sa = want
    n = edges[-1]
    q, k, v, decay = (t.clone() for t in x[:4])
    for t in (q, k, v, decay):
        t[:, n:] = float("nan")
    s = None if state == "none" else dev(x[4])
    cu = torch.tensor(edges, dtype=torch.int32, device="cuda")
    args = dict(initial_state=s, output_final_state=True, final_state=s if state == "in place" else None, cu_seqlens=cu)
    o, S = kda.kda_decay_chunk_fwd(dev(q), dev(k), dev(v), dev(decay), **args)
    torch.cuda.synchronize()
    longest = max(b - a for a, b in zip(edges, edges[1:]))
    f32 = (K + 128 + longest) * F32
    close(o[:, :n], o_ref[:, :n], f32 * oa[:, :n] + 1e-30, "o")
    close(S, S_ref, f32 * Sa + 1e-30, "state")
    if state == "given":
        again = kda.kda_decay_chunk_fwd(dev(q), dev(k), dev(v), dev(decay), **(args | dict(output_final_state=False)))
        assert torch.equal(again[0][:, :n], o[:, :n])


@pytest.mark.parametrize("B,T,H", [(2, 65, 2), (3, 300, 1), (1, 1000, 2)])
@pytest.mark.parametrize("inplace", [False, True])
def test_dense_float32(kda, B, T, H, inplace):  # noqa: F811
    check(kda, "kda_decay_chunk_fwd", inputs(T, B, T, H, 1, 96, 130, torch.float32, B, span=0.3), inplace=inplace)


@pytest.mark.parametrize("K,V,o_dtype", [(64, 64, None), (64, 128, None), (128, 64, None), (128, 128, None), (64, 128, torch.float32),
                                         (128, 128, torch.float32), (256, 256, None)])
@pytest.mark.parametrize("B,T,H", [(2, 1081, 8), (1, 1400, 6), (3, 200, 60)])
def test_the_same_bits_from_cold_caches(kda, K, V, o_dtype, B, T, H):  # noqa: F811
    """Loads that take their time, which shows a product that does not wait for its operand: segments, whole and
    cut sequences, every result the same as the first."""
    x = [dev(t) for t in inputs(T, B, T, H, H, K, V, BF, B, span=0.3)]
    first, cold = None, torch.empty(1 << 26, device="cuda")
    for i in range(40):
        cold.fill_(i)  # (256 MB, twice the L2)
        got = kda.kda_decay_chunk_fwd(*x[:4], initial_state=x[4], output_final_state=True, o_dtype=o_dtype)
        first = first or got
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1]), i
    o_ref, S_ref, oa, Sa = ref.decay_attention(*(t[:1, :, :2].cpu() for t in x[:4]), x[4][:1, :2].cpu())
    f32 = (K + 128 + T) * F32
    operand = HALF[BF] * (1 + 2.0 ** -6) if o_dtype is None else 0.0
    o, S = first
    close(o[:1, :, :2], o_ref, HALF[o.dtype] * o_ref.abs() + (operand + f32) * oa + 1e-30, "o")
    close(S[:1, :2], S_ref, f32 * Sa + 1e-30, "state")
