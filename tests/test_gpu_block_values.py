"""Decayed attention on values at the edge of its types, against float64: what is not finite stays behind
its token and in its channel, large states do not overflow before float32 does.

Bounds as in test_gpu_block (u = 2^-24, w = 2^-8).
"""
import pytest
import torch

import block_reference as ref
from block_reference import F32, HALF
from test_gpu_block import BF, check, close, dev, inputs, kda  # noqa: F401

pytestmark = pytest.mark.gpu
FORMS = ["kda_decay_chunk_fwd", "kda_decay_recurrent_fwd"]


def compare_elsewhere(fn, x, o, S, spoiled_o, spoiled_S):
    """o and S against the reference of x (whose values are all finite) but for the places that are
    marked, and those are not finite."""
    q, k, v, decay, S0 = x
    o_ref, S_ref, oa, Sa = ref.decay_attention(q, k, v, decay, S0)
    f32 = (q.shape[3] + 128 + q.shape[1]) * F32
    operand = HALF[BF] * (1 + 2.0 ** -6) if "chunk" in fn and q.dtype == BF else 0.0
    assert not torch.isfinite(o.cpu()[spoiled_o]).any() and not torch.isfinite(S.cpu()[spoiled_S]).any()
    o, S = o.double().cpu(), S.double().cpu()
    o[spoiled_o], S[spoiled_S] = o_ref[spoiled_o], S_ref[spoiled_S]
    half = HALF[BF] if q.dtype == BF else F32
    close(o, o_ref, half * o_ref.abs() + (operand + f32) * oa + 1e-30, "o")
    close(S, S_ref, f32 * Sa + 1e-30, "state")


@pytest.mark.parametrize("fn", FORMS)
@pytest.mark.parametrize("dtype,o_dtype", [(torch.float32, None), (BF, None), (BF, torch.float32)])
@pytest.mark.parametrize("K,V", [(128, 128), (64, 64), (128, 64), (256, 256), (40, 72)])
@pytest.mark.parametrize("T,at", [(200, 0), (200, 37), (200, 64), (200, 199), (700, 300)])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_a_value_that_is_not_finite(kda, fn, dtype, o_dtype, K, V, T, at, bad):  # noqa: F811
    """One element of v: outputs before its token, of other channels and of other heads stay right."""
    q, k, v, decay, S0 = x = inputs(T + at, 1, T, 2, 2, K, V, dtype, 1, span=0.1)
    d = (7 * at + 3) % V
    v[0, at, 1, d] = 0
    bad_v = v.clone()
    bad_v[0, at, 1, d] = bad
    o, S = getattr(kda, fn)(dev(q), dev(k), dev(bad_v), dev(decay), initial_state=dev(S0), output_final_state=True,
                            o_dtype=o_dtype)
    so, sS = torch.zeros(o.shape, dtype=torch.bool), torch.zeros(S.shape, dtype=torch.bool)
    so[0, at:, 1, d], sS[0, 1, :, d] = True, True
    compare_elsewhere(fn, x, o, S, so, sS)


@pytest.mark.parametrize("fn", FORMS)
@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("K,V", [(128, 128), (256, 64), (40, 72)])
@pytest.mark.parametrize("T,at", [(200, 0), (200, 1), (200, 37), (200, 64), (200, 199), (700, 300)])
def test_a_decay_that_is_no_number(kda, fn, dtype, K, V, T, at):  # noqa: F811
    """Outputs before its token and of other heads stay right."""
    q, k, v, decay, S0 = x = inputs(T + at, 1, T, 2, 2, K, V, dtype, 1, span=0.1)
    bad = decay.clone()
    bad[0, at, 1] = float("nan")
    o, S = getattr(kda, fn)(dev(q), dev(k), dev(v), dev(bad), initial_state=dev(S0), output_final_state=True)
    so, sS = torch.zeros(o.shape, dtype=torch.bool), torch.zeros(S.shape, dtype=torch.bool)
    so[0, at:, 1], sS[0, 1] = True, True
    compare_elsewhere(fn, x, o, S, so, sS)


@pytest.mark.parametrize("fn", FORMS)
@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("K", [128, 256])
@pytest.mark.parametrize("power", [-70, 100, 110])
@pytest.mark.parametrize("rate", [0.0125, 0.1])
def test_large_and_small_values(kda, fn, dtype, K, power, rate):  # noqa: F811
    """States and values far from 1 under decays that add up over many chunks, in one whole sequence."""
    q, k, v, decay, S0 = inputs(power, 1, 2200, 1, 1, K, 64, dtype, 1, fixed=True)
    decay.fill_(-rate)
    try:
        kda.kda_test_hooks(sm_count=1)
        check(kda, fn, (q, k, v * 2.0 ** power, decay, S0 * 2.0 ** power), chunked="chunk" in fn)
    finally:
        kda.kda_test_hooks()


@pytest.mark.parametrize("fn", FORMS)
@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("K,V", [(128, 128), (64, 64), (128, 64), (256, 256), (40, 72)])
@pytest.mark.parametrize("T,at", [(200, 0), (200, 37), (200, 199), (700, 300)])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_a_state_of_a_value_that_is_not_finite(kda, fn, dtype, K, V, T, at, bad):  # noqa: F811
    """An infinite value makes an infinite state, with its key's signs; other channels have nothing of it."""
    q, k, v, decay, S0 = inputs(T + at, 1, T, 2, 2, K, V, dtype, 1, span=0.1)
    d = (7 * at + 3) % V
    v[0, at, 1, d] = 0
    k[0, at, 1] = torch.where(k[0, at, 1] == 0, torch.ones((), dtype=dtype), k[0, at, 1])  # (0 x inf is no number)
    _, S_ref, _, Sa = ref.decay_attention(q, k, v, decay, S0)
    v[0, at, 1, d] = bad
    _, S = getattr(kda, fn)(dev(q), dev(k), dev(v), dev(decay), initial_state=dev(S0), output_final_state=True)
    S = S.double().cpu()
    want = torch.sign(k[0, at, 1].double()) * bad
    assert torch.equal(S[0, 1, :, d].nan_to_num(nan=5.0), want.nan_to_num(nan=5.0))
    S[0, 1, :, d] = S_ref[0, 1, :, d]
    close(S, S_ref, (K + 128 + T) * F32 * Sa + 1e-30, "state")


SHAPES = [(1, 200, 2, 2, 128, 128), (2, 150, 4, 2, 64, 64), (1, 130, 2, 1, 64, 128), (1, 321, 3, 3, 128, 64), (1, 1100, 2, 2, 128, 128),
          (1, 777, 1, 1, 256, 256), (2, 190, 2, 2, 64, 256), (1, 2100, 1, 1, 64, 64), (1, 63, 1, 1, 256, 64), (1, 1, 2, 2, 128, 128)]


@pytest.mark.parametrize("B,T,H,Hk,K,V", SHAPES)
@pytest.mark.parametrize("span", [0.0, 0.1, 3.0])
@pytest.mark.parametrize("state", [False, True])
def test_a_float32_output_of_bf16_inputs(kda, B, T, H, Hk, K, V, span, state):  # noqa: F811
    """No operand of its sums is rounded to bf16: the bounds of float32 arithmetic alone, for whole sequences and
    for segments, whole units and cut ones."""
    x = inputs(T + K, B, T, H, Hk, K, V, BF, B, span=span, state=state)
    o_ref, S_ref, oa, Sa = ref.decay_attention(*x)
    for sms in (0, 1, 3):
        try:
            kda.kda_test_hooks(sm_count=sms)
            o, S = kda.kda_decay_chunk_fwd(*(dev(t) for t in x[:4]), initial_state=dev(x[4]), output_final_state=True,
                                           o_dtype=torch.float32)
        finally:
            kda.kda_test_hooks()
        f32 = (K + 128 + T) * F32
        close(o, o_ref, f32 * oa + 1e-30, "o")
        close(S, S_ref, f32 * Sa + 1e-30, "state")


def test_a_float32_output_packed(kda):  # noqa: F811
    edges = [0, 0, 1, 1, 70, 200, 264, 900]
    x = inputs(4, 1, edges[-1], 2, 1, 128, 128, BF, len(edges) - 1, span=0.5)
    o_ref, S_ref, oa, Sa = ref.decay_attention(*x, edges)
    cu = torch.tensor(edges, dtype=torch.int32, device="cuda")
    s = dev(x[4])
    o, S = kda.kda_decay_chunk_fwd(*(dev(t) for t in x[:4]), initial_state=s, final_state=s, cu_seqlens=cu, o_dtype=torch.float32)
    f32 = (128 + 128 + 636) * F32
    close(o, o_ref, f32 * oa + 1e-30, "o")
    close(S, S_ref, f32 * Sa + 1e-30, "state")


@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("rate", [1e-6, 3.3e-6, 1e-5, 1e-4, 0.002])
@pytest.mark.parametrize("one_sign", [True, False])
def test_slow_decays_over_long_sequences(kda, dtype, rate, one_sign):  # noqa: F811
    """A decay that all tokens share: what each token's is off by adds up.  The state's bound: a chunk's sum of 64
    products (bf16: twelve cuts of 2^-23), one rounded addition for each chunk (bf16: each segment) behind it, the decays'
    own 2^-33 a token, a few u for the factors and, for each multiplication by a chunk's (a segment's) decay, two u."""
    T, H, K = 32768, 2, 64
    g = torch.Generator(device="cuda").manual_seed(int(rate * 1e7))
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    q, k = (torch.nn.functional.normalize(r(1, T, H, K), dim=-1).to(dtype) for _ in range(2))
    v = r(1, T, H, K).to(dtype)
    if one_sign:
        k, v = k.abs(), v.abs()
    a = torch.full((H,), -rate, device="cuda")
    w = torch.exp(a[0].double() * torch.arange(T - 1, -1, -1, device="cuda"))
    want = torch.einsum("t,thk,thv->hkv", w, k[0].double(), v[0].double())[None]
    size = torch.einsum("t,thk,thv->hkv", w, k[0].double().abs(), v[0].double().abs())[None]
    _, S = kda.kda_decay_chunk_fwd(q, k, v, a, output_final_state=True)
    # (152 multiprocessors: two heads in segments of seven chunks; planned for fewer, the segments are longer)
    chunks = T // 64
    steps = chunks if dtype == torch.float32 else 76
    inside = 66 * F32 if dtype == torch.float32 else 7 * 12 * 2 * F32
    bound = inside + 4 * steps * F32 + T * 2.0 ** -33 + 16 * F32
    close(S, want.cpu(), (bound * size).cpu(), "state")


@pytest.mark.parametrize("rate", [0.0, 1e-6, 1e-4, 0.0023])
@pytest.mark.parametrize("one_sign", [True, False])
def test_the_documented_lean_of_a_state(kda, rate, one_sign):  # noqa: F811
    """Whole bf16 sequences: a chunk's twelve accumulations cut at most 2^-23 each of the sum of the absolute values,
    for each 64 tokens of the memory; the decays' own 2^-33 a token; a few u for the factors."""
    T, H, K = 32768, 2, 128
    g = torch.Generator(device="cuda").manual_seed(int(rate * 1e7) + 1)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    q, k = (torch.nn.functional.normalize(r(1, T, H, K), dim=-1).to(BF) for _ in range(2))
    v = r(1, T, H, 64).to(BF)
    if one_sign:
        k, v = k.abs(), v.abs()
    a = torch.full((H,), -rate, device="cuda")
    w = torch.exp(a[0].double() * torch.arange(T - 1, -1, -1, device="cuda"))
    want = torch.einsum("t,thk,thv->hkv", w, k[0].double(), v[0].double())[None]
    size = torch.einsum("t,thk,thv->hkv", w, k[0].double().abs(), v[0].double().abs())[None]
    try:
        kda.kda_test_hooks(sm_count=1)
        _, S = kda.kda_decay_chunk_fwd(q, k, v, a, output_final_state=True)
    finally:
        kda.kda_test_hooks()
    memory = min(T, 1 / rate) if rate else T
    close(S, want.cpu(), ((12 * 2.0 ** -23 * (memory / 64 + 1) + T * 2.0 ** -33 + 16 * F32) * size).cpu(), "state")


@pytest.mark.parametrize("fn", FORMS)
@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("K", [96, 128])
@pytest.mark.parametrize("lo,hi", [(129, 130), (1, 130), (3, 93)])
def test_tokens_out_of_a_batch_with_few_heads(kda, fn, dtype, K, lo, hi):  # noqa: F811
    """Slices of one sequence are contiguous as they are; two heads' decays then lie at multiples of 8 bytes."""
    x = inputs(hi, 1, 130, 2, 2, K, K, dtype, 1)
    q, k, v, decay = (dev(t)[:, lo:hi] for t in x[:4])
    assert decay.is_contiguous() and decay.data_ptr() % 16 == 8
    o, S = getattr(kda, fn)(q, k, v, decay, initial_state=dev(x[4]), output_final_state=True)
    same = getattr(kda, fn)(q, k, v, decay.clone(), initial_state=dev(x[4]), output_final_state=True)
    assert torch.equal(o, same[0]) and torch.equal(S, same[1])
    o_ref, S_ref, oa, Sa = ref.decay_attention(*(t[:, lo:hi] for t in x[:4]), x[4])
    close(S, S_ref, (K + 128 + 130) * F32 * Sa + 1e-30, "state")


@pytest.mark.parametrize("o_dtype", [None, torch.float32])
@pytest.mark.parametrize("sms", [0, 1])
def test_a_wait_that_gives_up_among_values_that_are_not_finite(kda, o_dtype, sms):  # noqa: F811
    """A forced give-up while tiles are being cleared, with either output: reported, and the next call is right."""
    x = inputs(3, 1, 700, 4, 4, 128, 128, BF, 1)
    bad = x[2].clone()
    bad[0, ::50, :, ::7] = float("nan")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kda.kda_fused_wait_timeouts(reset=True)
    try:
        for chunk in (0, 1, 3):
            kda.kda_test_hooks(wait_timeout_chunk=chunk, sm_count=sms)
            status.zero_()
            kda.kda_decay_chunk_fwd(dev(x[0]), dev(x[1]), dev(bad), dev(x[3]), initial_state=dev(x[4]),
                                    output_final_state=True, status=status, o_dtype=o_dtype)
            torch.cuda.synchronize()
            assert int(status) == 1 and kda.kda_fused_wait_timeouts(reset=True) > 0
    finally:
        kda.kda_test_hooks()
    check(kda, "kda_decay_chunk_fwd", x, o_dtype=o_dtype)
    assert kda.kda_fused_wait_timeouts() == 0


@pytest.mark.parametrize("rate", [0.0, 1e-6, 1e-4, 0.0023, 0.3])
@pytest.mark.parametrize("one_sign", [True, False])
@pytest.mark.parametrize("K", [64, 128, 256])
@pytest.mark.parametrize("T", [64, 4096, 32768])
def test_a_state_does_not_lean_with_its_memory(kda, rate, one_sign, K, T):  # noqa: F811
    """Whole bf16 sequences: a chunk's twelve accumulations cut at most 2^-23 each of that chunk's own sum, a rounded
    addition for each chunk of the memory, the decays' own 2^-33 a token, a few u for the factors (those of the
    scaled sums: 2^-24 in the exponent)."""
    H = 2
    g = torch.Generator(device="cuda").manual_seed(int(rate * 1e7) + K)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    q, k = (torch.nn.functional.normalize(r(1, T, H, K), dim=-1).to(BF) for _ in range(2))
    v = r(1, T, H, 64).to(BF)
    if one_sign:
        k, v = k.abs(), v.abs()
    a = torch.full((H,), -rate, device="cuda")
    w = torch.exp(a[0].double() * torch.arange(T - 1, -1, -1, device="cuda"))
    want = torch.einsum("t,thk,thv->hkv", w, k[0].double(), v[0].double())[None]
    size = torch.einsum("t,thk,thv->hkv", w, k[0].double().abs(), v[0].double().abs())[None]
    try:
        kda.kda_test_hooks(sm_count=1)
        _, S = kda.kda_decay_chunk_fwd(q, k, v, a, output_final_state=True)
    finally:
        kda.kda_test_hooks()
    memory = min(T, 1 / rate) if rate else T
    bound = 12 * 2.0 ** -23 + (memory / 64 + 1) * F32 + T * 2.0 ** -33 + 16 * F32
    close(S, want.cpu(), (bound * size).cpu(), "state")
    # random roundings: their 2-norm is as float32 sums have it, whatever the memory
    if not one_sign:
        assert (S.double() - want).norm() <= (1e-6 + T * 2.0 ** -33) * want.norm()
