"""The gated delta rule with one decay a head against the float64 recurrence.

Tolerances.  Keys are rows of norm 1 and beta is in [0, 1], so the rule's transition contracts: an error made in
one token does not grow.  In float32 an output, and a state's element, is a sum over at most K channels, the
chunk's tokens in the inverse, in U and in P U (64 each) and a chunk's addition (64), each term rounded: in the norm
at most (K + 256) 2^-24.  A bf16 output is rounded once more (2^-8 of itself); where it is formed on the tensor
cores from bf16 inputs the state that the queries read is rounded to bf16 (2^-8 of |q| |S|) and the operands of the
chunk's own part to tf32, cut and not rounded (2 x 2^-10 of the sum of its terms' absolute values)."""
import pytest
import torch

from delta_reference import F32, HALF, delta, gate

pytestmark = pytest.mark.gpu

kda = pytest.importorskip("chunked_kda_gb300")
DEV = "cuda"


def make(B, T, H, K, V, dtype, Hk=None, seed=0, raw=False, edges=None, state=True, slow=False):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    Hk = Hk or H
    q, k = (torch.nn.functional.silu(r(B, T, Hk, K)) for _ in range(2))
    if not raw:
        q, k = (x / x.norm(dim=-1, keepdim=True).clamp_min(1e-6) for x in (q, k))
    x = dict(q=q.to(dtype), k=k.to(dtype), v=r(B, T, H, V).to(dtype))
    N = B if edges is None else len(edges) - 1
    if raw:
        x |= dict(g=r(B, T, H).to(dtype), beta=r(B, T, H).to(dtype), A_log=torch.log(1 + 15 * torch.rand(H, generator=gen)),
                  dt_bias=r(H) - 3)
    else:
        x |= dict(g=-(1e-3 if slow else 0.3) * torch.rand(B, T, H, generator=gen), beta=torch.sigmoid(r(B, T, H)).to(dtype))
    x["S0"] = 0.1 * r(N, H, K, V) if state else None
    return x


def reference(x, raw=False, edges=None):
    a = gate(x["g"], x.get("A_log"), x.get("dt_bias"))
    b = torch.sigmoid(x["beta"].double()) if raw else x["beta"]
    return delta(x["q"], x["k"], x["v"], a, b, x["S0"], edges, raw, raw)


def call(fn, x, raw=False, edges=None, **kw):
    d = {n: None if t is None else t.to(DEV) for n, t in x.items()}
    if raw:
        kw |= dict(A_log=d["A_log"], dt_bias=d["dt_bias"], mode=kda.GATE_NONSAFE,
                   flags=kda.FLAG_Q_L2NORM | kda.FLAG_K_L2NORM | kda.FLAG_BETA_LOGITS)
    if edges is not None:
        kw["cu_seqlens"] = torch.tensor(edges, dtype=torch.int32, device=DEV)
    kw = dict(initial_state=d["S0"], output_final_state=True) | kw
    o, S = fn(d["q"], d["k"], d["v"], d["g"], d["beta"], **kw)
    torch.cuda.synchronize()
    return o, S


def check(got, want, dtype, K, o_dtype=None, rows=None):
    (o, S), (ro, rS, inter, intra) = got, want
    o_dtype = o_dtype or dtype
    assert o.dtype == o_dtype and S.dtype == torch.float32
    tol = (K + 256) * F32
    o, S = o.double().cpu(), S.double().cpu()
    if rows is not None:
        o, ro, inter, intra = (t[:, :rows] for t in (o, ro, inter, intra))
    if o_dtype == torch.float32:
        assert (o - ro).norm() <= tol * ro.norm() + 1e-30
    else:
        bound = 2 ** -8 * ro.abs() + 1.01 * (2 ** -8 * inter + 2 ** -9 * intra) + tol * ro.norm() / max(1, ro.numel()) ** 0.5 * 8
        assert ((o - ro).abs() <= bound).all(), ((o - ro).abs() / bound).max()
        assert (o - ro).norm() <= 3.5e-3 * ro.norm()  # two rounded parts, each spread over its half step: 2^-8 sqrt(2 / 3)
    assert (S - rS).norm() <= tol * rS.norm() + 1e-30


SHAPES = [(1, 1, 1, 64, 64), (2, 63, 2, 128, 128), (1, 64, 3, 128, 128), (1, 65, 2, 128, 64), (2, 200, 2, 128, 128),
          (1, 130, 2, 96, 96), (1, 70, 2, 128, 256), (1, 129, 1, 64, 128), (1, 100, 2, 17, 33), (1, 90, 1, 256, 72),
          (3, 2, 2, 40, 8), (1, 300, 1, 1, 1), (1, 150, 2, 8, 200)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,T,H,K,V", SHAPES)
@pytest.mark.parametrize("form", ["chunk", "recurrent"])
def test_against_float64(form, dtype, B, T, H, K, V):
    x = make(B, T, H, K, V, dtype, seed=T)
    fn = kda.kda_delta_chunk_fwd if form == "chunk" else kda.kda_delta_recurrent_fwd
    check(call(fn, x), reference(x), dtype, K)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("form", ["chunk", "recurrent"])
@pytest.mark.parametrize("K,V", [(128, 128), (64, 48), (36, 36)])
def test_raw_inputs_and_shared_heads(form, dtype, K, V):
    x = make(2, 140, 6, K, V, dtype, Hk=2, raw=True, seed=5)
    fn = kda.kda_delta_chunk_fwd if form == "chunk" else kda.kda_delta_recurrent_fwd
    check(call(fn, x, raw=True), reference(x, raw=True), dtype, K)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("form", ["chunk", "recurrent"])
def test_packed_sequences(form, dtype):
    edges = [0, 0, 1, 66, 66, 130, 194, 323, 323]  # empty first, in the middle and last; whole chunks and parts
    x = make(1, 340, 3, 128, 128, dtype, Hk=1, edges=edges, seed=7)
    want = reference(x, edges=edges)
    fn = kda.kda_delta_chunk_fwd if form == "chunk" else kda.kda_delta_recurrent_fwd
    for name in "qkv":  # rows behind the last sequence are not read into anything, and not written
        x[name][:, 323:] = float("nan")
    o = torch.full((1, 340, 3, 128), 7.0, dtype=dtype, device=DEV)
    got = call(fn, x, edges=edges, o=o)
    check(got, want, dtype, 128, rows=323)
    assert (o[:, 323:] == 7).all()
    for n in (0, 3, 7):
        assert torch.equal(got[1][n].cpu(), x["S0"][n])


@pytest.mark.parametrize("form", ["chunk", "recurrent"])
@pytest.mark.parametrize("K,V", [(128, 128), (40, 72)])
def test_float32_output_of_bf16_inputs(form, K, V):
    x = make(1, 150, 2, K, V, torch.bfloat16, seed=9)
    fn = kda.kda_delta_chunk_fwd if form == "chunk" else kda.kda_delta_recurrent_fwd
    check(call(fn, x, o_dtype=torch.float32), reference(x), torch.bfloat16, K, torch.float32)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("form", ["chunk", "recurrent"])
def test_float32_gates_and_options(form, dtype):
    x = make(1, 100, 2, 128, 128, dtype, seed=11, state=False)
    x["beta"] = x["beta"].float()
    x["g"] = x["g"].bfloat16()
    fn = kda.kda_delta_chunk_fwd if form == "chunk" else kda.kda_delta_recurrent_fwd
    o, S = call(fn, x, output_final_state=False)
    assert S is None
    check((o, call(fn, x)[1]), reference(x), dtype, 128)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("form", ["chunk", "recurrent"])
def test_decays_from_none_to_all(form, dtype):
    x = make(1, 200, 3, 128, 128, dtype, seed=13)
    x["g"][:, :, 0] = 0
    x["g"][:, 70, 1] = -float("inf")
    x["g"][:, 71, 1] = -2000.0
    x["g"][:, 128, 1] = -float("inf")
    x["g"][:, :, 2] *= 200
    x["beta"][:, 30:60] = 0
    x["beta"][:, 60:64] = 1
    fn = kda.kda_delta_chunk_fwd if form == "chunk" else kda.kda_delta_recurrent_fwd
    check(call(fn, x), reference(x), dtype, 128)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_one_key_again_and_again(dtype):
    """beta = 1 and one key: each value takes the last one's place; the inverse has long chains."""
    x = make(1, 200, 2, 128, 128, dtype, seed=15)
    x["k"][:] = x["k"][:, :1]
    x["beta"][:] = 1
    x["g"][:] = 0
    k = x["k"][0, 0].double()
    assert (k.norm(dim=-1) - 1).abs().max() < 4e-3
    check(call(kda.kda_delta_chunk_fwd, x), reference(x), dtype, 128)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_parts_carry_the_state_on(dtype):
    x = make(2, 257, 2, 128, 128, dtype, seed=17)
    want = reference(x)
    parts, S = [], x["S0"].to(DEV)
    for lo, hi, fn in ((0, 100, kda.kda_delta_chunk_fwd), (100, 256, kda.kda_delta_chunk_fwd),
                       (256, 257, kda.kda_delta_recurrent_fwd)):
        part = {n: x[n][:, lo:hi].contiguous() for n in ("q", "k", "v", "g", "beta")} | {"S0": None}
        o, S1 = call(fn, part, initial_state=S, final_state=S)  # in place
        assert S1 is S
        parts.append(o)
    check((torch.cat(parts, 1), S), want, dtype, 128)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("form", ["chunk", "recurrent"])
@pytest.mark.parametrize("what", ["v", "k", "g", "beta", "q"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_what_is_not_finite_does_not_reach_back(form, dtype, what, bad):
    x = make(1, 150, 2, 128, 128, dtype, seed=19)
    fn = kda.kda_delta_chunk_fwd if form == "chunk" else kda.kda_delta_recurrent_fwd
    clean = call(fn, x)[0]
    t = 70
    x[what][0, t, 1] = bad if what in ("g", "beta") else x[what][0, t, 1]
    if what in "qkv":
        x[what][0, t, 1, 3] = bad
    o, S = call(fn, x)
    assert torch.equal(o[:, :, 0], clean[:, :, 0])
    assert torch.equal(o[:, :t], clean[:, :t])
    if what == "q":
        assert torch.equal(o[:, t + 1:], clean[:, t + 1:]) and torch.isfinite(S).all()
        assert not torch.isfinite(o[0, t, 1]).any()
    elif what == "v":
        others = [c for c in range(128) if c != 3]
        assert torch.equal(o[..., others], clean[..., others])
        assert not torch.isfinite(o[0, t, 1, 3])
        assert not torch.isfinite(S[0, 1, :, 3]).all() and torch.isfinite(S[0, 1][:, others]).all()
    else:
        assert not torch.isfinite(o[0, t, 1]).all()
        assert not torch.isfinite(S[0, 1]).all() and torch.isfinite(S[0, 0]).all()


def test_no_sequences_and_no_tokens():
    x = make(1, 0, 2, 64, 64, torch.bfloat16)
    for fn in (kda.kda_delta_chunk_fwd, kda.kda_delta_recurrent_fwd):
        o, S = call(fn, x)
        assert o.shape == (1, 0, 2, 64) and torch.equal(S.cpu(), x["S0"])
        x0 = make(0, 5, 2, 64, 64, torch.bfloat16)
        o, S = call(fn, x0)
        assert o.shape == (0, 5, 2, 64) and S.shape == (0, 2, 64, 64)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_captured_and_on_other_streams(dtype):
    xs = [make(1, 200, 2, 128, 128, dtype, seed=s) for s in (21, 22)]
    want = [call(kda.kda_delta_chunk_fwd, x) for x in xs]
    d = {n: t.to(DEV) for n, t in xs[0].items()}
    fixed = lambda: kda.kda_delta_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], initial_state=d["S0"],  # noqa: E731
                                            output_final_state=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        fixed()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, S = fixed()
    for x, (wo, wS) in zip(xs, want):
        for n in d:
            d[n].copy_(x[n])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, wo) and torch.equal(S, wS)
    # two calls at once, on two streams
    streams, got = [torch.cuda.Stream() for _ in xs], []
    dev = [{n: t.to(DEV) for n, t in x.items()} for x in xs]
    torch.cuda.synchronize()
    for st, y in zip(streams, dev):
        got.append(kda.kda_delta_chunk_fwd(y["q"], y["k"], y["v"], y["g"], y["beta"], initial_state=y["S0"],
                                           output_final_state=True, stream=st))
    torch.cuda.synchronize()
    for (o, S), (wo, wS) in zip(got, want):
        assert torch.equal(o, wo) and torch.equal(S, wS)
