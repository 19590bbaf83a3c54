"""The norm and rotation of query and key heads against float64.

Tolerances: a row's sum of squares of D terms and its root are off by at most (D / 2 + 4) 2^-24 relative (the root
halves the sum's), the weight's and the rotation's products by 2^-24 each; a cosine or sine is off by 2^-22 at most
(its argument is a float32 of at most half a turn: pi 2^-25, and the function's own), of the pair's length."""
import pytest
import torch

from delta_reference import F32, HALF, delta, gate, qk
from block_reference import gated_norm

pytestmark = pytest.mark.gpu

kda = pytest.importorskip("chunked_kda_gb300")
DEV = "cuda"


def freq(R, base=1e4):
    return base ** (-torch.arange(0, R, 2, dtype=torch.float64) / max(R, 1)).float()


def check(y, x, want, dtype, D, R, interleaved):
    assert y.dtype == dtype and y.shape == x.shape
    y = y.double().cpu()
    size = want.abs().clone()  # a pair's length, where there is one
    half = R // 2
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, half + i)
        size[..., a] = size[..., b] = torch.hypot(want[..., a], want[..., b])
    bound = (D / 2 + 16) * F32 * size + HALF[dtype] * want.abs() * 1.001
    bad = (y - want).abs() > bound
    assert not bad.any(), ((y - want).abs() / bound)[bad].max()


CASES = [  # B, T, Hq, Hk, D, R, norm, axes, interleaved, sliced
    (2, 7, 4, 2, 128, 128, 1, 1, False, True),
    (1, 33, 8, 8, 64, 64, 2, 1, False, False),
    (3, 1, 5, 1, 256, 64, 1, 3, False, True),
    (1, 100, 2, 1, 128, 64, 1, 2, True, True),
    (1, 3, 1, 0, 96, 96, 1, 1, False, False),
    (2, 5, 3, 1, 66, 50, 1, 4, False, True),
    (2, 5, 3, 2, 66, 66, 2, 1, True, True),
    (1, 9, 2, 2, 17, 6, 1, 1, False, False),
    (1, 9, 2, 2, 1, 0, 2, 1, False, False),
    (1, 40, 32, 4, 32, 0, 1, 1, False, True),
    (1, 5000, 1, 1, 8, 8, 0, 1, False, True),
    (4, 1, 70, 7, 40, 24, 1, 3, True, False),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,T,Hq,Hk,D,R,norm,axes,interleaved,sliced", CASES)
def test_against_float64(dtype, B, T, Hq, Hk, D, R, norm, axes, interleaved, sliced):
    gen = torch.Generator().manual_seed(D + R)
    rows = torch.randn(B, T, Hq + 2 * Hk, D, generator=gen).to(dtype)
    dev = rows.to(DEV)
    parts = lambda z: (z[:, :, :Hq], z[:, :, Hq:Hq + Hk] if Hk else None)  # noqa: E731
    (q, k), (dq, dk) = parts(rows), parts(dev)
    if not sliced:
        dq, dk = dq.contiguous(), dk.contiguous() if Hk else None
    wq, wk = (1 + 0.1 * torch.randn(D, generator=gen) for _ in range(2))
    if norm == 2:
        wq = wk = None
    pos = torch.randint(-5, 2 ** 20, (axes, B, T), generator=gen, dtype=torch.int32) if R else None
    if R and axes == 1:
        pos = pos[0]
    f = freq(R) if R else None
    pair_axes = [i % axes for i in range(R // 2)] if axes > 1 else None
    m = 1.25 if R else 1.0
    c = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    yq, yk = kda.kda_qk_norm_rope_fwd(dq, dk, c(wq), c(wk) if Hk else None, norm=norm, positions=c(pos), inv_freq=c(f),
                                      pair_axes=pair_axes, interleaved=interleaved, rope_scale=m)
    check(yq, q, qk(q, wq, norm, pos, f, pair_axes, interleaved, m), dtype, D, R, interleaved)
    if Hk:
        check(yk, k, qk(k, wk, norm, pos, f, pair_axes, interleaved, m), dtype, D, R, interleaved)
    else:
        assert yk is None
    # in place, the values between left alone
    before = dev.clone()
    if sliced:
        kda.kda_qk_norm_rope_fwd(dq, dk, c(wq), c(wk) if Hk else None, norm=norm, positions=c(pos), inv_freq=c(f),
                                 pair_axes=pair_axes, interleaved=interleaved, rope_scale=m, q_out=dq, k_out=dk)
        assert torch.equal(dq, yq) and (not Hk or torch.equal(dk, yk))
        assert torch.equal(dev[:, :, Hq + Hk:], before[:, :, Hq + Hk:])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_of_zeros_and_what_is_not_finite(dtype):
    x = torch.randn(1, 6, 2, 64, generator=torch.Generator().manual_seed(3)).to(dtype)
    x[0, 1] = 0
    x[0, 2, 0, 5] = float("nan")
    x[0, 3, 1, 7] = float("inf")
    y, _ = kda.kda_qk_norm_rope_fwd(x.to(DEV), norm=kda.NORM_L2)
    y = y.cpu()
    assert (y[0, 1] == 0).all() and y[0, 2, 0].isnan().all()
    assert (y[0, 3, 1, :7] == 0).all() and y[0, 3, 1, 7].isnan()
    rest = torch.ones(6, 2, dtype=torch.bool)
    rest[2, 0] = rest[3, 1] = False
    assert torch.isfinite(y[0][rest]).all()
    f = freq(64)
    f[4] = float("inf")
    y, _ = kda.kda_qk_norm_rope_fwd(x[:, 4:5].contiguous().to(DEV), positions=torch.ones(1, 1, dtype=torch.int32, device=DEV),
                                    inv_freq=f.to(DEV))
    bad = torch.zeros(64, dtype=torch.bool)
    bad[[4, 36]] = True
    assert (y.cpu().isnan() == bad).all()


def test_no_tokens():
    y, z = kda.kda_qk_norm_rope_fwd(torch.zeros(0, 4, 2, 64, device=DEV), torch.zeros(0, 4, 1, 64, device=DEV))
    assert y.shape == (0, 4, 2, 64) and z.shape == (0, 4, 1, 64)


def test_arguments_that_are_refused():
    x = torch.zeros(2, 3, 4, 64, device=DEV)
    pos, f = torch.zeros(2, 3, dtype=torch.int32, device=DEV), freq(64).to(DEV)
    fn = kda.kda_qk_norm_rope_fwd
    for bad, err in ((dict(positions=pos), ValueError), (dict(inv_freq=f), ValueError),
                     (dict(positions=pos.long(), inv_freq=f), TypeError), (dict(positions=pos[:1], inv_freq=f), ValueError),
                     (dict(positions=pos, inv_freq=f.repeat(2)), kda.KdaError),
                     (dict(positions=pos, inv_freq=f, pair_axes=[0] * 31), ValueError),
                     (dict(positions=pos, inv_freq=f, pair_axes=[1] * 32), ValueError),
                     (dict(q_weight=f), ValueError), (dict(k_weight=f), ValueError), (dict(k=x.bfloat16()), TypeError),
                     (dict(k=x[:, :2]), ValueError), (dict(q_out=x.transpose(1, 2)), ValueError), (dict(norm=3), kda.KdaError),
                     (dict(eps=-1.0), kda.KdaError), (dict(eps=float("nan")), kda.KdaError)):
        with pytest.raises(err):
            fn(x, **bad)
    with pytest.raises(ValueError):
        fn(x[..., ::2])
    with pytest.raises(ValueError):
        fn(x[:, ::2].expand(2, 2, 4, 64)[:, :, ::2])
    with pytest.raises(ValueError):
        fn(x[:, :1].expand(2, 3, 4, 64))  # every token the same row
    with pytest.raises(kda.KdaError):
        fn(x[:1, :1].expand(1, 3, 4, 64))
    wide = torch.zeros(6, 8, 64, device=DEV).view(2, 3, 8, 64)
    with pytest.raises(kda.KdaError):
        fn(wide[:, :, :4], wide[:, :, 4:], q_out=wide[:, :, 2:6])
    with pytest.raises(ValueError):
        fn(x.requires_grad_())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_the_operators_one_after_another(dtype):
    """Rows of norm 1 with their positions, the delta rule over a prompt and then token by token, the gated norm."""
    B, T, H, Hk, D = 2, 130, 4, 2, 128
    gen = torch.Generator().manual_seed(31)
    rows = torch.randn(B, T, 2 * Hk, D, generator=gen).to(dtype)
    v, z = (torch.randn(B, T, H, D, generator=gen).to(dtype) for _ in range(2))
    g, beta = -0.2 * torch.rand(B, T, H, generator=gen), torch.rand(B, T, H, generator=gen).to(dtype)
    w = 1 + 0.1 * torch.randn(D, generator=gen)
    pos, f = torch.arange(T, dtype=torch.int32).expand(B, T).contiguous(), freq(64)
    d = [t.to(DEV) for t in (rows, v, z, g, beta, w, pos, f)]
    q, k = kda.kda_qk_norm_rope_fwd(d[0][:, :, :Hk], d[0][:, :, Hk:], norm=kda.NORM_L2, positions=d[6], inv_freq=d[7])
    S, o, cut = torch.zeros(B, H, D, D, device=DEV), [], 128
    part = lambda x, lo, hi: x[:, lo:hi].contiguous()  # noqa: E731
    o.append(kda.kda_delta_chunk_fwd(*(part(x, 0, cut) for x in (q, k, d[1], d[3], d[4])), initial_state=S, final_state=S)[0])
    for t in range(cut, T):
        o.append(kda.kda_delta_recurrent_fwd(*(part(x, t, t + 1) for x in (q, k, d[1], d[3], d[4])), initial_state=S,
                                             final_state=S)[0])
    o = torch.cat(o, 1)
    y = kda.kda_gated_norm_fwd(o, d[2], d[5], act=kda.ACT_SILU)
    # each step against the reference of what it was given, and the whole within what the steps add up to
    for got, x in ((q, rows[:, :, :Hk]), (k, rows[:, :, Hk:])):
        check(got, x, qk(x, None, 2, pos, f), dtype, D, 64, False)
    ro, rS, inter, intra = delta(q.cpu(), k.cpu(), v, gate(g), beta)
    tol = (D + 256) * F32
    assert (S.double().cpu() - rS).norm() <= tol * rS.norm()
    assert (o.double().cpu() - ro).norm() <= (tol if dtype == torch.float32 else 3.5e-3) * ro.norm()
    ry = gated_norm(o.cpu(), z, w, 1e-6, 2)
    assert ((y.double().cpu() - ry).abs() <= (D + 16) * F32 * ry.abs() + HALF[dtype] * ry.abs() * 1.001).all()
