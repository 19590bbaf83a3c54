"""The norm and rotation of many rows of query and key heads, which warps take through shared memory: against float64
at odd head counts, partial rotations and strides, in place, and in a graph.  Tolerances: those of few rows."""
import pytest
import torch

from delta_reference import qk
from test_gpu_qk_norm import check, freq, kda

pytestmark = pytest.mark.gpu
DEV = "cuda"

CASES = [  # Hq, Hk, D, R, norm, axes, interleaved, sliced; at least two groups of 2 KB a token
    (16, 4, 64, 64, 1, 1, False, True),
    (10, 3, 256, 64, 1, 3, False, True),
    (20, 20, 48, 32, 1, 2, True, True),
    (9, 8, 128, 0, 2, 1, False, False),
    (33, 16, 128, 128, 2, 1, True, False),
    (70, 0, 32, 16, 0, 1, False, False),
    (65, 65, 16, 16, 1, 4, False, True),
    # multiples of 8 only
    (16, 4, 128, 104, 1, 1, False, True),
    (13, 13, 40, 40, 2, 1, False, False),
    (9, 5, 248, 56, 1, 2, True, True),
    (40, 0, 24, 8, 0, 1, False, False),
    # heads or rotations that are not whole vectors
    (5, 2, 244, 36, 1, 2, False, True),
    (7, 1, 130, 130, 2, 1, False, False),
    (6, 3, 36, 20, 1, 1, True, True),
    (4, 2, 128, 34, 1, 3, False, True),
    (3, 1, 101, 66, 1, 1, False, True),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("Hq,Hk,D,R,norm,axes,interleaved,sliced", CASES)
def test_many_rows_against_float64(dtype, Hq, Hk, D, R, norm, axes, interleaved, sliced):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    B, T = (1, 64 * sms + 7) if Hq != 10 else (2, 32 * sms + 3)
    gen = torch.Generator().manual_seed(D + R + Hq)
    rows = torch.randn(B, T, Hq + 2 * Hk, D, generator=gen).to(dtype)
    rows[0, 3, 0, 1] = float("nan")  # stays in its row
    dev = rows.to(DEV)
    parts = lambda z: (z[:, :, :Hq], z[:, :, Hq:Hq + Hk] if Hk else None)  # noqa: E731
    (q, k), (dq, dk) = parts(rows), parts(dev)
    if not sliced:
        dq, dk = dq.contiguous(), dk.contiguous() if Hk else None
    wq, wk = (1 + 0.1 * torch.randn(D, generator=gen) for _ in range(2))
    if norm != 1:
        wq = wk = None
    pos = torch.randint(-5, 2 ** 20, (axes, B, T), generator=gen, dtype=torch.int32) if R else None
    if R and axes == 1:
        pos = pos[0]
    f = freq(R) if R else None
    kw = dict(norm=norm, pair_axes=[i % axes for i in range(R // 2)] if axes > 1 else None, interleaved=interleaved,
              rope_scale=1.25 if R else 1.0)
    c = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    wq_, wk_, pos_, f_ = c(wq), c(wk) if Hk else None, c(pos), c(f)
    yq, yk = kda.kda_qk_norm_rope_fwd(dq, dk, wq_, wk_, positions=pos_, inv_freq=f_, **kw)
    for x, y, w in ((q, yq, wq), (k, yk, wk))[:2 if Hk else 1]:
        want = qk(x, w, norm, pos, f, kw["pair_axes"], interleaved, kw["rope_scale"])
        if x is q:  # the row with the NaN: all of it behind a norm, else its pair
            row = y[0, 3, 0].clone()
            assert row.isnan().all() if norm else row.isnan().sum() == 2
            y, want, x = y.clone(), want.clone(), x.clone()
            y[0, 3, 0], want[0, 3, 0] = 0, 0
        check(y, x, want, dtype, D, R, interleaved)
    # again, in a graph: the same
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        zq, zk = kda.kda_qk_norm_rope_fwd(dq, dk, wq_, wk_, positions=pos_, inv_freq=f_, **kw)
    g.replay()
    same = lambda a, b: torch.equal(a.nan_to_num(1e30), b.nan_to_num(1e30))  # noqa: E731
    assert same(zq, yq) and (not Hk or same(zk, yk))
    # in place, the values between left alone
    before = dev.clone()
    kda.kda_qk_norm_rope_fwd(dq, dk, wq_, wk_, positions=pos_, inv_freq=f_, q_out=dq, k_out=dk, **kw)
    assert same(dq, yq) and (not Hk or same(dk, yk))
    if sliced:
        assert same(dev[:, :, Hq + Hk:], before[:, :, Hq + Hk:])
    assert kda.kda_fused_wait_timeouts() == 0
