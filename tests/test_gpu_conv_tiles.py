"""The short convolution in tiles of 8, 16 and 64 rows (and more, where a grid would be too long), against
float64: sequences that start at the edges of the tiles, within the W - 1 rows behind them, and are empty there.

The rows a tile has follow from the number of tiles and the multiprocessors planned for, so a pretended count
of one brings the long tiles into small cases.  Bounds as in test_gpu_block: half a step of the output's type,
float32 sums of W products, the activation's exponential.
"""
import pytest
import torch

from block_reference import F32, HALF
from test_gpu_block import BF, close, kda  # noqa: F401

pytestmark = pytest.mark.gpu


def reference(x, w, S0, edges):
    """(y, sums of absolute values, final state) in float64, all rows at once; x [T, D], S0 [N, W - 1, D]."""
    W, T = w.shape[1], edges[-1]
    lens = torch.tensor(edges[1:], device=x.device) - torch.tensor(edges[:-1], device=x.device)
    owner = torch.repeat_interleave(torch.arange(len(lens), device=x.device), lens)
    place = torch.arange(T, device=x.device) - torch.tensor(edges, device=x.device)[owner]
    y = torch.zeros(T, x.shape[1], dtype=torch.float64, device=x.device)
    size = torch.zeros_like(y)
    for tap in range(W):
        back = W - 1 - tap
        past = x[(torch.arange(T, device=x.device) - back).clamp_min(0)].double()
        old = S0[owner, (place - back + W - 1).clamp(0, W - 2)].double()
        term = w[:, tap].double() * torch.where((place < back)[:, None], old, past)
        y += term
        size += term.abs()
    last = S0.clone()
    for n, (a, b) in enumerate(zip(edges, edges[1:])):
        m = min(b - a, W - 1)
        if m:
            last[n] = torch.cat([S0[n, m:], x[b - m:b]])
    return y, size, last


def check(kda, dtype, edges, D, W, inplace, pad=13):  # noqa: F811
    g = torch.Generator(device="cuda").manual_seed(D + W + edges[-1])
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    T, N = edges[-1], len(edges) - 1
    x, S0, w = r(T + pad, D).to(dtype), r(N, W - 1, D).to(dtype), r(D, W)
    y64, size, last = reference(x, w, S0, edges)
    x[T:] = float("nan")
    out, s = torch.full((1, T + pad, D), 7.0, dtype=dtype, device="cuda"), S0.clone()
    cu = torch.tensor(edges, dtype=torch.int32, device="cuda")
    y, S = kda.kda_short_conv_fwd(x[None], w, act=kda.ACT_SILU, initial_state=s, output_final_state=True, cu_seqlens=cu,
                                  out=out, final_state=s if inplace else None)
    torch.cuda.synchronize()
    assert torch.equal(S, last) and bool((y[0, T:] == 7.0).all())
    want = y64 * torch.sigmoid(y64)
    fast = 2.0 ** -17 if dtype == BF else 24 * F32
    bound = (HALF[dtype] + fast) * want.abs() + 1.1 * (W + 3) * F32 * size + 1e-30  # |d act / d z| <= 1.1
    close(y[0, :T], want.cpu(), bound.cpu(), "y")


def edges_around(tile, W, T):
    """Starts at, before and within W rows behind the tiles' edges, empty sequences there, long runs between."""
    at = {0, T}
    for t in range(tile, T, 3 * tile):
        at |= {t, t + 1, t + W - 2, t + W - 1, t + tile - 1, t + tile + W}
    at = sorted(a for a in at if a <= T)
    return sorted(at + [a for i, a in enumerate(at) if i % 3 == 0])  # (twice: an empty sequence)


@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("D", [1032, 1025])
@pytest.mark.parametrize("W", range(2, 9))
@pytest.mark.parametrize("tile,T", [(16, 61), (64, 700)])
@pytest.mark.parametrize("inplace", [False, True])
def test_tiles(kda, dtype, D, W, tile, T, inplace):  # noqa: F811
    """D = 1032: 3 blocks of vectors; 1025: 9 blocks of single channels.  61 rows: fewer than 8 blocks of 64-row
    tiles (16-row tiles: 12 or 36); 700 rows: 33 or 99 of 64."""
    if tile == 16 and D == 1025:
        T = 45  # (nine blocks of 64 rows are eight already: here only the starts differ)
    try:
        kda.kda_test_hooks(sm_count=1)
        check(kda, dtype, edges_around(tile, W, T), D, W, inplace)
        check(kda, dtype, [0, T], D, W, inplace)
        check(kda, dtype, [0, 0, T - 3, T - 3, T, T], D, W, inplace)
    finally:
        kda.kda_test_hooks()


@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("W", [2, 4, 6])
@pytest.mark.parametrize("T", [2000, 3500])
def test_as_the_device_is(kda, dtype, W, T):  # noqa: F811
    """24 blocks of channels: 16 rows a tile up to some 3200 rows, then 64."""
    check(kda, dtype, edges_around(64, W, T), 12288, W, True)
    check(kda, dtype, [0, 5, 5, T // 2 + 1, T], 12288, W, False)


@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_more_tiles_than_a_grid_holds(kda, dtype):  # noqa: F811
    T = 65536 * 64 + 100
    check(kda, dtype, [0, 3, 3, 65536 * 64 - 1, 65536 * 64 + 1, T], 4, 4, True)


@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_dense(kda, dtype):  # noqa: F811
    """Sequences of one length, without offsets, whose starts lie anywhere in the tiles."""
    B, T, D, W = 7, 210, 1032, 4
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn(B, T, D, generator=g, device="cuda").to(dtype)
    S0 = torch.randn(B, W - 1, D, generator=g, device="cuda").to(dtype)
    w = torch.randn(D, W, generator=g, device="cuda")
    y64, size, last = reference(x.view(B * T, D), w, S0, list(range(0, B * T + 1, T)))
    try:
        kda.kda_test_hooks(sm_count=1)
        y, S = kda.kda_short_conv_fwd(x, w, act=kda.ACT_NONE, initial_state=S0, final_state=S0)
    finally:
        kda.kda_test_hooks()
    assert S is S0 and torch.equal(S, last)
    close(y.view(B * T, D), y64.cpu(), (HALF[dtype] * y64.abs() + (W + 3) * F32 * size + 1e-30).cpu(), "y")
