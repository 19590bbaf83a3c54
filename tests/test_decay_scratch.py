"""Scratch of the decayed attention's FP32 chunks: a state for each 64 tokens and head, however many sequences
share them (no GPU needed)."""
import pytest

from test_block_refusals import BF16, F32, lib  # noqa: F401


@pytest.mark.parametrize("dtype,K,V", [(F32, 128, 128), (F32, 64, 64), (BF16, 96, 96), (F32, 256, 256), (BF16, 255, 3)])
@pytest.mark.parametrize("T,n", [(4096, 4096), (4096, 1), (65, 65000), (20000, 300), (100, 100)])
@pytest.mark.parametrize("H", [1, 32])
def test_scratch_does_not_grow_with_the_sequences(lib, dtype, K, V, T, n, H):  # noqa: F811
    state = H * K * V * 4
    factors = (T // 64 + n + 1) * H * 4  # one float a chunk and head
    assert lib.kda_decay_chunk_workspace_bytes(dtype, 1, T, H, K, V, n) <= T // 64 * state + factors + 1024


@pytest.mark.parametrize("B,T", [(3, 65), (2, 1000), (700, 128)])
def test_dense(lib, B, T):  # noqa: F811
    """Nothing is kept for a sequence's first chunk, which reads the initial state."""
    chunks = -(-T // 64)
    assert lib.kda_decay_chunk_workspace_bytes(F32, B, T, 4, 128, 128, 0) <= B * (chunks - 1) * 4 * 128 * 128 * 4 + B * chunks * 4 * 4 + 1024
