"""How near a bf16 output of the gated delta rule's chunks comes to a rounding of the exact result.

Tolerances.  The kernel rounds y, which is off the exact result r by e at most; the rounding of y is at least as near to y
as r's own rounding is, so an output is off r by no more than r's rounding and 2 e.  On the tensor cores e is made of:
the state that the queries read, U and P, each an operand of two bf16 terms (a rounding of at most 2^-8, and one as good of what it
left: 2^-16), the product of U's and P's second terms, which is left out (2^-8 of either), and the tensor cores' sums, which cut what
they add (2^-23 a product of 16 channels, 32 of them), all of the sums of their terms' absolute values (inter, intra); and
what FP32 is off by in the state and in U, (K + 256) 2^-24 in the norm, 8 times the root mean square at most in one place (as in the
tests of the other shapes)."""
import pytest
import torch

from delta_reference import F32
from test_gpu_delta import call, kda, make, reference

pytestmark = pytest.mark.gpu


def near(got, want, K, rows=None):
    o, (ro, _, inter, intra) = got[0].double().cpu(), want
    if rows is not None:
        o, ro, inter, intra = (t[:, :rows] for t in (o, ro, inter, intra))
    cut = 32 * 2.0 ** -23
    e = 1.01 * ((2.0 ** -16 + cut) * inter + (3 * 2.0 ** -16 + cut) * intra) + 8 * (K + 256) * F32 * ro.square().mean().sqrt()
    off = (o - ro).abs() - (ro.bfloat16().double() - ro).abs()
    assert (off <= 2 * e).all(), (off / e).max()


SHAPES = [(1, 200, 2, 128, 128), (2, 64, 2, 128, 128), (1, 130, 2, 64, 72), (1, 100, 2, 128, 256), (1, 130, 2, 40, 128)]


@pytest.mark.parametrize("B,T,H,K,V", SHAPES)
def test_outputs_of_the_state(B, T, H, K, V):
    """Large incoming states that hardly decay, small corrections: the queries' product with the state is the output."""
    x = make(B, T, H, K, V, torch.bfloat16, seed=71 + K, slow=True)
    x["S0"] *= 30
    x["beta"] *= 0.02
    near(call(kda.kda_delta_chunk_fwd, x), reference(x), K)


@pytest.mark.parametrize("B,T,H,K,V", SHAPES)
def test_outputs_of_the_chunk(B, T, H, K, V):
    """No incoming state, each chunk behind a decay that clears it: the chunk's own corrections are the output."""
    x = make(B, T, H, K, V, torch.bfloat16, seed=73 + V, state=False, slow=True)
    x["g"][:, ::64] = -float("inf")
    x["beta"][:] = 1
    x["q"][:] = x["k"] * 2
    near(call(kda.kda_delta_chunk_fwd, x), reference(x), K)


@pytest.mark.parametrize("K,V", [(128, 128), (64, 96)])
def test_outputs_of_packed_raw_rows(K, V):
    edges = [0, 70, 71, 71, 260]
    x = make(1, 260, 4, K, V, torch.bfloat16, Hk=2, raw=True, edges=edges, seed=75)
    near(call(kda.kda_delta_chunk_fwd, x, raw=True, edges=edges), reference(x, raw=True, edges=edges), K)
