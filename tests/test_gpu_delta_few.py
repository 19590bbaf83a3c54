"""A few tokens a sequence in the gated delta rule's chunked form, on both sides of the borders between its ways (few units,
more than the device has multiprocessors, many): against float64, and without scratch where the call says so."""
import pytest
import torch

from test_gpu_delta import call, check, kda, make, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,T", [(torch.bfloat16, t) for t in (3, 4, 5, 6, 7, 8)] + [(torch.float32, t) for t in (6, 7, 12, 13, 16, 17)])
@pytest.mark.parametrize("per", [0, 1, 4])
@pytest.mark.parametrize("K,V", [(64, 32), (16, 136)])
def test_few_tokens(dtype, T, per, K, V):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    n = per * sms + 3
    units = n * (-(-V // 128) if dtype == torch.bfloat16 else 1)
    most = ((3, 5, 7) if dtype == torch.bfloat16 else (6, 12, 16))[0 if units <= sms else 1 if units <= 4 * sms else 2]
    size = kda.kda_delta_chunk_workspace_bytes(dtype, 1, T, n, K, V)
    assert size == 0 if T <= most else size > 0 or dtype == torch.bfloat16
    x = make(1, T, n, K, V, dtype, seed=T + per)
    got = call(kda.kda_delta_chunk_fwd, x)
    check(got, reference(x), dtype, K)
    if T <= most:
        same = call(kda.kda_delta_recurrent_fwd, x)
        assert torch.equal(got[0], same[0]) and torch.equal(got[1], same[1])
