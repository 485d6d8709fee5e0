"""Written-prefix counters of the 8-bit append at positions no sequence has: a counter becomes at least position + 1
(as an int32 can hold it), and a position below zero counts nothing."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rot", [64, 62, 0])
def test_counters_at_positions_of_any_size(cuda_device, rot):
    import torch
    import paged_kv_looped_gb300 as rlt
    rlt.rlt_get_device_error()
    pos = [5, -1, -2, -(1 << 32) + 5, -(1 << 63), (1 << 31) - 1, (1 << 31) + 3, (1 << 32) + 9, (1 << 63) - 1, 0]
    n, dev = len(pos), cuda_device
    pool = rlt.KV8Pool.empty(1, 1, 2, 16, 64, dev)
    k = torch.randn(n, 2, 64, device=dev).bfloat16()
    written = torch.full((1, n), 2, dtype=torch.int32, device=dev)
    rlt.rlt_kv8_append_rope(pool, 0, k, k.clone(), torch.tensor(pos, device=dev), torch.arange(n, device=dev), rot, 1e4,
                            request=torch.arange(n, dtype=torch.int32, device=dev), written=written)
    torch.cuda.synchronize()
    top = (1 << 31) - 1
    assert written[0].tolist() == [max(2, min(p + 1, top)) for p in pos]
    assert rlt.rlt_get_device_error() == 0
