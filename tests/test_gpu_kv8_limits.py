"""The largest numbers of the 8-bit cache's and the prompts' calls: where rows and sums stop being finite."""
import numpy as np
import pytest


pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev(cuda_device):
    import paged_kv_looped_gb300 as rlt
    rlt.load()
    rlt.rlt_get_device_error()
    return cuda_device


@pytest.mark.parametrize("d,rot", [(64, 64), (128, 30)])
def test_rows_at_the_top_of_the_range(dev, d, rot):
    """Values below 1.9375 * 2^127 are held as finite ones; from there on as 2^128, an infinity in bf16."""
    import torch
    import paged_kv_looped_gb300 as rlt
    below, at = (1 + 119 / 128) * 2.0 ** 127, 1.9375 * 2.0 ** 127
    v = torch.zeros(2, 1, d, dtype=torch.bfloat16, device=dev)
    v[0, 0, 1], v[0, 0, 5] = below, -below
    v[1, 0, 1], v[1, 0, 5] = at, -at
    pool = rlt.KV8Pool.empty(1, 1, 1, 16, d, dev)
    ko, vo = torch.empty_like(v), torch.empty_like(v)
    pos = torch.zeros(2, dtype=torch.int64, device=dev)
    rlt.rlt_kv8_append_rope(pool, 0, v, v.clone(), pos, torch.arange(2, device=dev), rot, 1e4, k_out=ko, v_out=vo)
    torch.cuda.synchronize()
    for x in (ko, vo):
        assert x[0, 0, 1] == 240 * 2.0 ** 120 and x[0, 0, 5] == -240 * 2.0 ** 120 and torch.isfinite(x[0]).all()
        assert x[1, 0, 1] == float("inf") and x[1, 0, 5] == float("-inf")
    assert pool.k_exp[0, 0, 0, :2].tolist() == [247, 247]
    # keys whose pair's norm stays below it stay finite through any rotation
    k = torch.zeros(8, 1, d, dtype=torch.bfloat16, device=dev)
    h = rot // 2
    k[..., 0] = k[..., h] = 1.3671875 * 2.0 ** 127              # 1.3671875 * sqrt 2 = 1.9335
    pos = torch.arange(8, device=dev)
    rlt.rlt_kv8_append_rope(pool, 0, k, k.clone(), pos, pos, rot, 1e4, k_out=(ko := torch.empty_like(k)))
    torch.cuda.synchronize()
    assert torch.isfinite(ko).all()


@pytest.mark.parametrize("hq,hkv,d", [(2, 1, 128), (1, 1, 64)])
@pytest.mark.parametrize("n", [129, 512, 2000])
def test_prompt_values_at_the_bound_of_the_sums(dev, hq, hkv, d, n):
    """Every key but the first 128 outweighs a row's first ones by nearly the 2^8 that the reference maximum may lie
    behind: sums stay finite for values below 2^120 / (number of keys)."""
    import torch
    import paged_kv_looped_gb300 as rlt
    top = 2.0 ** (120 - int(np.ceil(np.log2(n)))) * 0.99
    q = torch.zeros(n, hq, d, dtype=torch.bfloat16, device=dev)
    k, v = torch.zeros(n, hkv, d, dtype=torch.bfloat16, device=dev), torch.full((n, hkv, d), top, device=dev).bfloat16()
    q[..., 0] = 1.0
    k[128:, :, 0] = 7.9375 / 1.4427                             # in powers of two: 7.9375, rounded to bf16: below 8
    lse = torch.empty(n, hq, device=dev)
    out = rlt.rlt_prefill_attn(q, k, v, rlt.rlt_plan_prefill([n], hq // hkv), lse_out=lse, scale=1.0)
    torch.cuda.synchronize()
    # a mean of one value: that value up to the weights' roundings (2^-8 each, the sum's share of them) and its own
    assert float(k[128:, :, 0].float().max()) * 1.4427 < 8
    want = v.double()[:1].max()
    assert ((out.double() - want).abs() <= 2 * 2.0 ** -8 * want + 2.0 ** -14 * want).all()
    assert rlt.rlt_get_device_error() == 0
