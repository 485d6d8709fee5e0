"""Prompts whose values hold infinities and NaN in the tiles of the queries' own keys, which two query tiles share: the
same bits every time, nothing where a query may not look."""
import pytest

from test_gpu_prefill import rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev(cuda_device):
    import paged_kv_looped_gb300 as rlt
    rlt.load()
    rlt.rlt_get_device_error()
    return cuda_device


@pytest.mark.parametrize("hq,hkv,d", [(3, 1, 64), (1, 1, 128), (3, 3, 128), (2, 1, 128), (8, 2, 64)])
def test_an_infinity_whose_weight_underflows(dev, hq, hkv, d):
    """A key far below every other's score, with an infinite value: an infinity or a NaN for the queries that see it, the
    same one in every run, and nothing for the others."""
    import torch
    import paged_kv_looped_gb300 as rlt
    lens = [300, 513, 130]
    n = sum(lens)
    q, k, v = rows(torch, dev, n, hq, hkv, d, 31, fused=False)
    q[..., 0] = 1.0
    odd = [(0, 70, 3), (0, 200, 5), (1, 511, d - 1), (2, 129, 0)]
    first = [0, 300, 813]
    for s, i, c in odd:
        k[first[s] + i, :, 0] = -8000.0
        v[first[s] + i, :, c] = 0.0
    plan = rlt.rlt_plan_prefill(lens, hq // hkv).to(dev)
    clean_lse, lse = torch.empty(n, hq, device=dev), torch.empty(n, hq, device=dev)
    clean = rlt.rlt_prefill_attn(q, k, v, plan, lse_out=clean_lse)
    sees = torch.zeros(n, hq, d, dtype=torch.bool, device=dev)
    for s, i, c in odd:
        v[first[s] + i, :, c] = float("inf")
        sees[first[s] + i: first[s] + lens[s], :, c] = True
    outs = [rlt.rlt_prefill_attn(q, k, v, plan, lse_out=lse).view(torch.int16) for _ in range(40)]
    torch.cuda.synchronize()
    for o in outs[1:]:
        assert torch.equal(o, outs[0])
    out = outs[0].view(torch.bfloat16)
    assert torch.equal(out[~sees], clean[~sees]) and torch.equal(lse, clean_lse)
    assert (out[sees].isnan() | (out[sees] == float("inf"))).all()
    # a query of weight 1 on it (the key itself, where it is the sequence's first) would not underflow: none here is
    assert rlt.rlt_get_device_error() == 0


@pytest.mark.parametrize("hq,hkv,d", [(2, 1, 128), (4, 2, 128), (8, 2, 64), (3, 1, 128), (1, 1, 64)])
def test_nan_in_every_quarter_of_ragged_prompts(dev, hq, hkv, d):
    import torch
    import paged_kv_looped_gb300 as rlt
    g = torch.Generator().manual_seed(hq + d)
    lens = torch.randint(1, 420, (60,), generator=g).tolist()
    n = sum(lens)
    q, k, v = rows(torch, dev, n, hq, hkv, d, 33, fused=False)
    hit = torch.zeros(n, hkv, d, dtype=torch.bool)
    at = 0
    for m in lens:
        for _ in range(3):
            i, h, c = (int(torch.randint(0, x, (1,), generator=g)) for x in (m, hkv, d))
            hit[at + i, h, c] = True
        at += m
    hit = hit.to(dev)
    v.masked_fill_(hit, 0.0)
    plan = rlt.rlt_plan_prefill(lens, hq // hkv).to(dev)
    clean = rlt.rlt_prefill_attn(q, k, v, plan)
    v.masked_fill_(hit, float("nan"))
    outs = [rlt.rlt_prefill_attn(q, k, v, plan) for _ in range(20)]
    torch.cuda.synchronize()
    sees, at = torch.zeros(n, hkv, d, dtype=torch.bool, device=dev), 0
    for m in lens:
        sees[at:at + m] = hit[at:at + m].cumsum(0) > 0
        at += m
    sees = sees.repeat_interleave(hq // hkv, 1)
    for o in outs:
        assert torch.equal(o.isnan(), sees) and torch.equal(o[~sees], clean[~sees])
    assert rlt.rlt_get_device_error() == 0
