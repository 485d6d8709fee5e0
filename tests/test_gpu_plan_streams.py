"""Calls launched on a stream of their own: what a call allocates or uploads on torch's current stream stays until the
call has run, although nothing on the current stream refers to it any more."""
import pytest

from test_gpu_prefill import rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev(cuda_device):
    import paged_kv_looped_gb300 as rlt
    rlt.load()
    rlt.rlt_get_device_error()
    return cuda_device


def occupy(torch, dev, sizes, rounds=40):
    """Takes memory of these sizes from the current stream's pool again and again, and fills it."""
    kept = []
    for i in range(rounds):
        for n in sizes:
            kept.append(torch.full((max(n, 1),), i % 3, dtype=torch.uint8, device=dev))
    return kept


@pytest.mark.parametrize("form", ["made in the call", "uploaded before", "handle", "current stream"])
def test_prompt_plan_that_dies(dev, form):
    import torch
    import paged_kv_looped_gb300 as rlt
    lens = [300, 77, 512, 1, 130] * 4
    n, hq, hkv, d = sum(lens), 4, 2, 64
    q, k, v = rows(torch, dev, n, hq, hkv, d, 41)
    want = rlt.rlt_prefill_attn(q, k, v, rlt.rlt_plan_prefill(lens, hq // hkv))
    size = rlt.rlt_plan_prefill(lens, hq // hkv).items.nbytes
    side = torch.cuda.Stream()
    out, lse = torch.empty_like(want), torch.empty(n, hq, device=dev)
    torch.cuda.synchronize()
    for _ in range(3):
        out.zero_()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)                       # (some 10 ms) the call starts long after it returned
        if form == "made in the call":
            rlt.rlt_prefill_attn(q, k, v, rlt.rlt_plan_prefill(lens, hq // hkv), out=out, lse_out=lse, stream=side)
        elif form == "current stream":
            plan = rlt.rlt_plan_prefill(lens, hq // hkv).to(dev)
            with torch.cuda.stream(side):
                rlt.rlt_prefill_attn(q, k, v, plan, out=out, lse_out=lse)
            del plan
        else:
            rlt.rlt_prefill_attn(q, k, v, rlt.rlt_plan_prefill(lens, hq // hkv).to(dev), out=out, lse_out=lse,
                                 stream=side if form == "uploaded before" else side.cuda_stream)
        kept = occupy(torch, dev, [size])
        torch.cuda.synchronize()
        del kept
        assert torch.equal(out, want)
    assert rlt.rlt_get_device_error() == 0
