"""The 8-bit decode's and the prompt kernel's bounded waits give up, report it, and leave the device usable.

As test_gpu_timeout.py: rlt_debug_fault_next_decode leaves one copy of the next call unissued and gives its waits a limit
of a few milliseconds, on the host and without any GPU fault.  Checked: the call returns at once, the error word
holds exactly the timeout bit, nothing outside the outputs and the workspace changes, every row that the dropped copy
does not feed is right, and the next ordinary call is right everywhere.
"""
import time

import numpy as np
import pytest

import kv8_ref as R
from test_gpu_guards import Guarded
from test_gpu_kv8_decode import Case
from test_gpu_prefill import check, rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev(cuda_device):
    import paged_kv_looped_gb300 as rlt
    rlt.load()
    rlt.rlt_get_device_error()
    return cuda_device


@pytest.mark.parametrize("d,hq,hkv", [(128, 4, 2), (64, 8, 2)])
def test_decode(dev, d, hq, hkv):
    import torch
    import paged_kv_looped_gb300 as rlt
    c = Case(dev, [300, 170, 5], hq, hkv, d, 16, seed=d)
    B, G, longest = 3, hq // hkv, 300
    ws = Guarded(rlt.rlt_paged_decode_kv8_workspace_size(B, hq, hkv, d, longest, 64), dev)
    out, lse = Guarded(B * hq * d * 2, dev), Guarded(B * hq * 4, dev)
    o, l = out.view(torch.bfloat16, (B, hq, d)), lse.view(torch.float32, (B, hq))

    def call():
        rlt.rlt_paged_decode_attn_kv8(c.pool, c.bank, c.q, c.table, c.seq, longest, out=o, lse_out=l, workspace=ws.bytes(),
                                      split_tokens=64)
        torch.cuda.synchronize()

    ref = c.reference()
    call()
    c.check(o, l, ref)
    rlt.rlt_debug_fault_next_decode(2_000_000)
    t0 = time.perf_counter()
    call()
    elapsed = time.perf_counter() - t0
    assert rlt.rlt_get_device_error() == rlt.DEVERR_TIMEOUT
    assert elapsed < 0.5, elapsed                               # 2 ms waits ran out, not the 1 s default
    assert out.intact() and lse.intact() and ws.intact()
    keep = np.ones((B, hq), bool)
    keep[0, :G] = False                                         # request 0's heads of kv head 0
    go, gl = o.double().cpu().numpy(), l.double().cpu().numpy()
    assert np.isfinite(go).all()
    assert np.all(np.abs(go - ref[0])[keep] <= R.attention_bound(ref[0], ref[2], ref[3], 2.0 ** -11)[keep])
    assert np.all(np.abs(gl - ref[1])[keep] <= R.lse_bound(ref[1], ref[3], d)[keep])
    # warp 0's first 32 tokens of the first split are missing: the sum of the others' weights is what is left
    kk = c.k[[c.tables[0, i // 16] for i in range(32, 300)], 0, [i % 16 for i in range(32, 300)]]
    rest = np.log(np.exp(c.q[0, :G].double().cpu().numpy() @ kk.T * c.scale).sum(1))
    assert np.all(np.abs(gl[0, :G] - rest) <= R.lse_bound(rest, ref[3][0, :G], d))
    call()                                                      # the switch was one-shot
    assert rlt.rlt_get_device_error() == 0
    c.check(o, l, ref)


@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 128), (3, 1, 64), (2, 2, 128)])
@pytest.mark.parametrize("lens", [[100, 40], [700, 300, 257]])
def test_prompts(dev, hq, hkv, d, lens):
    import torch
    import paged_kv_looped_gb300 as rlt
    n, G = sum(lens), hq // hkv
    q, k, v = rows(torch, dev, n, hq, hkv, d, 51)
    out, lse = Guarded(n * hq * d * 2, dev), Guarded(n * hq * 4, dev)
    o, l = out.view(torch.bfloat16, (n, hq, d)), lse.view(torch.float32, (n, hq))
    plan = rlt.rlt_plan_prefill(lens, G).to(dev)

    def call():
        o.fill_(9.0), l.fill_(9.0)
        rlt.rlt_prefill_attn(q, k, v, plan, out=o, lse_out=l)
        torch.cuda.synchronize()

    call()
    check(o, l, q, k, v, lens, 1 / np.sqrt(d))
    want, want_lse = o.clone(), l.clone()
    rlt.rlt_debug_fault_next_decode(2_000_000)
    t0 = time.perf_counter()
    call()
    elapsed = time.perf_counter() - t0
    assert rlt.rlt_get_device_error() == rlt.DEVERR_TIMEOUT
    assert elapsed < 0.5, elapsed
    assert out.intact() and lse.intact()
    # block 0: the plan's first item, heads 0 and 1 of an even group, else head 0 at up to 256 rows
    row0, length, q0, _ = (int(x) for x in plan.items[0])
    lost = torch.zeros(n, hq, dtype=torch.bool, device=dev)
    if G % 2 == 0:
        lost[row0 + q0: row0 + min(q0 + 128, length), :2] = True
    else:
        lost[row0 + q0: row0 + min(q0 + 256, length), :1] = True
    assert (o[lost] == 9).all() and (l[lost] == 9).all()
    assert torch.equal(o[~lost], want[~lost]) and torch.equal(l[~lost], want_lse[~lost])
    for _ in range(3):                                          # one-shot, and nothing of the SM was kept
        call()
        assert rlt.rlt_get_device_error() == 0
        assert torch.equal(o, want) and torch.equal(l, want_lse)
