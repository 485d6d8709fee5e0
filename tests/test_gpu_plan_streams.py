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


@pytest.mark.parametrize("call", ["decode", "prefix", "extend", "kv8"])
def test_workspaces_plans_and_outputs_of_one_call(dev, call):
    """The bf16 pool's calls and the 8-bit decode with nothing kept by the caller but the result."""
    import numpy as np
    import torch
    import paged_kv_looped_gb300 as rlt
    import workloads as W
    from helpers import bf16_dev, i32_dev
    lens = [3000, 2900, 3100, 1500, 700, 2333]
    case = W.custom(B=6, Hq=16, Hkv=2, D=128, ps=16, seq_lens=lens, shared_frac=0.8, seed=21)
    h = W.host_tensors(case)
    pool = rlt.KVPool(bf16_dev(h.k_pool, dev)[None].contiguous(), bf16_dev(h.v_pool, dev)[None].contiguous())
    q, pt, sl = bf16_dev(h.q, dev), i32_dev(case.page_table, dev), i32_dev(case.seq_lens, dev)
    new = [64, 1, 130, 0, 700, 2]
    qx = bf16_dev(W.bf16_normal(np.random.default_rng(3), (sum(new), 16, 128)), dev)
    prefix = lambda: rlt.rlt_plan_prefix(case.page_table, case.seq_lens, 16, 2, False, case.group)        # noqa: E731
    extend = lambda: rlt.rlt_plan_extend(case.seq_lens, new, 16, 2, case.group)                           # noqa: E731
    shape = (1, *h.k_pool.shape)
    k8 = [torch.zeros(shape, dtype=torch.uint8, device=dev).random_(0, 120).view(torch.float8_e4m3fn) for _ in range(2)]
    pool8 = rlt.KV8Pool(*k8, *(torch.full(shape[:4], 120, dtype=torch.uint8, device=dev) for _ in range(2)))
    ws = rlt.rlt_paged_decode_workspace_size(6, 16, 2, 128, case.max_seq_len, 64)
    arrays, run = {
        "decode": ([], lambda **kw: rlt.rlt_paged_decode_attn(pool, 0, q, pt, sl, case.max_seq_len, split_tokens=64, **kw)),
        "kv8": ([], lambda **kw: rlt.rlt_paged_decode_attn_kv8(pool8, 0, q, pt, sl, case.max_seq_len, split_tokens=64, **kw)),
        "prefix": ([prefix().segments, prefix().members, prefix().member_limit, prefix().request_prefix],
                   lambda **kw: rlt.rlt_paged_decode_attn_prefix(pool, 0, q, pt, sl, case.max_seq_len, prefix(),
                                                                 split_tokens=64, **kw)),
        "extend": ([extend().segments, extend().members, extend().row_prefix, extend().row_len],
                   lambda **kw: rlt.rlt_paged_extend_attn(pool, 0, qx, pt, extend(), **kw)),
    }[call]
    want = run()
    sizes = [a.nbytes for a in arrays] + [ws, want.nbytes]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        got = run(stream=stream)
        kept = occupy(torch, dev, sizes, 12)
        torch.cuda.synchronize()
        del kept
        assert torch.equal(got, want)
    assert rlt.rlt_get_device_error() == 0


@pytest.mark.parametrize("call", ["decode", "kv8", "append"])
def test_a_captured_stream_that_is_not_the_current_one(dev, call):
    """An output made by the call while another stream than torch's current one is being captured."""
    import torch
    import paged_kv_looped_gb300 as rlt
    import workloads as W
    from helpers import bf16_dev, i32_dev
    case = W.custom(B=2, Hq=4, Hkv=2, D=128, ps=16, seq_lens=[100, 37], seed=5)
    h = W.host_tensors(case)
    pool = rlt.KVPool(bf16_dev(h.k_pool, dev)[None].contiguous(), bf16_dev(h.v_pool, dev)[None].contiguous())
    q, pt, sl = bf16_dev(h.q, dev), i32_dev(case.page_table, dev), i32_dev(case.seq_lens, dev)
    shape = (1, *h.k_pool.shape)
    pool8 = rlt.KV8Pool(*(torch.zeros(shape, dtype=torch.uint8, device=dev).random_(0, 120).view(torch.float8_e4m3fn)
                          for _ in range(2)), *(torch.full(shape[:4], 120, dtype=torch.uint8, device=dev) for _ in range(2)))
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=dev)
    k, pos = torch.randn(2, 2, 128, device=dev).bfloat16(), torch.tensor([100, 37], device=dev)
    run = {"decode": lambda **kw: rlt.rlt_paged_decode_attn(pool, 0, q, pt, sl, 100, workspace=ws, **kw),
           "kv8": lambda **kw: rlt.rlt_paged_decode_attn_kv8(pool8, 0, q, pt, sl, 100, workspace=ws, **kw),
           "append": lambda **kw: rlt.rlt_kv8_append_rope(pool8, 0, k, k, pos, pos, 128, 1e4, q=q, **kw)}[call]
    want = run()
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(other):
        torch.empty_like(want)                                  # (its memory is there to be used again)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side, capture_error_mode="relaxed"):
        with torch.cuda.stream(other):
            got = run(stream=side)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    assert rlt.rlt_get_device_error() == 0
