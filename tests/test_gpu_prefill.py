"""Causal attention over packed prompts, against the 64-bit reference."""
import numpy as np
import pytest

import kv8_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev(cuda_device):
    import paged_kv_looped_gb300 as rlt
    rlt.load()
    rlt.rlt_get_device_error()
    return cuda_device


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def rows(torch, dev, n, hq, hkv, d, seed, fused=True, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    if fused:
        x = (torch.randn(n, hq + 2 * hkv, d, generator=g) * scale).bfloat16().to(dev)
        return x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    return tuple((torch.randn(n, h, d, generator=g) * scale).bfloat16().to(dev) for h in (hq, hkv, hkv))


def check(out, lse, q, k, v, lens, scale):
    o, l, mag, terms = R.prefill(f64(q), f64(k), f64(v), lens, scale)
    n = sum(lens)
    go, gl = f64(out)[:n], f64(lse)[:n]
    o, l, mag, terms = o[:n], l[:n], mag[:n], terms[:n]
    assert np.isfinite(go).all()
    assert np.all(np.abs(gl - l) <= R.lse_bound(l, terms, o.shape[-1])), np.abs(gl - l).max()
    assert np.all(np.abs(go - o) <= R.attention_bound(o, mag, terms, 2.0 ** -8)), np.abs(go - o).max()


def run(dev, lens, hq, hkv, d, *, seed=0, fused=True, behind=0, scale=0.0, spread=1.0):
    import torch
    import paged_kv_looped_gb300 as rlt
    n = sum(lens) + behind
    q, k, v = rows(torch, dev, n, hq, hkv, d, seed, fused, spread)
    out = torch.full((n, hq, d), 9.0, dtype=torch.bfloat16, device=dev)
    lse = torch.full((n, hq), 9.0, device=dev)
    plan = rlt.rlt_plan_prefill(lens, hq // hkv)
    got = rlt.rlt_prefill_attn(q, k, v, plan, out=out, lse_out=lse, scale=scale)
    torch.cuda.synchronize()
    assert got is out and rlt.rlt_get_device_error() == 0
    check(out, lse, q, k, v, lens, scale or 1 / np.sqrt(d))
    assert (out[sum(lens):] == 9).all() and (lse[sum(lens):] == 9).all()


@pytest.mark.parametrize("n", [1, 2, 63, 127, 128, 129, 255, 256, 257, 384, 385, 640])
@pytest.mark.parametrize("hq,hkv,d", [(2, 2, 128), (4, 2, 64), (3, 1, 128), (1, 1, 64)])
def test_one_sequence(dev, n, hq, hkv, d):
    run(dev, [n], hq, hkv, d, seed=n)


@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 64), (16, 16, 128), (8, 1, 128), (6, 2, 128), (20, 4, 64), (14, 2, 128),
                                      (64, 8, 128)])
def test_packed_sequences(dev, hq, hkv, d):
    run(dev, [100, 0, 1, 300, 128, 5, 0, 257, 64], hq, hkv, d, seed=hq, behind=37)


def test_long_and_scales(dev):
    run(dev, [2500], 2, 1, 128, seed=1)
    run(dev, [1900, 300], 2, 2, 64, seed=2, fused=False)
    run(dev, [700], 4, 2, 128, seed=3, scale=0.03)
    run(dev, [700], 4, 2, 128, seed=4, spread=4.0)              # peaked weights: the running maximum moves
    run(dev, [900], 1, 1, 128, seed=5, spread=0.01)


def test_rising_scores(dev):
    """Each key tile beats the one before by far: every tile moves the reference maximum."""
    import torch
    import paged_kv_looped_gb300 as rlt
    q, k, v = rows(torch, dev, 1000, 2, 2, 128, 6, fused=False)
    q.fill_(0.0), k.fill_(0.0)
    q[..., 0] = 8.0
    k[..., 0] = torch.arange(1000, device=dev)[:, None].bfloat16() * 0.125
    lse = torch.empty(1000, 2, device=dev)
    out = rlt.rlt_prefill_attn(q, k, v, rlt.rlt_plan_prefill([1000]), lse_out=lse, scale=1.0)
    torch.cuda.synchronize()
    check(out, lse, q, k, v, [1000], 1.0)
    k.neg_()
    out = rlt.rlt_prefill_attn(q, k, v, rlt.rlt_plan_prefill([1000]), lse_out=lse, scale=1.0)
    torch.cuda.synchronize()
    check(out, lse, q, k, v, [1000], 1.0)


def test_first_keys_of_score_minus_infinity(dev):
    """Scores of -inf (an infinite key component) weigh nothing, also where a row's first tiles hold nothing else."""
    import torch
    import paged_kv_looped_gb300 as rlt
    q, k, v = rows(torch, dev, 400, 2, 1, 64, 13, fused=False)
    q[..., 0] = 1.0
    k[:200, :, 0] = float("-inf")
    k[200:, :, 0] = -3000.0                                     # finite, and far below anything's first guess
    lse = torch.empty(400, 2, device=dev)
    out = rlt.rlt_prefill_attn(q, k, v, rlt.rlt_plan_prefill([400], 2), lse_out=lse)
    torch.cuda.synchronize()
    assert torch.isneginf(lse[:200]).all()
    # rows 200..: as if the first 200 keys were not there
    kk, vv = f64(k)[200:], f64(v)[200:]
    o, l, mag, terms = R.prefill(f64(q)[200:], kk, vv, [200], 1 / 8)
    assert np.all(np.abs(f64(lse)[200:] - l) <= R.lse_bound(l, terms, 64))
    assert np.all(np.abs(f64(out)[200:] - o) <= R.attention_bound(o, mag, terms, 2.0 ** -8))
    assert rlt.rlt_get_device_error() == 0


def test_neighbours_and_rows_behind_hold_anything(dev):
    import torch
    import paged_kv_looped_gb300 as rlt
    lens, n = [70, 50, 200], 400
    q, k, v = rows(torch, dev, n, 4, 2, 128, 7, fused=False)
    for x in (q, k, v):
        x[70:120] = float("nan")
        x[320:] = float("inf")
    out = torch.full((n, 4, 128), 9.0, dtype=torch.bfloat16, device=dev)
    lse = torch.full((n, 4), 9.0, device=dev)
    rlt.rlt_prefill_attn(q, k, v, rlt.rlt_plan_prefill(lens, 2), out=out, lse_out=lse)
    torch.cuda.synchronize()
    keep = list(range(70)) + list(range(120, 320))
    check(out[keep], lse[keep], q[keep], k[keep], v[keep], [70, 200], 1 / np.sqrt(128))
    assert torch.isnan(out[70:120]).all() and torch.isnan(lse[70:120]).all()
    assert (out[320:] == 9).all() and (lse[320:] == 9).all()


@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 128), (3, 3, 64), (3, 1, 128), (8, 2, 64)])
def test_values_a_query_may_not_see(dev, hq, hkv, d):
    """Infinities and NaN in V reach exactly the queries at or behind them (as the formula has it: a NaN every one of
    them, an infinity unless it meets its opposite); NaN in K of later keys reaches nobody before."""
    import torch
    import paged_kv_looped_gb300 as rlt
    lens = [300, 90, 260]
    n = sum(lens)
    q, k, v = rows(torch, dev, n, hq, hkv, d, 11, fused=False)
    plan = rlt.rlt_plan_prefill(lens, hq // hkv)
    lse, clean_lse = torch.empty(n, hq, device=dev), torch.empty(n, hq, device=dev)
    clean = rlt.rlt_prefill_attn(q, k, v, plan, lse_out=clean_lse)
    odd = [(70, 3, float("nan")), (200, d - 1, float("inf")), (200, 5, float("-inf")), (299, 0, float("nan")),
           (300, 7, float("inf")), (389, 7, float("-inf")), (640, 9, float("nan"))]
    want = clean.clone()
    first = [0, 300, 390]
    for row, c, x in odd:
        v[row, 0, c] = x
        seq = max(i for i in range(3) if first[i] <= row)
        want[row:first[seq] + lens[seq], :hq // hkv, c] = float("nan") if x != x or (row, c) == (389, 7) else x
    out = rlt.rlt_prefill_attn(q, k, v, plan, lse_out=lse)
    torch.cuda.synchronize()
    assert torch.equal(torch.isnan(out), torch.isnan(want))
    same = ~torch.isnan(want)
    assert torch.equal(torch.isinf(out[same]), torch.isinf(want[same])) and torch.equal(out[same].sign(), want[same].sign())
    fin = torch.isfinite(want)
    assert torch.equal(out[fin], clean[fin]) and torch.equal(lse, clean_lse)
    v.copy_(torch.where(torch.isfinite(v), v, 0.0))
    base = rlt.rlt_prefill_attn(q, k, v, plan)
    k[250] = float("nan")
    out = rlt.rlt_prefill_attn(q, k, v, plan, lse_out=lse)
    torch.cuda.synchronize()
    keep = list(range(250)) + list(range(300, n))
    assert torch.equal(out[keep], base[keep]) and torch.isnan(out[250:300]).all() and torch.isnan(lse[250:300]).all()
    assert rlt.rlt_get_device_error() == 0


def test_many_items(dev):
    """More work than the GPU holds at once, of every size: blocks hand their work over to running ones."""
    import torch
    import paged_kv_looped_gb300 as rlt
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 400, (300,), generator=g).tolist()
    for hq, hkv, d in ((8, 2, 128), (3, 1, 64)):
        n = sum(lens)
        q, k, v = rows(torch, dev, n, hq, hkv, d, 12)
        plan = rlt.rlt_plan_prefill(lens, hq // hkv).to(dev)
        lse = torch.empty(n, hq, device=dev)
        out = [rlt.rlt_prefill_attn(q, k, v, plan, lse_out=lse) for _ in range(5)]
        torch.cuda.synchronize()
        assert all(torch.equal(o, out[0]) for o in out[1:])
        assert rlt.rlt_get_device_error() == 0
        check(out[0], lse, q, k, v, lens, 1 / np.sqrt(d))


def test_streams_and_graph(dev):
    import torch
    import paged_kv_looped_gb300 as rlt
    a, b = rows(torch, dev, 900, 8, 2, 128, 8), rows(torch, dev, 700, 4, 4, 64, 9)
    pa, pb = rlt.rlt_plan_prefill([500, 400], 4).to(dev), rlt.rlt_plan_prefill([700], 1).to(dev)
    la, lb = torch.empty(900, 8, device=dev), torch.empty(700, 4, device=dev)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = [(rlt.rlt_prefill_attn(*a, pa, lse_out=la, stream=s1), rlt.rlt_prefill_attn(*b, pb, lse_out=lb, stream=s2))
            for _ in range(4)]
    torch.cuda.synchronize()
    check(outs[0][0], la, *a, [500, 400], 1 / np.sqrt(128))
    check(outs[0][1], lb, *b, [700], 1 / np.sqrt(64))
    for x, y in outs:
        assert torch.equal(x, outs[0][0]) and torch.equal(y, outs[0][1])
    out = torch.empty_like(outs[0][0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rlt.rlt_prefill_attn(*a, pa, out=out, lse_out=la)
        rlt.rlt_prefill_attn(*a, pa, out=out, lse_out=la, early_start=True)
    for x in a:
        x.mul_(-0.5)
    graph.replay()
    torch.cuda.synchronize()
    check(out, la, *a, [500, 400], 1 / np.sqrt(128))


def test_plan_of_other_sequences(dev):
    """Items that point outside the rows are skipped and flagged."""
    import torch
    import paged_kv_looped_gb300 as rlt
    q, k, v = rows(torch, dev, 300, 2, 2, 64, 10)
    plan = rlt.rlt_plan_prefill([300], 1).to(dev)
    bad = torch.tensor([[0, 301, 0, 0], [-1, 5, 0, 0], [10, 20, 20, 0], [10, 0, 0, 0], [0, 300, 64, 0],
                        [1 << 30, 1 << 30, 0, 0]], dtype=torch.int32, device=dev)
    plan.dev, plan.num_items = bad, 6
    out = torch.full((300, 2, 64), 9.0, dtype=torch.bfloat16, device=dev)
    rlt.rlt_prefill_attn(q, k, v, plan, out=out)
    torch.cuda.synchronize()
    assert rlt.rlt_get_device_error() == rlt.DEVERR_BAD_LEN and (out == 9).all()


@pytest.mark.parametrize("hq,hkv,d,ps", [(8, 2, 128, 16), (4, 2, 64, 32), (6, 2, 128, 16)])
def test_prompt_then_tokens(dev, hq, hkv, d, ps):
    """The three operators as a server runs them: the prompts' rows are rotated and appended, attended to as the
    cache holds them, then two tokens per request are appended and decoded over the cache."""
    import torch
    import paged_kv_looped_gb300 as rlt
    lens, base = [130, 1, 77, 300], 10000.0
    B, N, width = len(lens), sum(lens), 22
    g = torch.Generator().manual_seed(5)
    pool = rlt.KV8Pool.empty(2, B * width, hkv, ps, d, dev)
    for x in (pool.k, pool.v):
        x.view(torch.uint8).fill_(0x7F)
    table = torch.randperm(B * width, generator=g).view(B, width).to(dev)
    slot = lambda b, p: table[b, p // ps] * ps + p % ps          # noqa: E731
    owner = torch.tensor(np.repeat(np.arange(B), lens), device=dev)
    pos = torch.tensor(np.concatenate([np.arange(n) for n in lens]), device=dev)
    x = torch.randn(N, hq + 2 * hkv, d, generator=g).bfloat16().to(dev)
    k_held, v_held = (torch.empty(N, hkv, d, dtype=torch.bfloat16, device=dev) for _ in range(2))
    q_rot = rlt.rlt_kv8_append_rope(pool, 1, x[:, hq:hq + hkv], x[:, hq + hkv:], pos, slot(owner, pos), d, base,
                                    q=x[:, :hq], k_out=k_held, v_out=v_held)
    lse = torch.empty(N, hq, device=dev)
    out = rlt.rlt_prefill_attn(q_rot, k_held, v_held, rlt.rlt_plan_prefill(lens, hq // hkv), lse_out=lse)
    torch.cuda.synchronize()
    check(out, lse, q_rot, k_held, v_held, lens, 1 / np.sqrt(d))
    # the last prompt row, decoded over the cache, is the prompt attention's last row up to the weights' roundings
    last = torch.tensor(np.cumsum(lens) - 1, device=dev)
    seq = torch.tensor(lens, dtype=torch.int32, device=dev)
    t32 = table.int().contiguous()
    again = rlt.rlt_paged_decode_attn_kv8(pool, 1, q_rot[last].contiguous(), t32, seq, max(lens))
    held = [[k_held[owner == b], v_held[owner == b]] for b in range(B)]
    for step in range(3):
        if step:
            y = torch.randn(B, hq + 2 * hkv, d, generator=g).bfloat16().to(dev)
            p = seq.long()
            kn, vn = (torch.empty(B, hkv, d, dtype=torch.bfloat16, device=dev) for _ in range(2))
            qn = rlt.rlt_kv8_append_rope(pool, 1, y[:, hq:hq + hkv], y[:, hq + hkv:], p,
                                         slot(torch.arange(B, device=dev), p), d, base, q=y[:, :hq], k_out=kn, v_out=vn)
            seq += 1
            again = rlt.rlt_paged_decode_attn_kv8(pool, 1, qn, t32, seq, max(lens) + step)
            held = [[torch.cat([h[0], kn[b:b + 1]]), torch.cat([h[1], vn[b:b + 1]])] for b, h in enumerate(held)]
            q_now = qn
        else:
            q_now = q_rot[last]
        torch.cuda.synchronize()
        for b in range(B):
            kk, vv, qq = f64(held[b][0]), f64(held[b][1]), f64(q_now[b])
            for h in range(hq):
                kh, vh = kk[:, h // (hq // hkv)], vv[:, h // (hq // hkv)]
                o, _, m = R.softmax_rows(qq[h][None] @ kh.T / np.sqrt(d), vh)
                terms = np.array((np.abs(qq[h]) @ np.abs(kh).T).max() / np.sqrt(d))
                assert np.all(np.abs(f64(again[b, h]) - o[0]) <= R.attention_bound(o[0], m[0], terms, 2.0 ** -11))
    assert rlt.rlt_get_device_error() == 0
