"""Append to the 8-bit paged cache with rotation, against the 64-bit reference."""
import numpy as np
import pytest

import kv8_ref as R

pytestmark = pytest.mark.gpu

BASE = 10000.0


@pytest.fixture(scope="module")
def dev(cuda_device):
    import paged_kv_looped_gb300 as rlt
    rlt.load()
    rlt.rlt_get_device_error()
    return cuda_device


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def make_pool(rlt, torch, dev, banks, pages, hkv, ps, d, seed):
    g = torch.Generator().manual_seed(seed)
    shape = (banks, pages, hkv, ps, d)
    return rlt.KV8Pool(*(torch.randint(0, 127, shape, generator=g, dtype=torch.uint8).to(dev).view(torch.float8_e4m3fn)
                         for _ in range(2)),
                       *(torch.randint(63, 200, shape[:4], generator=g, dtype=torch.uint8).to(dev) for _ in range(2)))


def run_case(dev, n, hq, hkv, d, rot, ps, *, banks=2, bank=1, skip=0, far=131072, seed=0, fused=True, edit=None,
             outs=True, inplace=False):
    import torch
    import paged_kv_looped_gb300 as rlt
    g = torch.Generator().manual_seed(seed)
    if fused:
        x = torch.randn(n, hq + 2 * hkv, d, generator=g).bfloat16().to(dev)
        q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    else:
        q, k, v = (torch.randn(n, h, d, generator=g).bfloat16().to(dev) for h in (hq, hkv, hkv))
    if edit is not None:
        edit(k, v)
    pages = n // ps + 2
    pool = make_pool(rlt, torch, dev, banks, pages, hkv, ps, d, seed + 1)
    before = [t.view(torch.uint8).clone() for t in (pool.k, pool.v, pool.k_exp, pool.v_exp)]
    slots = torch.randperm(pages * ps, generator=g)[:n]
    gone = torch.randperm(n, generator=g)[:skip]
    slots[gone] = -1
    pos = torch.randint(0, far, (n,), generator=g)
    q_in, k_in, v_in = f64(q), f64(k), f64(v)
    qo = q if inplace else torch.full((n, hq, d), 7.0, dtype=torch.bfloat16, device=dev)
    ko = (k if inplace else torch.full((n, hkv, d), 7.0, dtype=torch.bfloat16, device=dev)) if outs else None
    vo = (v if inplace else torch.full((n, hkv, d), 7.0, dtype=torch.bfloat16, device=dev)) if outs else None
    got = rlt.rlt_kv8_append_rope(pool, bank, k, v, pos.to(dev), slots.to(dev), rot, BASE, q=q, q_out=qo, k_out=ko,
                                  v_out=vo)
    torch.cuda.synchronize()
    assert got is qo and rlt.rlt_get_device_error() == 0
    live = (slots >= 0).numpy()
    slot, p = slots.numpy()[live], pos.numpy()
    page, off = slot // ps, slot % ps
    # queries: bf16 of the rotation
    ref = R.rotate(q_in, p, rot, BASE)
    norm = np.sqrt((q_in ** 2).sum(-1, keepdims=True))      # bounds every pair's norm
    gq = f64(qo)
    assert np.all(np.abs(gq - ref)[live] <= (2.0 ** -8 * np.abs(ref) + 2.0 ** -22 * norm)[live])
    assert np.all(gq[~live] == (q_in[~live] if inplace else 7.0))
    for raw, rotated, x8, xe, held in ((k_in, R.rotate(k_in, p, rot, BASE), pool.k, pool.k_exp, ko),
                                       (v_in, v_in, pool.v, pool.v_exp, vo)):
        e = R.row_exponent(raw)
        got_e = xe[bank].cpu().numpy()[page, :, off].astype(np.int64) - 127
        assert np.array_equal(got_e, e[live])
        want = rotated * np.exp2(-e)[..., None]
        g8 = f64(x8[bank])[page, :, off]
        fine = np.isfinite(raw).all(-1)[live]
        if rotated is raw:
            assert np.array_equal(g8[fine], R.e4m3(want)[live][fine])
        else:
            slack = 2.0 ** -22 * np.sqrt((raw ** 2).sum(-1, keepdims=True)) * np.exp2(-e)[..., None]
            assert np.all((np.abs(g8 - want[live]) <= (R.e4m3_half_step(want) + slack)[live])[fine])
        if held is not None:
            gh = f64(held)
            assert np.array_equal(gh[live][fine], (g8 * np.exp2(got_e)[..., None])[fine])
            assert np.all(gh[~live] == (raw[~live] if inplace else 7.0))
    # every other row of the pool is as it was
    for t, b in zip((pool.k, pool.v, pool.k_exp, pool.v_exp), before):
        a, b = t.view(torch.uint8).cpu().numpy(), b.cpu().numpy()
        mask = np.ones(a.shape[:2] + (a.shape[3],), bool)
        mask[bank, page, off] = False
        a, b = np.moveaxis(a, 3, 2), np.moveaxis(b, 3, 2)
        assert np.array_equal(a[mask], b[mask])
    return pool, qo, ko, vo


@pytest.mark.parametrize("n,hq,hkv,d,rot,ps", [
    (1, 4, 2, 64, 64, 16), (1, 1, 1, 128, 128, 16), (4, 4, 2, 64, 32, 16), (7, 6, 2, 128, 128, 32),
    (33, 16, 16, 128, 64, 16), (64, 16, 16, 128, 128, 64), (65, 5, 1, 128, 62, 256), (31, 3, 3, 64, 2, 48),
    (257, 32, 8, 128, 126, 16), (128, 64, 8, 128, 96, 128), (100, 14, 2, 64, 48, 16), (1031, 8, 1, 128, 128, 16),
    (19, 8, 2, 64, 16, 16), (19, 8, 2, 128, 16, 16),
])
def test_append_matches_reference(dev, n, hq, hkv, d, rot, ps):
    run_case(dev, n, hq, hkv, d, rot, ps, skip=n // 5, seed=n + rot)


@pytest.mark.parametrize("d,rot", [(64, 64), (128, 128), (128, 30)])
def test_separate_arrays_no_rotation_and_in_place(dev, d, rot):
    run_case(dev, 50, 8, 4, d, rot, 16, fused=False, skip=6, seed=3)
    run_case(dev, 50, 8, 4, d, 0, 16, fused=False, skip=6, seed=4)
    run_case(dev, 50, 8, 4, d, rot, 16, fused=False, skip=6, seed=5, inplace=True)
    run_case(dev, 50, 8, 4, d, rot, 16, outs=False, seed=6)


@pytest.mark.parametrize("far", [1, 1 << 20, (1 << 31) - 1])
def test_positions_near_and_far(dev, far):
    # at position 2^31 the reference's own angle is good to 2^31 * 2^-53 = 2^-22 turns' radians
    run_case(dev, 40, 4, 2, 128, 128, 16, far=far, seed=8)


@pytest.mark.parametrize("d,rot", [(64, 64), (128, 128), (128, 50)])
def test_extreme_rows(dev, d, rot):
    def edit(k, v):
        for x in (k, v):
            x[0] = 0.0
            x[1] *= 2.0 ** -60
            x[2] *= 2.0 ** 100
            x[3] = 0.0
            x[3, :, 0] = 2.0 ** -133                       # a denormal row: below the exponent's floor
            x[4, :, 3] = float("inf")
            x[5, :, d - 1] = float("nan")
            x[6] = 448.0
            x[7] = -1.9921875                              # the largest mantissa: 1.9921875 = 2 - 2^-7
    pool, _, ko, vo = run_case(dev, 24, 2, 2, d, rot, 16, seed=9, edit=edit)
    v = f64(vo)
    assert np.isnan(v[5, :, d - 1]).all() and np.isinf(v[4, :, 3]).all()      # 448 * 2^121 is past bf16's largest
    assert (v[4, :, :3] == 0).all() and np.isnan(f64(ko)[5]).any()


def test_bad_slots_counters_and_graph(dev):
    import torch
    import paged_kv_looped_gb300 as rlt
    n, hkv, d, ps = 6, 2, 64, 16
    pool = make_pool(rlt, torch, dev, 2, 2, hkv, ps, d, 1)
    before = [t.view(torch.uint8).clone() for t in (pool.k, pool.v, pool.k_exp, pool.v_exp)]
    k, v, q = (torch.randn(n, hkv, d, device=dev, dtype=torch.bfloat16) for _ in range(3))
    pos = torch.tensor([3, 9, 4, 0, 7, 5], device=dev)
    request = torch.tensor([0, 1, 0, 2, 9, -1], dtype=torch.int32, device=dev)
    written = torch.zeros(2, 3, dtype=torch.int32, device=dev)
    loc = torch.tensor([1, -1, 2, 32, 1 << 40, -5], device=dev)
    out = torch.full_like(q, 3.0)
    rlt.rlt_kv8_append_rope(pool, 1, k, v, pos, loc, d, BASE, q=q, q_out=out, request=request, written=written)
    torch.cuda.synchronize()
    assert rlt.rlt_get_device_error() == rlt.DEVERR_BAD_SLOT
    assert (out[[1, 3, 4, 5]] == 3.0).all() and not (out[[0, 2]] == 3.0).any()
    assert written.tolist() == [[0, 0, 0], [5, 0, 0]]
    changed = (pool.k_exp != before[2]).any(2)              # [bank][page][offset]
    assert not changed[0].any() and changed[1].nonzero().tolist() in ([[0, 1], [0, 2]], [[0, 1]], [[0, 2]], [])
    # a request outside the counters is flagged, its rows are still appended
    rlt.rlt_kv8_append_rope(pool, 0, k[4:5], v[4:5], pos[4:5], loc[:1], d, BASE, request=request[4:5], written=written)
    torch.cuda.synchronize()
    assert rlt.rlt_get_device_error() == rlt.DEVERR_BAD_SLOT and written.tolist() == [[0, 0, 0], [5, 0, 0]]
    # captured and replayed with new contents
    ok = torch.tensor([1, -1, 2, 20, 21, 22], device=dev)
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=s):
        rlt.rlt_kv8_append_rope(pool, 1, k, v, pos, ok, d, BASE, q=q, q_out=out)
    q.normal_(), k.normal_(), pos.add_(100)
    want = make_pool(rlt, torch, dev, 2, 2, hkv, ps, d, 1)
    wout = torch.full_like(q, 3.0)
    graph.replay()
    rlt.rlt_kv8_append_rope(want, 1, k, v, pos, ok, d, BASE, q=q, q_out=wout)
    torch.cuda.synchronize()
    used = ok[ok >= 0]
    assert torch.equal(out[ok >= 0], wout[ok >= 0])
    assert torch.equal(pool.k.view(torch.uint8)[1].transpose(1, 2).reshape(-1, hkv, d)[used],
                       want.k.view(torch.uint8)[1].transpose(1, 2).reshape(-1, hkv, d)[used])
    assert rlt.rlt_get_device_error() == 0


def test_negative_positions_and_other_bases(dev):
    """Positions of any sign, a base below one: the angle is reduced in whole turns either way."""
    import torch
    import paged_kv_looped_gb300 as rlt
    for base in (10000.0, 0.5, 1.0, 500000.0):
        q = torch.randn(9, 2, 64, device=dev).bfloat16()
        k = torch.zeros(9, 1, 64, device=dev).bfloat16()
        pos = torch.tensor([-1, -77, -100000, 0, 1, 5, 63, -4096, 131071], device=dev)
        pool = rlt.KV8Pool.empty(1, 1, 1, 16, 64, dev)
        out = rlt.rlt_kv8_append_rope(pool, 0, k, k, pos, torch.arange(9, device=dev), 64, base, q=q)
        torch.cuda.synchronize()
        ref = R.rotate(f64(q), pos.cpu().numpy(), 64, base)
        norm = np.sqrt((f64(q) ** 2).sum(-1, keepdims=True))
        # a base below one: frequencies up to 2, angles up to 2^18 radians, off by 2^-53 of themselves on both sides
        assert np.all(np.abs(f64(out) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -22 * norm)


def test_binding_refusals(dev):
    import torch
    import paged_kv_looped_gb300 as rlt
    pool = make_pool(rlt, torch, dev, 1, 2, 2, 16, 64, 1)
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device=dev)
    i = torch.zeros(3, dtype=torch.int64, device=dev)
    call = lambda **kw: rlt.rlt_kv8_append_rope(**{**dict(pool=pool, bank=0, k_new=k, v_new=k.clone(), positions=i,   # noqa: E731
                                                          out_loc=i - 1, rot_dim=64, rope_base=BASE), **kw})
    call()
    for err, kw in ((TypeError, dict(k_new=k.cpu())), (TypeError, dict(k_new=k.float())), (ValueError, dict(k_new=k[:2])),
                    (ValueError, dict(v_new=k.transpose(0, 1).contiguous().transpose(0, 1))), (TypeError, dict(positions=i.int())),
                    (ValueError, dict(q_out=k)), (ValueError, dict(q=k[0])), (ValueError, dict(k_out=k[:2])),
                    (ValueError, dict(written=torch.zeros(1, 3, dtype=torch.int32, device=dev))),
                    (ValueError, dict(k_out=torch.zeros(3, 2, 128, dtype=torch.bfloat16, device=dev)[..., ::2])),
                    (rlt.RltError, dict(bank=1)), (rlt.RltError, dict(rot_dim=5)),
                    (rlt.RltError, dict(k_new=torch.zeros(1, 2, 64, dtype=torch.bfloat16, device=dev).expand(3, 2, 64)))):
        with pytest.raises(err):
            call(**kw)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device=dev)
    table, lens = torch.zeros(2, 1, dtype=torch.int32, device=dev), torch.zeros(2, dtype=torch.int32, device=dev)
    dec = lambda **kw: rlt.rlt_paged_decode_attn_kv8(**{**dict(pool=pool, bank=0, q=q, page_table=table, seq_lens=lens,  # noqa: E731
                                                               max_seq_len=16), **kw})
    assert (dec() == 0).all()
    for err, kw in ((TypeError, dict(q=q.cpu())), (TypeError, dict(q=q.half())), (ValueError, dict(q=q[..., :32])),
                    (ValueError, dict(page_table=table[0])), (ValueError, dict(seq_lens=lens[:1])),
                    (ValueError, dict(out=q[:1])), (TypeError, dict(page_table=table.long())),
                    (ValueError, dict(q=q.transpose(0, 1).contiguous().transpose(0, 1))),
                    (rlt.RltError, dict(max_seq_len=5000, split_tokens=16, workspace=torch.empty(16, dtype=torch.uint8, device=dev)))):
        with pytest.raises(err):
            dec(**kw)
    plan = rlt.rlt_plan_prefill([3], 1)
    pre = lambda **kw: rlt.rlt_prefill_attn(**{**dict(q=k, k=k.clone(), v=k.clone(), plan=plan), **kw})   # noqa: E731
    pre()
    for err, kw in ((TypeError, dict(q=k.cpu())), (TypeError, dict(v=k.float())), (ValueError, dict(k=k[:2])),
                    (ValueError, dict(plan=rlt.rlt_plan_prefill([4], 1))), (ValueError, dict(plan=rlt.rlt_plan_prefill([3], 2))),
                    (ValueError, dict(out=k[:2])), (ValueError, dict(lse_out=torch.zeros(3, 4, device=dev))),
                    (rlt.RltError, dict(out=k))):
        with pytest.raises(err):
            pre(**kw)


def test_no_tokens(dev):
    import torch
    import paged_kv_looped_gb300 as rlt
    pool = make_pool(rlt, torch, dev, 1, 1, 2, 16, 64, 1)
    e = torch.empty(0, 2, 64, dtype=torch.bfloat16, device=dev)
    i = torch.empty(0, dtype=torch.int64, device=dev)
    assert rlt.rlt_kv8_append_rope(pool, 0, e, e, i, i, 64, BASE, q=e).shape == (0, 2, 64)
