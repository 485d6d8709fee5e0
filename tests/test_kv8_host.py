"""Refusals of the 8-bit cache's entry points: host checks that fail before any launch."""
import ctypes

import numpy as np
import pytest

import kv8_ref as R
import paged_kv_looped_gb300 as rlt
from paged_kv_looped_gb300 import build as rlt_build

OK, INVALID, RANGE, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3, 4
A = 1 << 20                                                     # a 16-byte aligned address, never dereferenced


@pytest.fixture(scope="module")
def lib():
    rlt_build.build()
    return rlt.load()


def pool(**kw):
    f = dict(k=A, v=A * 2, k_exp=A * 3, v_exp=A * 4, num_pages=4, num_banks=2, num_kv_heads=2, page_size=16,
             head_dim=128)
    f.update(kw)
    return rlt.rlt_kv8_pool(*(f[n] for n, _ in rlt.rlt_kv8_pool._fields_))


def append(lib, p=None, bank=0, **kw):
    f = dict(q=A * 5, hq=4, qs=512, k=A * 6, ks=256, v=A * 7, vs=256, pos=A * 8, loc=A * 9, n=3, rot=128, base=1e4,
             qo=A * 10, ko=A * 11, vo=A * 12, req=0, wr=0, batch=0)
    f.update(kw)
    return lib.rlt_kv8_append_rope(ctypes.byref(pool() if p is None else p), bank, f["q"], f["hq"], f["qs"], f["k"],
                                   f["ks"], f["v"], f["vs"], f["pos"], f["loc"], f["n"], f["rot"], f["base"], f["qo"],
                                   f["ko"], f["vo"], f["req"], f["wr"], f["batch"], 0)


def decode(lib, p=None, bank=0, **kw):
    f = dict(q=A * 5, hq=4, pt=A * 6, mp=4, sl=A * 7, b=2, msl=50, scale=0.0, out=A * 8, lse=0, ws=0, wsb=0, split=0,
             flags=0)
    f.update(kw)
    return lib.rlt_paged_decode_attn_kv8(ctypes.byref(pool() if p is None else p), bank, f["q"], f["hq"], f["pt"], f["mp"],
                                         f["sl"], f["b"], f["msl"], f["scale"], f["out"], f["lse"], f["ws"], f["wsb"],
                                         f["split"], f["flags"], 0)


POOLS = [(dict(k=0), INVALID), (dict(v_exp=0), INVALID), (dict(k=A + 8), INVALID), (dict(k_exp=A + 1), INVALID),
         (dict(num_pages=-1), INVALID), (dict(num_banks=0), INVALID), (dict(head_dim=96), UNSUPPORTED),
         (dict(page_size=24), UNSUPPORTED), (dict(num_pages=1 << 40), UNSUPPORTED),
         (dict(num_pages=1 << 26), UNSUPPORTED)]


@pytest.mark.parametrize("change,status", POOLS)
def test_pool_refusals(lib, change, status):
    assert append(lib, pool(**change)) == status
    assert decode(lib, pool(**change)) == status


@pytest.mark.parametrize("bank", [-1, 2])
def test_bank_out_of_range(lib, bank):
    assert append(lib, bank=bank) == RANGE and decode(lib, bank=bank) == RANGE


@pytest.mark.parametrize("change", [
    dict(n=-1), dict(rot=-2), dict(rot=3), dict(rot=130), dict(base=0.0), dict(base=float("nan")), dict(k=0), dict(v=0),
    dict(loc=0), dict(pos=0), dict(q=0), dict(qo=0), dict(hq=0), dict(k=A * 6 + 2), dict(qo=A * 10 + 8), dict(loc=A + 4),
    dict(ks=250), dict(ks=252), dict(vs=128), dict(qs=260), dict(qs=500), dict(wr=A, batch=4), dict(wr=A, req=A, batch=0),
    dict(qo=A * 6), dict(qo=A * 5 + 16), dict(ko=A * 7), dict(ko=A * 12), dict(qo=A * 5, qs=1024), dict(vo=A * 6),
    dict(rot=0, pos=0, wr=A, req=A, batch=1), dict(qo=A), dict(ko=A * 2 + 512), dict(vo=A * 3), dict(ko=A * 4 - 16)])
def test_append_refusals(lib, change):
    assert append(lib, **change) == INVALID


def test_append_of_nothing(lib):
    assert append(lib, n=0, k=0, v=0, loc=0, pos=0) == OK


@pytest.mark.parametrize("change,status", [
    (dict(b=-1), INVALID), (dict(msl=-1), INVALID), (dict(hq=0), INVALID), (dict(hq=5), INVALID),
    (dict(hq=18), UNSUPPORTED), (dict(split=8), INVALID), (dict(split=4096), INVALID), (dict(flags=2), INVALID),
    (dict(b=70000), UNSUPPORTED), (dict(q=0), INVALID), (dict(out=0), INVALID), (dict(pt=0), INVALID),
    (dict(mp=0), INVALID), (dict(q=A + 2), INVALID), (dict(scale=float("inf")), INVALID), (dict(ws=A + 4), INVALID),
    (dict(lse=A + 2), INVALID)])
def test_decode_refusals(lib, change, status):
    assert decode(lib, **change) == status


def test_decode_of_nothing(lib):
    assert decode(lib, b=0, q=0, out=0) == OK


def prefill(lib, **kw):
    f = dict(q=A, hq=4, qs=512, k=A * 2, ks=256, v=A * 3, vs=256, hkv=2, d=128, n=300, items=A * 4, ni=3, mt=3, tt=6, scale=0.0,
             out=A * 5, lse=A * 6, flags=0)
    f.update(kw)
    return lib.rlt_prefill_attn(f["q"], f["hq"], f["qs"], f["k"], f["ks"], f["v"], f["vs"], f["hkv"], f["d"], f["n"],
                                f["items"], f["ni"], f["mt"], f["tt"], f["scale"], f["out"], f["lse"], f["flags"], 0)


@pytest.mark.parametrize("change,status", [
    (dict(flags=4), INVALID), (dict(n=-1), INVALID), (dict(ni=-1), INVALID), (dict(mt=-1), INVALID), (dict(tt=-1), INVALID), (dict(hkv=0), INVALID), (dict(hq=5), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(d=96), UNSUPPORTED), (dict(ni=1 << 30), UNSUPPORTED), (dict(n=0), INVALID),
    (dict(q=0), INVALID), (dict(v=0), INVALID), (dict(items=0), INVALID), (dict(out=0), INVALID), (dict(k=A + 2), INVALID),
    (dict(items=A + 2), INVALID), (dict(lse=A + 1), INVALID), (dict(qs=256), INVALID), (dict(ks=260), INVALID),
    (dict(out=A), INVALID), (dict(out=A * 2 - 1024), INVALID),
    (dict(out=A * 5 + 16), INVALID)])
def test_prefill_refusals(lib, change, status):
    assert prefill(lib, **change) == status


def test_prefill_of_nothing(lib):
    assert prefill(lib, ni=0, n=0, q=0, out=0) == OK


@pytest.mark.parametrize("group,step", [(1, 256), (2, 128), (3, 256), (8, 128)])
def test_prefill_plan(lib, group, step):
    lens = [300, 0, 1, 1000, 128, 256]
    plan = rlt.rlt_plan_prefill(lens, group)
    first = np.concatenate([[0], np.cumsum(lens)[:-1]])
    want = {(int(first[b]), n, q0, 0) for b, n in enumerate(lens) for q0 in range(0, n, step)}
    assert plan.num_rows == sum(lens) and len(plan.items) == len(want)
    assert {tuple(int(x) for x in it) for it in plan.items} == want
    assert (np.diff(plan.items[:, 2]) <= 0).all()               # the items with the most keys first
    assert rlt.rlt_plan_prefill([], group).num_items == 0 and rlt.rlt_plan_prefill([0, 0], group).num_items == 0
    with pytest.raises(rlt.RltError):
        rlt.rlt_plan_prefill([5, -1], group)
    with pytest.raises(rlt.RltError):
        rlt.rlt_plan_prefill([1 << 30, 1 << 30], group)
    with pytest.raises(rlt.RltError):
        rlt.rlt_plan_prefill([5], 0)
    tiles = [-(-min(q0 + step, n) // 128) for _, n, q0, _ in want]
    assert plan.max_key_tiles == max(tiles) and plan.total_key_tiles == sum(tiles)
    sizes = np.zeros(4, np.int32)
    sl = np.array(lens, np.int32)
    items = np.zeros((1, 4), np.int32)
    p = lambda a: a.ctypes.data_as(ctypes.c_void_p)              # noqa: E731
    assert lib.rlt_plan_prefill(p(sl), len(lens), group, p(items), 1, p(sizes)) == RANGE
    assert sizes.tolist() == [len(want), sum(lens), max(tiles), sum(tiles)]


def test_reference_number_format():
    """The reference's e4m3 against torch's cast, and its row exponents at the edges."""
    import torch
    x = np.random.default_rng(0).standard_normal(20000) * np.exp2(np.random.default_rng(1).integers(-12, 8, 20000))
    x = np.concatenate([x, [0.0, 448.0, -448.0, 17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -9 * 7.5]])
    x = np.clip(x, -448, 448).astype(np.float32).astype(np.float64)
    assert np.array_equal(R.e4m3(x), torch.from_numpy(x).float().to(torch.float8_e4m3fn).double().numpy())
    rows = np.array([[1.0, 0], [1.99, 1], [2.0, 0], [0, 0], [2.0 ** -133, 0], [3e38, 1], [np.inf, 1], [np.nan, 0]])
    assert R.row_exponent(rows).tolist() == [-7, -7, -6, 0, -64, 120, 121, 121]
    assert np.abs(R.e4m3_half_step(np.array([1.0, 2.0 ** -8, 448]))).tolist() == [2.0 ** -4, 2.0 ** -10, 28.0]
