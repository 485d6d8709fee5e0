"""Decode over an 8-bit cache that holds value rows of zeros (a null or padding token) beside rows of small values.

A row of zeros is kept with the scale 2^0; it adds its weight to the softmax's sum and nothing to the output, so the
others' weights must not lose bits to it, whatever their scale and however high its score.
"""
import numpy as np
import pytest

import kv8_ref as R
from test_gpu_kv8_decode import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev(cuda_device):
    import paged_kv_looped_gb300 as rlt
    rlt.load()
    rlt.rlt_get_device_error()
    return cuda_device


def put(c, b, i, k0, zero=0x00):
    """Token i of request b: keys k0 in dim 0 and nothing else (a power of two), values of zeros."""
    pg, off = int(c.tables[b, i // c.ps]), i % c.ps
    k8, ke = R.e4m3(np.array([k0])), 127
    import torch
    byte = int(torch.tensor(k8).float().to(torch.float8_e4m3fn).view(torch.uint8)[0])
    kb = torch.zeros_like(c.pool.k.view(torch.uint8)[c.bank, pg, :, off])
    kb[:, 0] = byte
    c.pool.k.view(torch.uint8)[c.bank, pg, :, off] = kb
    c.pool.k_exp[c.bank, pg, :, off] = ke
    c.pool.v.view(torch.uint8)[c.bank, pg, :, off] = zero
    c.pool.v_exp[c.bank, pg, :, off] = 127
    c.k[pg, :, off] = 0.0
    c.k[pg, :, off, 0] = float(k8[0])
    c.v[pg, :, off] = 0.0


def shrink(c, by):
    """Every value of the pool 2^-by of what it was (the scales, not the held numbers)."""
    import torch
    e = c.pool.v_exp[c.bank].int()
    c.pool.v_exp[c.bank] = torch.where(e == 255, e, e - by).to(torch.uint8)
    c.v = c.v * 2.0 ** -by


# The largest weight x scale of the rows that are not zeros is what 2^-28 counts from (scores here spread over
# 2^10 at most, scales over 2^2), so the ordinary bound of 2^-11 a weight holds; outputs stay above 2^-126.
@pytest.mark.parametrize("hq,hkv,d,ps", [(4, 2, 128, 16), (8, 1, 64, 32), (5, 1, 128, 16)])
@pytest.mark.parametrize("small", [0, 20, 30, 45])
@pytest.mark.parametrize("boost", [0.0, 16.0, 40.0])            # of the zero rows' score, in powers of two
def test_rows_of_zeros_among_small_values(dev, hq, hkv, d, ps, small, boost):
    c = Case(dev, [3, 40, 130, 700], hq, hkv, d, ps, seed=hq + small, q_scale=0.5)
    # the score's own unit: scale * q0 * k0 * log2(e) = boost
    c.q[..., 0] = 8.0
    k0 = 2.0 ** np.round(np.log2(max(boost, 1e-30) / 1.4427 / 8 / c.scale)) if boost else 0.0
    shrink(c, small)
    for b, tokens in ((0, [0]), (1, [17, 39]), (2, [0, 1, 64, 129]), (3, [5, 333, 699])):
        for i in tokens:
            put(c, b, i, k0, zero=0x80 if i % 2 else 0x00)      # (a row of negative zeros is one too)
    ref = c.reference()
    for split in (0, 64):
        c.check(*c.run(split_tokens=split), ref)


def test_two_tokens(dev):
    """q = 0, one row of zeros and one of 2^-40: the output is half of it, 2^-41 exactly."""
    import torch
    c = Case(dev, [2], 2, 1, 128, 16, seed=1)
    c.q.zero_()
    put(c, 0, 0, 0.0)
    pg = int(c.tables[0, 0])
    c.pool.v.view(torch.uint8)[c.bank, pg, :, 1] = 0x70          # 128 = 2^7
    c.pool.v_exp[c.bank, pg, :, 1] = 127 - 47
    out, lse = c.run()
    torch.cuda.synchronize()
    assert (out.float() == 2.0 ** -41).all(), out.float().max()
    assert abs(float(lse[0, 0]) - np.log(2)) < 1e-5


def test_rows_of_zeros_behind_large_values(dev):
    """The zero rows' share of the sum stays where values of 2^90 follow them or come before."""
    import torch
    for first in (0, 199):
        c = Case(dev, [200], 2, 1, 64, 16, seed=3)
        c.q.zero_()
        shrink(c, 60)
        for i in range(200):
            if i != first:
                put(c, 0, i, 0.0)
        pg, off = int(c.tables[0, first // 16]), first % 16
        c.pool.v.view(torch.uint8)[c.bank, pg, :, off] = 0x70
        c.pool.v_exp[c.bank, pg, :, off] = 127 + 83
        for split in (0, 64):
            out, lse = c.run(split_tokens=split)
            torch.cuda.synchronize()
            # 2^90 / 200, one rounding to bf16 (2^-8) and some of fp32
            assert (out.double() / 2.0 ** 90 * 200 - 1).abs().max() <= 2.0 ** -8 + 2.0 ** -14
            assert (lse.double() - np.log(200)).abs().max() <= 2.0 ** -16


def test_nothing_but_zeros(dev):
    c = Case(dev, [70, 33], 4, 2, 128, 16, seed=5)
    for b, n in ((0, 70), (1, 33)):
        for i in range(n):
            put(c, b, i, 0.25)
    for split in (0, 32):
        out, lse = c.run(split_tokens=split)
        c.check(out, lse)
        assert (out == 0).all()


def test_rows_of_scale_one_that_are_not_zeros(dev):
    """Values between 128 and 256 have the same scale byte; one small dim beside zeros is enough to count."""
    import torch
    c = Case(dev, [90], 4, 1, 128, 16, seed=6)
    c.pool.v_exp[c.bank][c.pool.v_exp[c.bank] != 255] = 127
    live = c.pool.v_exp[c.bank].cpu().numpy() == 127
    for i in range(0, 90, 7):
        put(c, 0, i, 0.0)
        pg, off = int(c.tables[0, i // 16]), i % 16
        c.pool.v.view(torch.uint8)[c.bank, pg, :, off, i] = 0x71 # 144
    v = c.pool.v.view(torch.uint8)[c.bank].view(torch.float8_e4m3fn).double().cpu().numpy()
    c.v = np.where(live[..., None], v, 0.0)
    for split in (0, 16):
        c.check(*c.run(split_tokens=split))
