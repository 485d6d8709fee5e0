"""Rotation at positions far beyond any sequence's: the angle against exact arithmetic (60 digits)."""
import decimal
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

D = decimal.Decimal


def angles(positions, rot, base):
    """pos * base^(-2i/rot) modulo a turn, in radians, from 60-digit arithmetic: float64 [n][rot/2]."""
    with decimal.localcontext() as c:
        c.prec = 60
        x, term, n, pi = D(0), D(1), 0, D(0)
        for a, m in ((5, 16), (239, -4)):                       # pi = 16 atan(1/5) - 4 atan(1/239)
            term, n, x = D(1) / a, 0, D(0)
            while term > D(10) ** -58:
                x += term / (2 * n + 1) * (-1 if n % 2 else 1)
                term /= a * a
                n += 1
            pi += m * x
        freq = [(-D(2 * i) / rot * D(base).ln()).exp() for i in range(rot // 2)]
        return np.array([[float((D(p) * f).remainder_near(2 * pi)) for f in freq] for p in positions])


@pytest.mark.parametrize("d,rot,base", [(64, 64, 10000.0), (128, 128, 500000.0), (128, 62, 10000.0), (64, 48, 100.0)])
def test_angles_of_far_positions(cuda_device, d, rot, base):
    import torch
    import paged_kv_looped_gb300 as rlt
    rlt.rlt_get_device_error()
    pos = [0, 1, -1, 131071, (1 << 31) - 1, -(1 << 36) - 12345, (1 << 40) + 1, 3 ** 30, (1 << 50) - 77, -(1 << 50) + 1]
    n, hq = len(pos), 8
    q = torch.randn(n, hq, d, generator=torch.Generator().manual_seed(rot)).bfloat16()
    pool = rlt.KV8Pool.empty(1, 1, 1, 16, d, cuda_device)
    k = torch.zeros(n, 1, d, dtype=torch.bfloat16, device=cuda_device)
    out = rlt.rlt_kv8_append_rope(pool, 0, k, k.clone(), torch.tensor(pos, device=cuda_device),
                                  torch.arange(n, device=cuda_device), rot, base, q=q.to(cuda_device))
    torch.cuda.synchronize()
    a = angles(pos, rot, base)[:, None]
    x = q.double().numpy()
    h = rot // 2
    ref = x.copy()
    ref[..., :h] = x[..., :h] * np.cos(a) - x[..., h:rot] * np.sin(a)
    ref[..., h:rot] = x[..., h:rot] * np.cos(a) + x[..., :h] * np.sin(a)
    norm = np.hypot(x[..., :h], x[..., h:rot])
    norm = np.concatenate([norm, norm, np.zeros_like(x[..., rot:])], -1)
    # the rounding to bf16, fp32's share of a pair's norm, and the angle: a frequency is kept as a 64-bit fraction of a
    # turn (2^-64 turns = 2^-61.3 rad), made from a product chain of 64-bit mantissas: off by i 2^-62.4 of itself, and
    # i base^(-2i/rot) is at most rot / (2 e ln base) = 5.1 for 128 and 100: 2^-60 rad a position in all
    far = np.abs(np.array([float(p) for p in pos]))[:, None, None] * 2.0 ** -60
    slack = 2.0 ** -8 * np.abs(ref) + (2.0 ** -22 + far) * norm
    err = np.abs(out.double().cpu().numpy() - ref)
    assert np.all(err <= slack), (err / slack).max(axis=(1, 2))
    assert rlt.rlt_get_device_error() == 0
