"""64-bit reference of the 8-bit cache and its attention (numpy, test infrastructure only).

Shares nothing with the kernels: e4m3 by rounding to a multiple of the step, the rotation with
numpy's cos and sin, attention row by row.
"""
import numpy as np


def e4m3(x):
    """Nearest e4m3 value of float64 x, ties to even, |x| <= 448 (inf -> 448, NaN stays)."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(x), 448.0)
    _, ex = np.frexp(np.maximum(a, 2.0 ** -6))              # a = m 2^ex, m in [1/2, 1)
    step = np.exp2(ex - 4.0)
    with np.errstate(invalid="ignore"):
        return np.copysign(np.round(a / step) * step, x)


def e4m3_half_step(x):
    """Half the distance between e4m3 neighbours around x."""
    a = np.minimum(np.abs(np.asarray(x, np.float64)), 448.0)
    return np.maximum(a * 2.0 ** -4, 2.0 ** -10)


def row_exponent(rows):
    """e (unbiased) of bf16 rows given as float64 [..., D]."""
    a = np.abs(rows).max(-1)
    bad = ~np.isfinite(rows).all(-1)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.where(a > 0, np.maximum(np.frexp(np.where(bad, 1.0, a))[1] - 1 - 7, -64), 0)
    return np.where(bad, 121, e).astype(np.int64)


def rotate(x, positions, rot, base):
    """x float64 [n][heads][D]."""
    out = x.copy()
    half = rot // 2
    if half:
        ang = positions.astype(np.float64)[:, None] * base ** (-2.0 * np.arange(half) / rot)
        c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
        a, b = x[..., :half], x[..., half:rot]
        out[..., :half], out[..., half:rot] = a * c - b * s, b * c + a * s
    return out


def softmax_rows(s, v):
    """(softmax(s) v, lse, softmax(s) |v|) for s [n][m], v [m][D] in float64; no key: 0, -inf, 0."""
    if s.shape[1] == 0:
        z = np.zeros((s.shape[0], v.shape[1]))
        return z, np.full(s.shape[0], -np.inf), z
    top = s.max(1, keepdims=True)
    p = np.exp(s - top)
    total = p.sum(1, keepdims=True)
    p /= total
    with np.errstate(invalid="ignore"):
        return p @ v, (np.log(total) + top)[:, 0], p @ np.abs(v)


def decode(q, k, v, tables, lens, ps, scale):
    """q [B][Hq][D]; k, v [pages][Hkv][ps][D] float64 as held.  -> out, lse, softmax |v|,
    the scores' largest sum of term magnitudes."""
    B, Hq, D = q.shape
    Hkv = k.shape[1]
    out, mag, lse, terms = np.zeros((B, Hq, D)), np.zeros((B, Hq, D)), np.zeros((B, Hq)), np.zeros((B, Hq))
    for b in range(B):
        n = int(lens[b])
        pages = [int(x) for x in tables[b, : -(-n // ps)]]
        pos = np.arange(n)
        ok = np.array([0 <= pages[i // ps] < k.shape[0] for i in pos], bool)
        pg = np.array([pages[i // ps] for i in pos], np.int64)[ok]
        for h in range(Hq):
            g = h // (Hq // Hkv)
            kk, vv = k[pg, g, pos[ok] % ps], v[pg, g, pos[ok] % ps]
            o, l, m = softmax_rows((q[b, h] @ kk.T * scale)[None] if len(kk) else np.zeros((1, 0)),
                                   vv.reshape(-1, D))
            out[b, h], lse[b, h], mag[b, h] = o[0], l[0], m[0]
            if len(kk):
                terms[b, h] = (np.abs(q[b, h]) @ np.abs(kk).T).max() * scale
    return out, lse, mag, terms


def prefill(q, k, v, lens, scale):
    """Causal attention of packed sequences: q [N][Hq][D], k, v [N][Hkv][D] float64 -> out, lse, softmax |v|,
    the scores' largest sum of term magnitudes."""
    N, Hq, D = q.shape
    G = Hq // k.shape[1]
    out, mag, lse, terms = np.zeros((N, Hq, D)), np.zeros((N, Hq, D)), np.zeros((N, Hq)), np.zeros((N, Hq))
    at = 0
    for n in lens:
        n = int(n)
        mask = np.where(np.arange(n)[None, :] > np.arange(n)[:, None], -np.inf, 0.0)
        for h in range(Hq):
            s = q[at:at + n, h] @ k[at:at + n, h // G].T * scale + mask
            if n:
                out[at:at + n, h], lse[at:at + n, h], mag[at:at + n, h] = softmax_rows(s, v[at:at + n, h // G])
                big = np.abs(q[at:at + n, h]) @ np.abs(k[at:at + n, h // G]).T * scale
                terms[at:at + n, h] = np.where(mask == 0, big, 0.0).max(1)
        at += n
    return out, lse, mag, terms


# Tolerances.  An fp32 score of D products is off by at most (D + 4) 2^-24 of its terms' magnitudes' sum
# (`terms` bounds it over a row's keys), and by 2^-24 a few times of itself in the exponent's arithmetic:
# a log-sum-exp by that much, plus 2^-17 for exp2 (2^-22 each), the sum and the logarithm.  Outputs: the one
# rounding to bf16 (2^-8 of the value); each weight is rounded to 11 bits in the 8-bit cache's kernel
# (weight_step 2^-11, fp16) and to 8 in the prompt kernel (2^-8, bf16) and multiplies |v|, so these sum to at
# most weight_step of softmax(s)|v|; a score's error e changes weight and sum by e each.
def score_error(terms, D):
    return (D + 4) * 2.0 ** -24 * terms


def lse_bound(ref, terms, D):
    return 2.0 ** -17 + 2.0 ** -21 * np.abs(ref) + score_error(terms, D)


def attention_bound(ref, mag, terms, weight_step):
    slack = weight_step + 2.0 ** -14 + 2 * score_error(terms, ref.shape[-1])
    return 2.0 ** -8 * np.abs(ref) + slack[..., None] * mag + 1e-30
