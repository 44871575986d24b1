"""Plain 64-bit forms of the attention operators and the error bounds their tests use.

u = 2^-24 is fp32's unit roundoff, 2^-8 bf16's.  Sums of n terms are bounded
by 6 sqrt(n) u (rounding errors of random sign, six standard deviations)."""
import math

import numpy as np

U = 2.0 ** -24
UB = 2.0 ** -8


def attention(q, k, v, scale, valid=None):
    """q [N][Tq][Hq][D], k and v [N][Tk][Hkv][D] (float64), valid [N][Tk] or None.

    Returns out, lse and, for the bounds, wabs = sum_j p_j |v_j| and the
    largest sum of |scale q k| of each row."""
    N, Tq, Hq, D = q.shape
    Hkv = k.shape[2]
    out, wabs = np.zeros_like(q), np.zeros_like(q)
    lse = np.full((N, Hq, Tq), -np.inf)
    mag = np.zeros((N, Hq, Tq))
    for n in range(N):
        keep = np.arange(k.shape[1]) if valid is None else np.flatnonzero(valid[n])
        if keep.size == 0:
            continue
        for h in range(Hq):
            kk, vv = k[n, keep, h * Hkv // Hq], v[n, keep, h * Hkv // Hq]
            s = scale * (q[n, :, h] @ kk.T)
            mag[n, h] = scale * (np.abs(q[n, :, h]) @ np.abs(kk).T).max(axis=1)
            m = s.max(axis=1, keepdims=True)
            p = np.exp(s - m)
            l = p.sum(axis=1, keepdims=True)
            out[n, :, h] = p @ vv / l
            wabs[n, :, h] = p @ np.abs(vv) / l
            lse[n, h] = (m + np.log(l))[:, 0]
    return out, lse, wabs, mag


def score_error(D, mag):
    """Bound of one score's error: its fp32 dot product, the products' and the
    running maximum's rounding, and 2^x of the special function unit (2^-22)."""
    return U * (6 * math.sqrt(D) + 8) * mag + 2.0 ** -21


def out_bound(out, wabs, mag, D, Tk, bf16):
    ds = score_error(D, mag).transpose(0, 2, 1)[..., None]
    b = wabs * (2 * ds + (6 * math.sqrt(Tk) + 16) * U) + 1e-30
    if bf16:   # the weights enter the tensor cores as bf16; the output is rounded once
        b = b + UB * wabs + UB * np.abs(out)
    return b


def lse_bound(lse, mag, D, Tk):
    finite = np.where(np.isfinite(lse), np.abs(lse), 0.0)
    return score_error(D, mag) + (6 * math.sqrt(Tk) + 16) * U + 4 * U * finite


def frequencies(pairs, base=10000.0, rule=0, factor=1.0, original=0.0):
    if rule == 2:
        base = base * factor ** (pairs / (pairs - 1.0))
    f = base ** (-np.arange(pairs) / pairs)
    magnitude = 1.0
    if rule == 1:
        f = f / factor
    if rule == 3:
        turns = original * f / (2 * np.pi)
        keep = np.clip((turns - 1.0) / 31.0, 0.0, 1.0)
        f = f * keep + f / factor * (1.0 - keep)
        magnitude = 0.1 * math.log(factor) + 1.0
    return f, magnitude


def rotate(x, pos, rot, mode, axes, f, magnitude=1.0, inverse=False):
    """x [tokens][heads][D] float64, pos [axes][tokens]; returns y and |a| + |b| of each element's pair."""
    y, mag = x.copy(), np.abs(x)
    angle = np.concatenate([pos[a][:, None] * f[None, :] for a in range(axes)], axis=1)[:, None, :]
    c, s = magnitude * np.cos(angle), magnitude * np.sin(angle) * (-1 if inverse else 1)
    ia, ib = (np.arange(rot // 2), np.arange(rot // 2) + rot // 2) if mode == 0 else \
        (2 * np.arange(rot // 2), 2 * np.arange(rot // 2) + 1)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    mag[..., ia] = mag[..., ib] = (np.abs(a) + np.abs(b)) * magnitude
    return y, mag


def rms_norm(x, weight, eps):
    y = x / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps)
    return y if weight is None else y * weight
