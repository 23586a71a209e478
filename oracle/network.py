"""Operators of a network head that predicts Gaussians -- CPU oracle in numpy,
fp64 (GlobalSplat page, step (4) of its pipeline: heads that turn tokens into
Gaussian parameters).

TEST INFRASTRUCTURE ONLY: imported by the tests, never by the GPU library, and
it shares no code with it.  Plain formulas, no blocking, no rounding except
where a format is the point.
"""

from __future__ import annotations

import math

import numpy as np

_erf = np.vectorize(math.erf, otypes=[np.float64])
_erfc = np.vectorize(math.erfc, otypes=[np.float64])


# ---- root-mean-square norm --------------------------------------------------
def rms_norm(x, residual=None, gamma=None, eps=1e-6):
    """(s, rstd, y) of s = x + residual, y = s * rstd * gamma."""
    s = np.asarray(x, np.float64) + (0.0 if residual is None else np.asarray(residual, np.float64))
    rstd = 1.0 / np.sqrt(np.mean(s * s, axis=1) + eps)
    g = np.ones(s.shape[1]) if gamma is None else np.asarray(gamma, np.float64)
    return s, rstd, s * rstd[:, None] * g


def rms_norm_grads(s, rstd, dy, gamma=None, dsum=None):
    """(dx, dgamma); every term of the Jacobian written out:
    dy_j/ds_i = gamma_j (rstd delta_ij - rstd^3 s_i s_j / n)."""
    s, dy, rstd = np.asarray(s, np.float64), np.asarray(dy, np.float64), np.asarray(rstd, np.float64)[:, None]
    n = s.shape[1]
    w = dy * (1.0 if gamma is None else np.asarray(gamma, np.float64))
    dx = rstd * w - rstd ** 3 * s * (w * s).sum(axis=1, keepdims=True) / n
    if dsum is not None:
        dx = dx + np.asarray(dsum, np.float64)
    return dx, (dy * s * rstd).sum(axis=0)


# ---- 8-bit blocks -----------------------------------------------------------
def e4m3_table():
    """The value of every e4m3 code (127 and 255: NaN)."""
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10)
        out[c] = math.nan if c & 127 == 127 else -v if c & 128 else v
    return out


def mxfp8_quantize(v):
    """[m][n] -> (codes uint8 [m][n], scale bytes uint8 [m][n / 32])."""
    v = np.asarray(v, np.float64)
    m, n = v.shape
    b = v.reshape(m, n // 32, 32)
    codes, scales = np.zeros(b.shape, np.uint8), np.zeros(b.shape[:2], np.uint8)
    table = e4m3_table()
    mags = table[:127]
    for i in np.ndindex(b.shape[:2]):
        blk = b[i]
        if not np.isfinite(blk).all():
            scales[i] = 255
            continue
        top = np.abs(blk).max()
        e = -127
        while top > 448.0 * 2.0 ** e:
            e += 1
        scales[i] = e + 127
        u = np.abs(blk) / 2.0 ** e
        hi = np.clip(np.searchsorted(mags, u), 1, 126)
        lo = hi - 1
        dl, dh = u - mags[lo], mags[hi] - u
        up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))          # ties to the even code
        codes[i] = np.where(up, hi, lo).astype(np.uint8) | (np.signbit(blk).astype(np.uint8) << 7)
    return codes.reshape(m, n), scales


def mxfp8_value(codes, scales):
    f = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127.0))
    return e4m3_table()[codes] * np.repeat(f, 32, axis=1)


# ---- linear layer -----------------------------------------------------------
def activate(z, act):
    if act == "relu":
        return np.where(z < 0, 0.0, z)
    if act == "silu":
        return z / (1.0 + np.exp(-z))
    if act == "gelu":
        return z * 0.5 * _erfc(-z / math.sqrt(2.0))
    return z


def slope(z, act):
    if act == "relu":
        return (z > 0).astype(np.float64)
    if act == "silu":
        s = 1.0 / (1.0 + np.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    if act == "gelu":
        return 0.5 * _erfc(-z / math.sqrt(2.0)) + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    return np.ones_like(z)


def linear(x, w, bias=None, act="none", residual=None):
    """(z, y), both [m][n]."""
    z = np.asarray(x, np.float64) @ np.asarray(w, np.float64).T
    if bias is not None:
        z = z + np.asarray(bias, np.float64)
    y = activate(z, act)
    return z, y if residual is None else y + np.asarray(residual, np.float64)


def linear_grads(x, w, z, dy, act="none"):
    """(dx, dw, db, dz) for dy [m][n]."""
    dz = np.asarray(dy, np.float64) * (slope(np.asarray(z, np.float64), act) if act != "none" else 1.0)
    return dz @ np.asarray(w, np.float64), dz.T @ np.asarray(x, np.float64), dz.sum(axis=0), dz


# ---- orthogonalised update --------------------------------------------------
COEFFS = (3.4445, -4.7750, 2.0315)


def orthogonalize(u, steps=5, coeffs=COEFFS, eps=1e-7):
    """Newton-Schulz on one matrix through its singular values: an iteration
    maps each to a s + b s^3 + c s^5 and leaves the singular vectors."""
    u = np.asarray(u, np.float64)
    a, b, c = coeffs
    p, s, q = np.linalg.svd(u, full_matrices=False)
    s = s / (math.sqrt((u * u).sum()) + eps)
    for _ in range(steps):
        s = a * s + b * s ** 3 + c * s ** 5
    return (p * s) @ q


def muon_step(grad, momentum, weight, lr, beta, weight_decay, scale, nesterov=True, **kw):
    """(momentum, weight) after one step on one matrix."""
    g = np.asarray(grad, np.float64)
    mom = beta * np.asarray(momentum, np.float64) + g
    o = orthogonalize(g + beta * mom if nesterov else mom, **kw)
    return mom, np.asarray(weight, np.float64) * (1.0 - lr * weight_decay) - lr * scale * o
