"""Cross attention and group norm of a network that predicts Gaussians -- CPU
oracle in numpy, fp64 (GlobalSplat page, steps (2) and (3) of its pipeline:
an encoder of the input views, and scene tokens that read them).

TEST INFRASTRUCTURE ONLY: imported by the tests, never by the GPU library, and
it shares no code with it.  Plain formulas over one head or one group at a
time.
"""

from __future__ import annotations

import numpy as np


def seen_keys(batch, nk, lengths=None, mask=None):
    """Truth values [batch][nk]."""
    seen = np.ones((batch, nk), bool)
    for b in range(batch):
        if lengths is not None:
            seen[b, max(0, int(lengths[b])):] = False
        if mask is not None:
            seen[b] &= np.asarray(mask[b]) != 0
    return seen


def attention(q, k, v, scale, seen):
    """q [b][nq][h][d], k and v [b][nk][kv][d] -> out [b][nq][h][d],
    lse [b][h][nq] and P [b][h][nq][nk]."""
    b, nq, h, d = q.shape
    nk, g = k.shape[1], h // k.shape[2]
    out, lse, prob = np.zeros((b, nq, h, d)), np.full((b, h, nq), -np.inf), np.zeros((b, h, nq, nk))
    for i in range(b):
        js = np.nonzero(seen[i])[0]
        if not len(js):
            continue
        for n in range(h):
            s = scale * q[i, :, n] @ k[i, js, n // g].T
            top = s.max(axis=1, keepdims=True)
            e = np.exp(s - top)
            total = e.sum(axis=1, keepdims=True)
            lse[i, n] = (top + np.log(total))[:, 0]
            prob[i, n][:, js] = e / total
            out[i, :, n] = (e / total) @ v[i, js, n // g]
    return out, lse, prob


def attention_grads(q, k, v, scale, seen, out, lse, dout):
    """(dq, dk, dv, dS) from the kept out and lse; dS [b][h][nq][nk]."""
    b, nq, h, d = q.shape
    nk, g = k.shape[1], h // k.shape[2]
    dq, dk, dv, keep = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape), np.zeros((b, h, nq, nk))
    for i in range(b):
        js = np.nonzero(seen[i])[0]
        if not len(js):
            continue
        for n in range(h):
            ki, vi, qi, gi = k[i, js, n // g], v[i, js, n // g], q[i, :, n], dout[i, :, n]
            p = np.exp(scale * qi @ ki.T - lse[i, n][:, None])
            ds = p * (gi @ vi.T - (gi * out[i, :, n]).sum(axis=1, keepdims=True))
            dq[i, :, n] = scale * ds @ ki
            dk[i, js, n // g] += scale * ds.T @ qi
            dv[i, js, n // g] += p.T @ gi
            keep[i, n][:, js] = ds
    return dq, dk, dv, keep


# ---- group norm -------------------------------------------------------------
def _phi(z):
    from math import erfc
    return 0.5 * np.vectorize(erfc, otypes=[np.float64])(-z / 2 ** 0.5)


def act(z, name):
    if name == "relu":
        return np.maximum(z, 0.0)
    if name == "silu":
        return z / (1.0 + np.exp(np.minimum(-z, 700.0)))
    return z * _phi(z) if name == "gelu" else z


def act_slope(z, name):
    if name == "relu":
        return (z > 0) * 1.0
    if name == "silu":
        s = 1.0 / (1.0 + np.exp(np.minimum(-z, 700.0)))
        return s * (1.0 + z * (1.0 - s))
    if name == "gelu":
        return _phi(z) + z * np.exp(-0.5 * z * z) / (2 * np.pi) ** 0.5
    return np.ones_like(z)


def _per_channel(v, c):
    return np.repeat(np.asarray(v, np.float64), c // v.shape[1], axis=1)[:, None]


def group_norm(x, groups, gamma=None, beta=None, activation="none", eps=1e-5):
    """x [n][p][c] -> (mean, rstd) [n][groups], z and y [n][p][c]."""
    n, p, c = x.shape
    mean, rstd = np.zeros((n, groups)), np.zeros((n, groups))
    w = c // groups
    for i in range(n):
        for g in range(groups):
            v = x[i, :, g * w:(g + 1) * w]
            mean[i, g] = v.mean()
            rstd[i, g] = 1.0 / np.sqrt(((v - v.mean()) ** 2).mean() + eps)
    h = (x - _per_channel(mean, c)) * _per_channel(rstd, c)
    z = h * (1.0 if gamma is None else gamma) + (0.0 if beta is None else beta)
    return mean, rstd, z, act(z, activation)


def group_norm_grads(x, mean, rstd, dy, groups, gamma=None, beta=None, activation="none"):
    """(dx, dgamma, dbeta) from the kept mean and rstd: of the terms of
    dy_j/dx_i = gamma_j rstd (delta_ij - 1 / m - h_i h_j / m)."""
    n, p, c = x.shape
    m = p * c // groups
    r = _per_channel(rstd, c)
    h = (x - _per_channel(mean, c)) * r
    gam = np.ones(c) if gamma is None else gamma
    dz = dy * act_slope(h * gam + (0.0 if beta is None else beta), activation)
    u = dz * gam
    total = lambda v: _per_channel(v.reshape(n, p, groups, c // groups).sum(axis=(1, 3)), c)
    return r * (u - total(u) / m - h * total(u * h) / m), (dz * h).sum(axis=(0, 1)), dz.sum(axis=(0, 1))
