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
