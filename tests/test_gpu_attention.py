"""GPU parity of cross attention (gs_attention_fwd, gs_attention_bwd) against
the fp64 oracle.

Tolerances.  u is the unit roundoff of the type (2^-24 fp32, 2^-11 fp16, 2^-8
bf16) and e = 2^-24.
* A score S_ij is a sum of d products in fp32: off by at most (d + 20) e of the
  sum of their magnitudes, times scale; the exponential's argument by a few
  roundings of numbers of its size.  Together r_ij = (d + 20) e scale sum |q k| + 4 e (4 + |S_ij| + |lse_i|)
  is the relative error of P_ij before it is rounded to the type.
* out: every P rounded once (u), its normaliser off by the largest r, sums of
  nk terms in fp32: (u + 3 max_j r_ij + 2 (nk + 32) e) sum_j P |v|, and u |out|.  fp16
  P below its normal range are off by up to 2^-25 of a maximum between 1 and 2^8.
* gradients: dS_ij is off by (u + r_ij) of itself and P_ij times the error
  (d + 20) e (sum |dout v| + sum |dout out|) of what it multiplies; then products as above.
  fp16 rounds dS relative to its column's largest at 2^-35 or better where it is small.
"""

import numpy as np
import pytest
import torch

from gaussian_splatting_tile_amd import binding as B
from oracle import attention as A
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

T = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 1e-36, "f16": 2.0 ** -24, "bf16": 1e-36}
E = 2.0 ** -24


def _np(t):
    return t.detach().float().cpu().double().numpy()


def _make(rng, shape, t, scale=1.0):
    return torch.from_numpy(rng.standard_normal(shape) * scale).to(T[t]).cuda()


def _place(x, odd, heads_first=False):
    """x [b][n][h][d] as a view into a larger buffer of 77s: rows, heads and
    batches apart (`odd`: by odd numbers of elements from an odd address), or
    stored [b][h][n][d]."""
    b, n, h, d = x.shape
    if heads_first:
        size = (b, h, n, d)
        pad = (1, 3, 5) if odd else (0, 0, 0)
    else:
        size = (b, n, h, d)
        pad = (7, 5, 3) if odd else (0, 16, 8)
    s2 = size[3] + pad[2]
    s1 = size[2] * s2 + pad[1]
    s0 = size[1] * s1 + pad[0]
    buf = torch.full((max(1, size[0] * s0) + 16,), 77.0, device="cuda").to(x.dtype)
    v = buf.as_strided(size, (s0, s1, s2, 1), 8 if not odd else 3)
    v = v.transpose(1, 2) if heads_first else v
    v.copy_(x)
    return v, buf


def _untouched(v, buf):
    """Nothing outside the view v of buf was written."""
    v.fill_(77.0)
    return bool((buf.float() == 77.0).all())


def _ws(n):
    """A workspace of n bytes and a guard behind it."""
    ws = torch.full((int(n) + 256,), 0x5A, dtype=torch.uint8, device="cuda")
    return ws[:int(n)] if n else None, ws


def _guarded(ws, n):
    assert bool((ws[int(n):] == 0x5A).all()), "write past the workspace"


def _close(got, want, tol, what):
    got, want = np.asarray(got), np.asarray(want)
    tol = np.broadcast_to(tol, want.shape)
    assert got.shape == want.shape, what
    d = np.abs(got - want)
    same = (got == want)                                   # infinities
    bad = ~((d <= tol) | same)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(np.where(same, 0, d / np.maximum(tol, 1e-300))):.3g} x tolerance " \
                          f"at {np.unravel_index(np.argmax(np.where(bad, np.nan_to_num(d, nan=np.inf), -1)), d.shape)}"


def _run(q, k, v, dout, t, lengths=None, mask=None, scale=None, odd=False, heads_first=False, want=("dq", "dk", "dv"), poison=False):
    """Forward and backward against the oracle."""
    b, nq, h, d = q.shape
    nk, kv = k.shape[1:3]
    g = h // kv
    scale = d ** -0.5 if scale is None else scale
    seen = A.seen_keys(b, nk, None if lengths is None else lengths.cpu().numpy(), None if mask is None else mask.cpu().numpy())
    Q, K, V, D = _np(q), _np(k), _np(v), _np(dout)
    if poison:                                             # states that are not attended hold anything
        bad = torch.from_numpy(~seen).cuda()
        k, v = k.clone(), v.clone()
        k[bad], v[bad] = float("nan"), float("inf")
    K[~seen] = V[~seen] = 0.0
    (qv, _), (kv_, _), (vv, _), (dv_, _) = (_place(x, odd, heads_first) for x in (q, k, v, dout))
    out, ob = _place(torch.full_like(q, 5.0), odd, heads_first)
    lse = torch.full((b, h, nq), 5.0, device="cuda")
    a = B.attention_struct(qv, kv_, vv, out, lse=lse, kv_lengths=lengths, kv_mask=mask, scale=scale)
    nb = B.attention_fwd_workspace_bytes(a)
    ws, whole = _ws(nb)
    B.attention_fwd(a, ws)
    torch.cuda.synchronize()
    _guarded(whole, nb)
    out64, lse64, P = A.attention(Q, K, V, scale, seen)
    kr, vr = np.repeat(K, g, 2), np.repeat(V, g, 2)
    mags = scale * np.einsum("bihd,bjhd->bhij", np.abs(Q), np.abs(kr))
    S = scale * np.einsum("bihd,bjhd->bhij", Q, kr)
    r = (d + 20) * E * mags + 4 * E * (4 + np.abs(S) + np.abs(np.nan_to_num(lse64, neginf=0.0))[..., None])
    r = np.where(seen[:, None, None, :], r, 0.0)
    top = r.max(axis=3, initial=0.0, keepdims=True)
    weight = np.einsum("bhij,bjhd->bihd", P, np.abs(vr))
    low = np.einsum("bj,bjhd->bhd", seen * 1.0, np.abs(vr))[:, None] * 2.0 ** -25 if t == "f16" else 0.0
    u = U[t]
    far = np.transpose(u + 3 * top + 2 * (nk + 32) * E, (0, 2, 1, 3))
    _close(_np(out), out64, far * weight + low + u * np.abs(out64) + TINY[t], "out")
    _close(lse.cpu().double().numpy(), lse64, top[..., 0] + (nk + 32) * E + 4 * E * np.abs(np.nan_to_num(lse64, neginf=0.0)), "lse")

    # the backward's inputs are what the forward kept
    O, L = _np(out), lse.cpu().double().numpy()
    grads, bufs = {}, {}
    for name, x in (("dq", q), ("dk", k), ("dv", v)):
        grads[name], bufs[name] = _place(torch.full_like(x, 5.0), odd, heads_first) if name in want else (None, None)
    gr = B.attention_grads_struct(a, dv_, **grads)
    nb = B.attention_bwd_workspace_bytes(a, gr)
    ws, whole = _ws(nb)
    B.attention_bwd(a, gr, ws)
    torch.cuda.synchronize()
    _guarded(whole, nb)
    dq64, dk64, dv64, dS = A.attention_grads(Q, K, V, scale, seen, O, L, D)
    off = (d + 20) * E * (np.einsum("bihd,bjhd->bhij", np.abs(D), np.abs(vr)) + np.einsum("bihd,bihd->bhi", np.abs(D), np.abs(O))[..., None])
    ds_off = (u + 2 * r + 8 * E) * np.abs(dS) + P * (off + 4 * E)
    long = lambda n: (n + 32) * E
    small = 2.0 ** -34 if t == "f16" else 0.0
    tol = {"dq": scale * np.einsum("bhij,bjhd->bihd", ds_off + long(nk) * np.abs(dS) + small * np.abs(dS).max(axis=3, initial=0.0, keepdims=True), np.abs(kr))}
    by_key = lambda w, x: np.einsum("bhij,bihd->bjhd", w, x).reshape(b, nk, kv, g, d).sum(3)
    tol["dk"] = scale * by_key(ds_off + long(nq * g) * np.abs(dS) + small * np.abs(dS).max(axis=2, initial=0.0, keepdims=True), np.abs(Q))
    tol["dv"] = by_key((u + 2 * r + long(nq * g)) * P + (2.0 ** -38 if t == "f16" else 0.0), np.abs(D))
    for name, w in (("dq", dq64), ("dk", dk64), ("dv", dv64)):
        if name in want:
            _close(_np(grads[name]), w, tol[name] + u * np.abs(w) + TINY[t], name)
            if name != "dq":
                assert (_np(grads[name])[~seen] == 0).all(), name
    assert _untouched(out, ob) and all(_untouched(grads[n], bufs[n]) for n in want)


def _case(b, nq, nk, h, kv, d, t, seed=0, **how):
    say(f"[gpu] attention {b} x {nq} x {nk}, heads {h}/{kv} of {d}, {t} {sorted(x for x in how if how[x] is not None)}")
    rng = np.random.default_rng(seed + b + 3 * nq + 7 * nk + 11 * h + 13 * d)
    _run(_make(rng, (b, nq, h, d), t, 1.5), _make(rng, (b, nk, kv, d), t), _make(rng, (b, nk, kv, d), t), _make(rng, (b, nq, h, d), t, 1e-2), t, **how)


SIZES = [(1, 1, 1, 1, 1, 1), (1, 1, 70, 2, 1, 8), (2, 3, 65, 4, 2, 40), (1, 33, 31, 1, 1, 64), (2, 130, 200, 2, 2, 96), (1, 65, 129, 6, 2, 128),
         (3, 17, 64, 3, 1, 33), (1, 200, 1, 2, 2, 32), (1, 5, 1000, 8, 1, 80), (1, 257, 300, 1, 1, 127)]


@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("size", SIZES)
def test_attention(size, t):
    _case(*size, t)


@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("size", SIZES[2:7])
def test_attention_of_strided_tensors(size, t):
    _case(*size, t, odd=True)
    _case(*size, t, heads_first=True)
    _case(*size, t, odd=True, heads_first=True)


def _lengths(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("size,lengths", [((4, 40, 200, 2, 1, 64), (200, 0, 1, 64)), ((3, 9, 150, 4, 4, 40), (-5, 1000, 129)),
                                          ((2, 140, 333, 4, 2, 100), (65, 63)), ((2, 1, 5000, 2, 2, 32), (4999, 130)), ((2, 3, 70, 2, 1, 128), (0, 0))])
def test_attention_of_ragged_states(size, lengths, t):
    """Lengths outside 0 .. nk count as the nearer end; NaN and infinities
    behind them have no effect."""
    _case(*size, t, lengths=_lengths(lengths), poison=True)


@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("size", [(2, 40, 333, 2, 1, 64), (3, 9, 150, 4, 4, 40), (2, 140, 260, 4, 2, 128), (2, 2, 3000, 2, 2, 32)])
@pytest.mark.parametrize("kind", ["some", "runs", "one", "none in a row"])
def test_attention_of_masked_states(size, kind, t):
    b, _, nk = size[:3]
    rng = np.random.default_rng(5)
    mask = rng.random((b, nk)) < 0.7
    if kind == "runs":                                     # whole tiles of either kind
        mask = np.repeat(rng.random((b, nk // 70 + 1)) < 0.5, 70, axis=1)[:, :nk]
    if kind == "one":
        mask[:] = False
        mask[np.arange(b), rng.integers(0, nk, b)] = True
    if kind == "none in a row":
        mask[-1] = False
    wide = torch.from_numpy(np.where(np.pad(mask, ((0, 0), (0, 9)), constant_values=True), 255, 0).astype(np.uint8)).cuda()
    _case(*size, t, mask=wide[:, :nk], poison=True)
    _case(*size, t, mask=torch.from_numpy(mask).cuda(), lengths=_lengths([nk - 60 * i for i in range(b)]), poison=True, odd=True)


@pytest.mark.parametrize("want", [("dq",), ("dk",), ("dv",), ("dk", "dv")])
def test_attention_gradients_one_by_one(want):
    _case(2, 70, 130, 4, 2, 64, "bf16", want=want)
    _case(1, 3, 2500, 4, 2, 40, "f32", want=want)


@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
def test_attention_of_far_scores(t):
    """Scores of hundreds, rising and falling along the states, so that the
    running maximum moves late and early; a scale of its own."""
    rng = np.random.default_rng(3)
    b, nq, nk, h, d = 1, 70, 400, 2, 32
    q, k = rng.standard_normal((b, nq, h, d)), rng.standard_normal((b, nk, h, d)) * 0.2
    q[..., 0], k[..., 0] = 6.0, np.linspace(-30, 30, nk)[:, None]
    q[:, ::2, :, 0] = -6.0
    up = lambda x: torch.from_numpy(x).to(T[t]).cuda()
    _run(up(q), up(k), _make(rng, (b, nk, h, d), t), _make(rng, (b, nq, h, d), t, 1e-2), t, scale=0.7)


@pytest.mark.parametrize("size", [1e-6, 1.0, 300.0])
def test_attention_fp16_gradients_of_any_size(size):
    """dS in fp16 keeps its bits whatever the size of dout, and where columns
    meet much larger values late."""
    rng = np.random.default_rng(4)
    b, nq, nk, h, d = 1, 150, 500, 2, 64
    up = np.exp2(np.linspace(-12, 0, nq))[:, None, None] * (size / 2)
    q, k, v = (_make(rng, (b, n, h, d), "f16") for n in (nq, nk, nk))
    dout = torch.from_numpy(rng.standard_normal((b, nq, h, d)) * up).half().cuda()
    _run(q, k, v, dout, "f16")


def test_attention_of_nothing():
    e = lambda *s: torch.full(s, 7.0, dtype=torch.bfloat16, device="cuda")
    # no queries: zeros for keys and values
    q, k, v, out, dk, dv = e(2, 0, 4, 32), e(2, 9, 2, 32), e(2, 9, 2, 32), e(2, 0, 4, 32), e(2, 9, 2, 32), e(2, 9, 2, 32)
    lse = torch.empty(2, 4, 0, device="cuda")
    a = B.attention_struct(q, k, v, out, lse=lse)
    B.attention_fwd(a)
    g = B.attention_grads_struct(a, e(2, 0, 4, 32), dk=dk, dv=dv)
    B.attention_bwd(a, g, torch.empty(max(16, B.attention_bwd_workspace_bytes(a, g)), dtype=torch.uint8, device="cuda"))
    assert (dk == 0).all() and (dv == 0).all()
    # no states: zeros, and lse of nothing
    q, out, dq, none = e(2, 9, 4, 32), e(2, 9, 4, 32), e(2, 9, 4, 32), e(2, 0, 2, 32)
    lse = torch.empty(2, 4, 9, device="cuda")
    a = B.attention_struct(q, none, none, out, lse=lse)
    B.attention_fwd(a)
    g = B.attention_grads_struct(a, q, dq=dq, dk=none, dv=none)
    B.attention_bwd(a, g, torch.empty(max(16, B.attention_bwd_workspace_bytes(a, g)), dtype=torch.uint8, device="cuda"))
    assert (out == 0).all() and (dq == 0).all() and (lse == -float("inf")).all()
    # no batch
    a = B.attention_struct(e(0, 9, 4, 32), none[:0], none[:0], e(0, 9, 4, 32))
    B.attention_fwd(a)


@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
def test_attention_keeps_nans_and_infinities_in_their_rows(t):
    rng = np.random.default_rng(6)
    q, k, v = _make(rng, (1, 40, 1, 32), t), _make(rng, (1, 90, 1, 32), t), _make(rng, (1, 90, 1, 32), t)
    q[0, 3, 0, 5] = float("nan")
    v[0, 8, 0, 7] = float("inf")
    out, lse = torch.empty_like(q), torch.empty(1, 1, 40, device="cuda")
    a = B.attention_struct(q, k, v, out, lse=lse)
    ws, _ = _ws(B.attention_fwd_workspace_bytes(a))
    B.attention_fwd(a, ws)
    bad = ~torch.isfinite(out[0, :, 0])
    assert bad[3].all() and bad[:, 7].all() and int(bad.sum()) == 40 + 32 - 1
    assert torch.isnan(lse[0, 0, 3]) and int(torch.isfinite(lse).sum()) == 39


def test_broadcast_inputs():
    """One set of queries, or of states, for a whole batch and for all heads."""
    rng = np.random.default_rng(8)
    q, k, v = _make(rng, (1, 50, 1, 64), "bf16"), _make(rng, (1, 80, 1, 64), "bf16"), _make(rng, (1, 80, 1, 64), "bf16")
    wide = [x.expand(3, -1, 4, -1) for x in (q, k, v)]
    res = []
    for qi, ki, vi in (wide, [x.contiguous() for x in wide]):
        o, lse = torch.empty(3, 50, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(3, 4, 50, device="cuda")
        a = B.attention_struct(qi, ki, vi, o, lse=lse)
        B.attention_fwd(a, _ws(B.attention_fwd_workspace_bytes(a))[0])
        g = [torch.empty_like(o), torch.empty(3, 80, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(3, 80, 4, 64, dtype=torch.bfloat16, device="cuda")]
        gr = B.attention_grads_struct(a, q.expand(3, -1, 4, -1), dq=g[0], dk=g[1], dv=g[2])
        B.attention_bwd(a, gr, _ws(B.attention_bwd_workspace_bytes(a, gr))[0])
        res.append([o, lse] + g)
    for x, y in zip(*res):
        assert torch.equal(x, y)


def test_fp16_many_states_of_little_weight():
    """4095 states 2^-20.5 of the first one's weight make up all of out: as fp16
    times 1 they would lose 3 % (11.4 steps of 2^-24); times 2^6 half a step
    is 2^-10.5 of them.  To that come out's rounding, 2^-11, and 2^-12 for 4096
    additions in fp32.  1024 workgroups, which leave the states in one piece."""
    nq, h, nk, d, s = 8192, 16, 4096, 8, 14.203125
    k, v = torch.zeros(1, nk, 1, d), torch.ones(1, nk, 1, d)
    k[0, 1:, 0, 0], v[0, 0] = -s, 0.0
    k, v = k.half().cuda(), v.half().cuda()
    q = torch.ones(1, nq, 1, d, dtype=torch.float16, device="cuda").expand(1, nq, h, d)
    out = torch.empty(1, nq, h, d, dtype=torch.float16, device="cuda")
    a = B.attention_struct(q, k, v, out, scale=1.0)
    B.attention_fwd(a, torch.empty(max(16, B.attention_fwd_workspace_bytes(a)), dtype=torch.uint8, device="cuda"))
    mass = (nk - 1) * np.exp(-s)
    want = mass / (1 + mass)
    assert float((out.double() - want).abs().max()) <= want * (2.0 ** -10.5 + 2.0 ** -11 + 2.0 ** -12)
