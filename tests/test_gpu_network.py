"""GPU parity of the network-head operators (gs_rms_norm_*, gs_mxfp8_quantize,
gs_linear_*, gs_orthogonalize, gs_muon_step) against the fp64 oracle.

Tolerances.  u is the unit roundoff of the result's type (2^-24 fp32, 2^-11
fp16, 2^-8 bf16) and e = 2^-24.
* norm: a sum of n squares in lane chains and a tree is off by at most
  (n / 64 + 16) e, and the result by as much again for the products around it;
  plus u per element.  A gradient's row dot product by (n / 64 + 16) e of the sum
  of its terms' magnitudes.
* linear: a sum of k products is off by at most (k + 16) e of the sum of their
  magnitudes S (fp32's three limbs drop less than 2 e of S more); 8-bit
  products with a 16-bit result by 2^-12 S (the 8-bit matrix instruction
  aligns its products to the largest before adding).  Activations have slopes
  of at most 1.13, the 16-bit ones an absolute error of 2e-7 (1 + |z|).  Plus
  u |y|.  Gradients add u_dtype of the terms' magnitudes: dz is rounded once.
* orthogonalised update: a rounding in iteration i grows at most 3.4445-fold in
  each later one, 198-fold in all five; with about 8 roundings of relative size
  2^-24 (three limbs) or 2^-16 (two) per iteration the result is within 1e-4
  or 2.5e-2 of |O| (Frobenius), plus u.
"""

import numpy as np
import pytest
import torch

from gaussian_splatting_tile_amd import binding as B
from oracle import network as N
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

T = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 1e-37, "f16": 2.0 ** -24, "bf16": 1e-37}        # half the smallest subnormal and more
E = 2.0 ** -24


def _np(t):
    return None if t is None else t.detach().float().cpu().double().numpy()


def _make(rng, shape, t, scale=1.0):
    return torch.from_numpy(rng.standard_normal(shape) * scale).to(T[t]).cuda()


def _strided(t, extra, shift):
    """t's values as a view with `extra` elements between its rows and `shift`
    in front, and what lies around it."""
    r, c = t.shape
    buf = torch.full((r * (c + extra) + shift + 8,), 77.0, device=t.device).to(t.dtype)
    v = buf[shift:shift + r * (c + extra)].view(r, c + extra)[:, :c]
    v.copy_(t)
    return v, buf


def _untouched(v, buf):
    """Nothing outside the view v of buf was written."""
    mask = torch.ones(buf.numel(), dtype=torch.bool, device=buf.device)
    o = (v.data_ptr() - buf.data_ptr()) // buf.element_size()
    idx = o + torch.arange(v.shape[0], device=buf.device)[:, None] * v.stride(0) + torch.arange(v.shape[1], device=buf.device)
    mask[idx.reshape(-1)] = False
    return bool((buf[mask].float() == 77.0).all())


def _ws(n):
    return torch.empty(max(int(n), 16), dtype=torch.uint8, device="cuda")


def _close(got, want, tol, what):
    got, want, tol = np.asarray(got), np.asarray(want), np.broadcast_to(tol, np.shape(want))
    assert got.shape == want.shape, what
    d = np.abs(got - want)
    bad = ~(d <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(d / np.maximum(tol, 1e-300)):.3g} x tolerance " \
                          f"at {np.unravel_index(np.nanargmax(np.where(bad, d, -1)), d.shape)}"


# ---- norm -------------------------------------------------------------------
NORM = [(1, 1), (3, 8), (5, 37), (4, 512), (7, 513), (130, 1024), (2, 2048), (3, 2056), (9, 4099), (2, 8192), (3, 8200), (2, 20011)]


@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("m,n", NORM)
def test_norm_forward_and_backward(m, n, t):
    say(f"[gpu] norm {m}x{n} {t}")
    rng = np.random.default_rng(m * 100003 + n)
    odd = (m + n) % 2                                      # half of the shapes strided and misaligned
    size = np.exp(rng.standard_normal((m, 1)))
    x, r = (torch.from_numpy(rng.standard_normal((m, n)) * size).to(T[t]).cuda() for _ in range(2))
    g = torch.from_numpy(1 + 0.2 * rng.standard_normal(n)).float().cuda()
    views = [_strided(v, 3 * odd, odd) for v in (x, r, torch.zeros_like(x), torch.zeros_like(x))]
    (xv, _), (rv, _), (yv, yb), (sv, sb) = views
    rstd = torch.empty(m, device="cuda")
    B.rms_norm_fwd(xv, yv, gamma=g, residual=rv, sum_out=sv, rstd=rstd, eps=1e-5)
    torch.cuda.synchronize()
    s64, r64, y64 = N.rms_norm(_np(x), _np(r), _np(g), 1e-5)
    k = (n / 64 + 16) * E
    _close(_np(sv), s64, U[t] * np.abs(s64) + TINY[t], "sum")
    _close(_np(rstd), r64, 2 * k * r64, "rstd")
    _close(_np(yv), y64, (U[t] + 2 * k) * np.abs(y64) + TINY[t], "y")
    assert _untouched(yv, yb) and _untouched(sv, sb)
    # no residual, no gamma, nothing kept
    B.rms_norm_fwd(xv, yv, eps=1e-5)
    _close(_np(yv), N.rms_norm(_np(x), None, None, 1e-5)[2], (U[t] + 2 * k) * np.abs(N.rms_norm(_np(x), None, None, 1e-5)[2]) + TINY[t], "y plain")

    dy, ds = _make(rng, (m, n), t, 0.1), _make(rng, (m, n), t, 0.1)
    (dyv, _), (dsv, _), (dxv, dxb) = (_strided(v, 3 * odd, odd) for v in (dy, ds, torch.zeros_like(x)))
    dg = torch.full((n,), 2.0, device="cuda")
    ws = _ws(B.rms_norm_bwd_workspace_bytes(m, n))
    for acc in (False, True):
        B.rms_norm_bwd(sv, rstd, dyv, dxv, gamma=g, dsum=dsv, dgamma=dg, workspace=ws, accumulate=acc)
    torch.cuda.synchronize()
    S, R, DY, G = _np(sv), _np(rstd), _np(dy), _np(g)
    dx64, dg64 = N.rms_norm_grads(S, R, DY, G, _np(ds))
    h = S * R[:, None]
    terms = np.abs(R[:, None] * DY * G) + np.abs(R[:, None] * h) * np.abs(DY * G * h).mean(1, keepdims=True) + np.abs(_np(ds))
    _close(_np(dxv), dx64, U[t] * np.abs(dx64) + 2 * k * terms + TINY[t], "dx")
    _close(_np(dg), 2 * dg64, 2 * (m + 16) * E * np.abs(DY * h).sum(0) + E, "dgamma, added twice")
    assert _untouched(dxv, dxb)


# the widths of every group of lanes, rows that make the backward's workgroups go round, and one workgroup alone
@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("m,n", [(16, 120), (40, 129), (9000, 7), (4100, 65), (2500, 256), (1500, 600), (700, 1300), (1030, 2047), (300, 3001), (280, 5003)])
def test_norm_of_every_width(m, n, t):
    test_norm_forward_and_backward(m, n, t)


def test_norm_of_awkward_rows():
    x = torch.zeros(6, 64, device="cuda")
    x[1] = 1e-30
    x[2, 3] = float("inf")
    x[3, 3] = float("nan")
    x[4] = 1e15
    x[5, 0] = -5.0
    y, rstd = torch.empty_like(x), torch.empty(6, device="cuda")
    B.rms_norm_fwd(x, y, rstd=rstd, eps=0.0)
    got = y.cpu()
    B.rms_norm_fwd(x, y, rstd=rstd, eps=1e-6)
    z = y.cpu()
    assert (z[0] == 0).all() and (z[1].abs() < 1e-20).all()
    assert torch.isnan(z[2, 3]) and (z[2, :3] == 0).all() and torch.isnan(z[3]).all()
    assert torch.allclose(z[4], torch.ones(64)) and (z[5, 1:] == 0).all()
    want = -5.0 / np.sqrt(25.0 / 64.0 + 1e-6)
    assert abs(float(z[5, 0]) - want) <= (1 + 2 * 17) * E * abs(want)
    assert torch.isnan(got[0]).all()                # 0 / 0 without eps, as the formula has it


@pytest.mark.parametrize("m,n", [(1, 32), (5, 64), (3, 2048), (2, 2080), (2, 9600)])
@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_norm_to_8_bits_equals_norm_then_quantise(m, n, t):
    """Codes and scales against the oracle's quantisation of the fp32 norm: a
    code may differ only where its position is within the norm's error of a
    rounding boundary."""
    rng = np.random.default_rng(n)
    x, r = _make(rng, (m, n), t), _make(rng, (m, n), t)
    g = torch.from_numpy(np.exp(rng.standard_normal(n))).float().cuda()
    y, s = torch.empty(m, n, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(m, n // 32, dtype=torch.uint8, device="cuda")
    B.rms_norm_fwd(x, y, gamma=g, residual=r, y_scales=s)
    y64 = N.rms_norm(_np(x), _np(r), _np(g))[2]
    q64, s64 = N.mxfp8_quantize(y64)
    np.testing.assert_array_equal(s.cpu().numpy(), s64)
    v = N.mxfp8_value(y.view(torch.uint8).cpu().numpy(), s64)
    scale = np.repeat(2.0 ** (s64.astype(np.float64) - 127), 32, axis=1)
    step = np.maximum(2.0 ** np.floor(np.log2(np.maximum(np.abs(y64 / scale), 2.0 ** -6))), 2.0 ** -6) / 8 * scale
    _close(v, y64, 0.5 * step + 2 * (n / 64 + 16) * E * np.abs(y64), "8-bit y")
    assert (y.view(torch.uint8).cpu().numpy() != q64).mean() < 1e-3


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_quantise_is_exact(t):
    rng = np.random.default_rng(8)
    x = rng.standard_normal((67, 160)) * np.exp2(rng.integers(-12, 12, (67, 160)))
    x[0, :32] = 0.0
    x[1, 5], x[2, 40], x[3, 70] = np.inf, np.nan, -np.inf
    x[4, 0:32] = np.linspace(-448, 448, 32)
    if t == "f32":
        x[5, :32], x[6, :32] = 1e-42, 3e38
    xd = torch.from_numpy(x).to(T[t]).cuda()
    for extra, shift in ((0, 0), (5, 3)):
        xv, _ = _strided(xd, extra, shift)
        code_buf = torch.full((67, 160 + extra), 0x11, dtype=torch.uint8, device="cuda")
        s = torch.empty(67, 5, dtype=torch.uint8, device="cuda")
        B.mxfp8_quantize(xv, code_buf[:, :160].view(torch.float8_e4m3fn), s)
        q64, s64 = N.mxfp8_quantize(_np(xd))
        np.testing.assert_array_equal(s.cpu().numpy(), s64)
        ok = np.repeat(s64 != 255, 32, axis=1)
        got = code_buf[:, :160].cpu().numpy()
        z = q64 & 127 == 0
        assert ((got == q64) | (z & (got & 127 == 0)))[ok].all()
        assert (code_buf[:, 160:] == 0x11).all()


# ---- linear -----------------------------------------------------------------
def _linear_case(m, n, k, t, ty, act, planes, residual, keep, odd, seed=0):
    rng = np.random.default_rng(seed + m * 7 + n * 11 + k * 13)
    x, w = _make(rng, (m, k), t), _make(rng, (n, k), t, k ** -0.5)
    b = torch.from_numpy(rng.standard_normal(n)).float().cuda()
    shape = (n, m) if planes else (m, n)
    r = _make(rng, shape, ty) if residual else None
    xv, wv = _strided(x, 3 * odd, odd)[0], _strided(w, 5 * odd, odd)[0]
    yv, yb = _strided(torch.zeros(shape, dtype=T[ty], device="cuda"), 1 * odd, odd)
    zv, zb = _strided(torch.zeros((m, n), dtype=T[t], device="cuda"), 7 * odd, odd) if keep else (None, None)
    lin = B.linear_struct(xv, wv, yv, bias=b, residual=r, z=zv, act=act, planes=planes)
    nb = B.linear_fwd_workspace_bytes(lin)
    ws = torch.full((nb + 64,), 0x5A, dtype=torch.uint8, device="cuda")
    B.linear_fwd(lin, ws[:nb] if nb else None)
    torch.cuda.synchronize()
    assert (ws[nb:] == 0x5A).all(), "write past the workspace"
    X, W = _np(x), _np(w)
    z64, y64 = N.linear(X, W, _np(b), act, None if r is None else (_np(r).T if planes else _np(r)))
    S = np.abs(X) @ np.abs(W).T + np.abs(_np(b))
    tol = (k + 20) * E * S
    if keep:
        _close(_np(zv), z64, U[t] * np.abs(z64) + tol + TINY[t], "z")
        assert _untouched(zv, zb)
    got = _np(yv).T if planes else _np(yv)
    _close(got, y64, U[ty] * np.abs(y64) + 1.13 * tol + (0 if act in ("none", "relu") else 2e-7 * (1 + np.abs(z64)))
           + 4 * E * np.abs(y64 if r is None else _np(r).T if planes else _np(r)) + TINY[ty], "y")
    assert _untouched(yv, yb)


SIZES = [(1, 1, 1), (1, 64, 64), (3, 17, 31), (17, 8, 8), (64, 64, 32), (65, 59, 72), (100, 136, 333), (129, 200, 1000), (16, 300, 1024), (5, 4096, 136)]


@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_linear_forward(m, n, k, t):
    i = m + n + k
    say(f"[gpu] linear {m} {n} {k} {t}")
    acts = ["none", "relu", "silu", "gelu"]
    _linear_case(m, n, k, t, t, acts[i % 4], False, bool(i & 1), True, 0)
    _linear_case(m, n, k, t, "f32", acts[(i + 1) % 4], True, True, bool(i & 2), 0)
    _linear_case(m, n, k, t, t, acts[(i + 2) % 4], bool(i & 1), False, False, 1)


@pytest.mark.parametrize("m,n,k", [(1024, 1032, 264), (2050, 768, 128), (8200, 512, 520), (64, 96, 8200), (2000, 2048, 64)])
@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
def test_linear_forward_large_tiles_and_splits(m, n, k, t):
    say(f"[gpu] linear {m} {n} {k} {t}")
    _linear_case(m, n, k, t, t, "gelu", False, True, True, 0)
    _linear_case(m, n, k, t, "f32", "none", True, False, False, 0)


# few rows by 4 and 16 waves and by tiles, converted while loading by 64 and 128 tiles, packed, long k in many splits
@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,k", [(1, 70, 8200), (16, 4096, 2100), (16, 4100, 515), (17, 203, 13001), (40, 33, 9000), (3000, 200, 700), (700, 1000, 301),
                                   (2300, 1030, 64)])
def test_linear_forward_by_every_way(m, n, k, t):
    test_linear_forward(m, n, k, t)


def test_linear_residual_in_place_empty_and_no_bias():
    rng = np.random.default_rng(1)
    x, w, y = _make(rng, (70, 64), "bf16"), _make(rng, (40, 64), "bf16", 0.1), _make(rng, (70, 40), "bf16")
    want = N.linear(_np(x), _np(w), None, "silu", _np(y))[1]
    B.linear_fwd(B.linear_struct(x, w, y, residual=y, act="silu"))
    _close(_np(y), want, 2.0 ** -7 * np.abs(want) + 1e-4, "in place")
    before = y.clone()
    B.linear_fwd(B.linear_struct(x[:0], w, y[:0]))
    assert torch.equal(before, y)


@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_linear_keeps_infinities_and_nans_in_their_rows(t):
    rng = np.random.default_rng(2)
    x, w = _make(rng, (70, 72), t), _make(rng, (33, 72), t)
    x[3, 5], x[9, 0], x[20, 70] = float("inf"), float("nan"), -float("inf")
    w[7, 1] = float("nan")
    y = torch.empty(70, 33, dtype=T[t], device="cuda")
    B.linear_fwd(B.linear_struct(x, w, y))
    fin = torch.isfinite(y).cpu().numpy()
    want = np.ones((70, 33), bool)
    want[[3, 9, 20]] = False
    want[:, 7] = False
    np.testing.assert_array_equal(fin, want)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_activations_in_fp32_over_their_range(act):
    """y and its slope through a product with 1: absolute errors of fp32's
    rounding of values near 1, relative ones down the tail (its exponent's
    product is off by z^2 / 2 ulps), nothing left far below."""
    from math import erfc

    z = torch.cat([torch.linspace(-14, 14, 100001), torch.tensor([0.0, 1e-30, -1e-30, 300.0, -300.0, 3e38, -3e38])]).cuda().view(-1, 1)
    w, y, dx = torch.ones(1, 1, device="cuda"), torch.empty_like(z), torch.empty_like(z)
    lin = B.linear_struct(z, w, y, act=act)
    B.linear_fwd(lin, _ws(B.linear_fwd_workspace_bytes(lin)))
    back = B.linear_struct(z, w, None, z=z, act=act)
    gr = B.linear_grads_struct(back, torch.ones_like(z), dx=dx)
    B.linear_bwd(back, gr, _ws(B.linear_bwd_workspace_bytes(back, gr)))
    v = _np(z)[:, 0]
    if act == "gelu":
        phi = np.array([0.5 * erfc(-t / 2 ** 0.5) for t in v])
        want, slope = v * phi, phi + v * np.exp(-0.5 * np.minimum(np.abs(v), 1e3) ** 2) / (2 * np.pi) ** 0.5
    else:
        s = 1 / (1 + np.exp(np.minimum(-v, 700)))
        want, slope = v * s, s * (1 + v * (1 - s))
    a = np.minimum(np.abs(v), 20.0)
    # results under 2^-125 may be 0
    _close(_np(y)[:, 0], want, (8 + a * a) * E * np.abs(want) + 1e-35, "y")
    _close(_np(dx)[:, 0], slope, (8 + a * a) * E * (1 + a) * np.maximum(np.abs(slope), np.minimum(1, 4 * np.exp(-a))) + 1e-35, "slope")


def test_linear_f32_keeps_the_largest_and_smallest_values():
    x = torch.zeros(4, 32, device="cuda")
    w = torch.zeros(16, 32, device="cuda")
    top = torch.finfo(torch.float32).max
    x[0, 0], x[1, 1], x[2, 2], x[3, 3] = top, 1 + 2.0 ** -23, 2.0 ** -100, -top
    w[:, :4] = 1.0
    y = torch.empty(4, 16, device="cuda")
    B.linear_fwd(B.linear_struct(x, w, y))
    assert (y.cpu() == torch.tensor([top, 1 + 2.0 ** -23, 2.0 ** -100, -top])[:, None]).all()


@pytest.mark.parametrize("m,n,k", [(1, 16, 32), (3, 40, 96), (130, 64, 128), (257, 72, 288), (1030, 528, 640), (16, 64, 8192), (100, 33, 160)])
@pytest.mark.parametrize("ty,planes", [("bf16", False), ("f16", False), ("f32", False), ("f32", True), ("bf16", True)])
def test_linear_8_bits(m, n, k, ty, planes):
    say(f"[gpu] linear 8 bits {m} {n} {k} {ty} planes={planes}")
    rng = np.random.default_rng(m + n + k)
    size = np.exp2(rng.integers(-6, 7, (1, k)))
    x, w = _make(rng, (m, k), "f32"), _make(rng, (n, k), "f32", k ** -0.5)
    x *= torch.from_numpy(size).float().cuda()
    w /= torch.from_numpy(size).float().cuda()
    q = []
    for v in (x, w):
        pad = 16 if (m + n) % 2 else 3                     # aligned and unaligned code rows
        codes = torch.zeros(v.shape[0], k + pad, dtype=torch.uint8, device="cuda")[:, :k].view(torch.float8_e4m3fn)
        scales = torch.full((v.shape[0], k // 32 + 1), 255, dtype=torch.uint8, device="cuda")[:, :k // 32]
        B.mxfp8_quantize(v, codes, scales)
        q += [codes, scales]
    b = torch.from_numpy(rng.standard_normal(n)).float().cuda()
    shape = (n, m) if planes else (m, n)
    r = _make(rng, shape, ty)
    y = torch.empty(shape, dtype=T[ty], device="cuda")
    lin = B.linear_struct(q[0], q[2], y, bias=b, residual=r, act="silu", planes=planes, x_scales=q[1], w_scales=q[3])
    B.linear_fwd(lin, _ws(B.linear_fwd_workspace_bytes(lin)))
    X, W = (N.mxfp8_value(c.contiguous().view(torch.uint8).cpu().numpy(), s.cpu().numpy()) for c, s in ((q[0], q[1]), (q[2], q[3])))
    R = _np(r).T if planes else _np(r)
    z64, y64 = N.linear(X, W, _np(b), "silu", R)
    S = np.abs(X) @ np.abs(W).T + np.abs(_np(b))
    tol = 1.13 * S * ((k + 20) * E if ty == "f32" else 2.0 ** -12) + 2e-7 * (1 + np.abs(z64))
    _close(_np(y).T if planes else _np(y), y64, U[ty] * np.abs(y64) + tol + 4 * E * np.abs(R) + TINY[ty], "y")


@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (7, 8, 16), (65, 59, 40), (130, 136, 333), (300, 17, 72), (1000, 264, 520), (5000, 96, 136), (1, 512, 256)])
def test_linear_backward(m, n, k, t):
    acts = ["none", "relu", "silu", "gelu"]
    for planes, ty, act, odd in ((False, t, acts[(m + n) % 4], 0), (True, "f32", acts[(m + k) % 4], 0), (False, t, "none", 0),
                                 (bool(m & 1), t, acts[(n + k) % 4], 1)):
        say(f"[gpu] linear backward {m} {n} {k} {t} {act} planes={planes} odd={odd}")
        rng = np.random.default_rng(m + 3 * n + 5 * k)
        x, w = _strided(_make(rng, (m, k), t), 3 * odd, odd)[0], _strided(_make(rng, (n, k), t, k ** -0.5), 5 * odd, odd)[0]
        z = _strided(_make(rng, (m, n), t), 7 * odd, odd)[0] if act != "none" else None
        dy = _strided(_make(rng, (n, m) if planes else (m, n), ty, 0.1), odd, odd)[0]
        dx, dxb = _strided(torch.zeros((m, k), dtype=T[t], device="cuda"), odd, odd)
        tw = "f32" if (m + k) % 2 else t
        dw, dwb = _strided(torch.zeros((n, k), dtype=T[tw], device="cuda"), odd, odd)
        db = torch.zeros(n, device="cuda")
        lin = B.linear_struct(x, w, None, z=z, act=act, planes=planes)
        gr = B.linear_grads_struct(lin, dy, dx=dx, dw=dw, db=db)
        nb = B.linear_bwd_workspace_bytes(lin, gr)
        ws = torch.full((nb + 64,), 0xFF, dtype=torch.uint8, device="cuda")          # NaNs in any type
        B.linear_bwd(lin, gr, ws[:nb] if nb else None)
        torch.cuda.synchronize()
        assert (ws[nb:] == 0xFF).all(), "write past the workspace"
        DY = _np(dy).T if planes else _np(dy)
        dx64, dw64, db64, dz64 = N.linear_grads(_np(x), _np(w), None if z is None else _np(z), DY, act)
        a = np.abs(dz64) + (0 if act in ("none", "relu") else 2e-6 * np.abs(DY))
        uz = 0.0 if t == "f32" else U[t] + TINY[t]
        sx, sw = a @ np.abs(_np(w)), a.T @ np.abs(_np(x))
        slack = 0 if act in ("none", "relu") else 2e-6
        _close(_np(dx), dx64, U[t] * np.abs(dx64) + (uz + (n + 20) * E + slack) * sx + TINY[t] * (1 + n), "dx")
        _close(_np(dw), dw64, U[tw] * np.abs(dw64) + (uz + (m + 20) * E + slack) * sw + TINY[tw] * (1 + m), "dw")
        _close(_np(db), db64, ((m + 20) * E + slack) * a.sum(0) + 1e-30, "db")
        assert _untouched(dx, dxb) and _untouched(dw, dwb)
        # each alone, and added to what is there
        first = dw.float().clone()
        for kw in (dict(dx=dx), dict(dw=dw), dict(db=db)):
            gr = B.linear_grads_struct(lin, dy, accumulate=True, **kw)
            B.linear_bwd(lin, gr, _ws(B.linear_bwd_workspace_bytes(lin, gr)))
        _close(_np(dw), 2 * first.cpu().double().numpy(), 2 * U[tw] * np.abs(2 * _np(first)) + TINY[tw], "dw added to itself")
        _close(_np(db), 2 * db64, ((2 * m + 40) * E + 2 * slack) * a.sum(0) + 1e-30, "db added to itself")


# one row block and several, products converted while loading and packed, long sums over rows
@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,k", [(64, 300, 500), (65, 2048, 40), (9000, 47, 198), (900, 600, 58), (700, 640, 700), (3, 4099, 33)])
def test_linear_backward_by_every_way(m, n, k, t):
    test_linear_backward(m, n, k, t)


def test_linear_backward_matches_differences_of_the_forward():
    """dL/dw and dL/dx of L = sum(y dy) by central differences of the fp32
    forward: the step 2^-6 leaves a truncation error of about 1e-4 and a
    rounding error of about 1e-4 of the values of order 1."""
    rng = np.random.default_rng(4)
    x, w, dy = _make(rng, (5, 24), "f32"), _make(rng, (9, 24), "f32", 0.3), _make(rng, (5, 9), "f32")
    y, z = torch.empty(5, 9, device="cuda"), torch.empty(5, 9, device="cuda")

    def loss(x, w):
        lin = B.linear_struct(x, w, y, z=z, act="gelu")
        B.linear_fwd(lin, _ws(B.linear_fwd_workspace_bytes(lin)))
        return float((y.double() * dy.double()).sum())

    loss(x, w)
    lin = B.linear_struct(x, w, None, z=z.clone(), act="gelu")
    zk = z.clone()
    lin = B.linear_struct(x, w, None, z=zk, act="gelu")
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    gr = B.linear_grads_struct(lin, dy, dx=dx, dw=dw)
    B.linear_bwd(lin, gr, _ws(B.linear_bwd_workspace_bytes(lin, gr)))
    h = 2.0 ** -6
    for t, d, at in ((x, dx, (3, 7)), (x, dx, (0, 23)), (w, dw, (8, 0)), (w, dw, (2, 11))):
        keep = float(t[at])
        t[at] = keep + h
        up = loss(x, w)
        t[at] = keep - h
        down = loss(x, w)
        t[at] = keep
        assert abs((up - down) / (2 * h) - float(d[at])) < 2e-3


def test_linear_backward_of_no_rows():
    w = torch.zeros(8, 16, device="cuda")
    x, dy = torch.zeros(0, 16, device="cuda"), torch.zeros(0, 8, device="cuda")
    dw, db = torch.full((8, 16), 3.0, device="cuda"), torch.full((8,), 3.0, device="cuda")
    lin = B.linear_struct(x, w, None)
    B.linear_bwd(lin, B.linear_grads_struct(lin, dy, dw=dw, db=db, accumulate=True))
    assert (dw == 3).all() and (db == 3).all()
    B.linear_bwd(lin, B.linear_grads_struct(lin, dy, dw=dw, db=db))
    assert (dw == 0).all() and (db == 0).all()
    g = torch.full((16,), 3.0, device="cuda")
    B.rms_norm_bwd(x, torch.zeros(0, device="cuda"), x, x, dgamma=g)
    assert (g == 0).all()


def test_offsets_past_32_bits():
    """Rows more than 2^31 elements into x, z and y."""
    stride, m, n, k = 60000, 40000, 64, 72
    buf = torch.empty(m * stride, dtype=torch.bfloat16, device="cuda")
    view = lambda at, cols: buf.view(m, stride)[:, at:at + cols]
    x, y, z, dx = view(0, k), view(128, n), view(256, n), view(512, k)
    w = _make(np.random.default_rng(6), (n, k), "bf16", 0.1)
    x.normal_()
    B.linear_fwd(B.linear_struct(x, w, y, z=z, act="relu"))
    tail = slice(m - 70, m)
    z64, y64 = N.linear(_np(x[tail]), _np(w), None, "relu")
    _close(_np(y[tail]), y64, 2.0 ** -8 * np.abs(y64) + 1e-4, "y")
    dy = y
    db, dw = torch.empty(n, device="cuda"), torch.empty(n, k, device="cuda")
    lin = B.linear_struct(x, w, None, z=z, act="relu")
    gr = B.linear_grads_struct(lin, dy, dx=dx, dw=dw, db=db)
    B.linear_bwd(lin, gr, _ws(B.linear_bwd_workspace_bytes(lin, gr)))
    dx64 = N.linear_grads(_np(x[tail]), _np(w), _np(z[tail]), _np(dy[tail]), "relu")[0]
    _close(_np(dx[tail]), dx64, 2.0 ** -6 * (np.abs(_np(dy[tail])) @ np.abs(_np(w))), "dx")
    dz = dy.float() * (z > 0)
    want = dz.t().contiguous() @ x.float()
    assert torch.allclose(dw, want, rtol=0, atol=float(3e-3 * (dz.abs().t().contiguous() @ x.float().abs()).max()))
    B.rms_norm_fwd(x, dx, residual=None)
    _close(_np(dx[tail]), N.rms_norm(_np(x[tail]))[2], 2.0 ** -7 * np.abs(N.rms_norm(_np(x[tail]))[2]) + 1e-6, "norm")


# ---- orthogonalised update --------------------------------------------------
@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("e,r,f", [(1, 1, 1), (2, 1, 40), (1, 33, 5), (3, 32, 64), (2, 100, 70), (1, 300, 130), (2, 129, 520), (1, 640, 512)])
def test_orthogonalize(e, r, f, t):
    say(f"[gpu] orthogonalize {e}x{r}x{f} {t}")
    rng = np.random.default_rng(r + f)
    g = _make(rng, (e, r, f), t, 1e-3) + _make(rng, (e, r, 1), t, 1e-2) * _make(rng, (e, 1, f), t)
    for to in {t, "f32"}:
        out = torch.empty((e, r, f), dtype=T[to], device="cuda")
        mu = B.muon_struct(g, out=out)
        nb = B.muon_workspace_bytes(mu)
        ws = torch.full((nb + 64,), 0xFF, dtype=torch.uint8, device="cuda")
        B.orthogonalize(mu, ws[:nb])
        torch.cuda.synchronize()
        assert (ws[nb:] == 0xFF).all(), "write past the workspace"
        for i in range(e):
            want = N.orthogonalize(_np(g[i]))
            err = np.linalg.norm(_np(out[i]) - want) / np.linalg.norm(want)
            assert err <= (1e-4 if to == "f32" else 2.5e-2 + U[to]), (i, err)


# one workgroup a matrix or products by 128, 64 and 32 tiles, with and without splits of a long side
@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("e,r,f", [(1, 58, 700), (2, 64, 1500), (1, 32, 1000), (1, 704, 64), (300, 17, 33), (260, 64, 40), (3, 96, 96), (1, 128, 128),
                                   (2, 64, 384), (1, 260, 900), (5, 190, 30), (1, 20, 3000), (1, 1000, 1030)])
def test_orthogonalize_by_every_way(e, r, f, t):
    test_orthogonalize(e, r, f, t)


def test_orthogonalize_of_zeros_ranks_and_scales():
    rng = np.random.default_rng(9)
    g = torch.zeros(4, 40, 24, device="cuda")
    g[1] = _make(rng, (40, 1), "f32") * _make(rng, (1, 24), "f32")           # rank 1
    g[2] = g[1] * 1e12
    g[3] = g[1] * 1e-6
    out = torch.empty_like(g)
    mu = B.muon_struct(g, out=out)
    B.orthogonalize(mu, _ws(B.muon_workspace_bytes(mu)))
    o = _np(out)
    assert (o[0] == 0).all()
    want = N.orthogonalize(_np(g[1]))
    for i, eps in ((1, 1e-4), (2, 1e-4), (3, 1e-2)):                          # eps is no longer small beside 1e-6
        w = N.orthogonalize(_np(g[i]))
        assert np.linalg.norm(o[i] - w) <= eps * np.linalg.norm(want)
    g[0, 3, 4] = float("nan")
    B.orthogonalize(mu, _ws(B.muon_workspace_bytes(mu)))
    assert torch.isnan(out[0]).all() and torch.isfinite(out[1:]).all()


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("e,r,f", [(1, 96, 33), (3, 64, 128), (2, 200, 100)])
def test_muon_step(e, r, f, t, nesterov):
    rng = np.random.default_rng(r)
    g, w, mom = _make(rng, (e, r, f), t, 1e-2), _make(rng, (e, r, f), t, 0.1), _make(rng, (e, r, f), "f32", 1e-2)
    h = dict(lr=0.03, beta=0.9, weight_decay=0.1, scale=1.5)
    mo, wo = torch.empty_like(mom), torch.empty_like(w)
    mu = B.muon_struct(g, momentum=mom, weight=w, momentum_out=mo, weight_out=wo, nesterov=nesterov, **h)
    B.muon_step(mu, _ws(B.muon_workspace_bytes(mu)))
    for i in range(e):
        m64, w64 = N.muon_step(_np(g[i]), _np(mom[i]), _np(w[i]), nesterov=nesterov, **h)
        _close(_np(mo[i]), m64, 3 * E * np.abs(m64) + E * np.abs(_np(mom[i])) + 1e-12, "momentum")
        o = np.abs(w64 - _np(w[i]) * (1 - h["lr"] * h["weight_decay"])).max()
        _close(_np(wo[i]), w64, U[t] * np.abs(w64) + 4 * E * np.abs(_np(w[i])) + (1e-4 if t == "f32" else 2.5e-2) * o * np.sqrt(min(r, f)), "weight")
    # in place gives the same bits
    mu = B.muon_struct(g, momentum=mom, weight=w, nesterov=nesterov, **h)
    B.muon_step(mu, _ws(B.muon_workspace_bytes(mu)))
    assert torch.equal(mom, mo) and torch.equal(w, wo)


# ---- streams, graphs, reproducibility ----------------------------------------
def test_streams_graph_replays_and_reproducibility():
    """The calls run on the stream they are given, in a captured graph, and give
    the same bits every time."""
    rng = np.random.default_rng(12)
    m, n, k = 500, 264, 128
    x, w, w2 = _make(rng, (m, k), "bf16"), _make(rng, (n, k), "bf16", 0.1), _make(rng, (k, n), "bf16", 0.1)
    gamma = torch.ones(k, device="cuda")
    E_ = lambda *s, t=torch.bfloat16: torch.empty(s, dtype=t, device="cuda")
    s, y, rstd, z, hid, out = E_(m, k), E_(m, k), E_(m, t=torch.float32), E_(m, n), E_(m, n), E_(m, k)
    dh, dw2, db2, dw, db, dy, dx, dg = E_(m, n), E_(k, n), E_(k, t=torch.float32), E_(n, k), E_(n, t=torch.float32), E_(m, k), E_(m, k), E_(k, t=torch.float32)
    mom, mom_out, wout = torch.zeros(n, k, device="cuda"), E_(n, k, t=torch.float32), E_(n, k)
    l1 = B.linear_struct(y, w, hid, z=z, act="gelu")
    l2 = B.linear_struct(hid, w2, out, residual=s)
    g2 = B.linear_grads_struct(l2, out, dx=dh, dw=dw2, db=db2)
    g1 = B.linear_grads_struct(l1, dh, dx=dy, dw=dw, db=db)
    mu = B.muon_struct(dw, momentum=mom, weight=w, momentum_out=mom_out, weight_out=wout)
    ws = _ws(max(B.linear_fwd_workspace_bytes(l1), B.linear_fwd_workspace_bytes(l2), B.linear_bwd_workspace_bytes(l1, g1),
                 B.linear_bwd_workspace_bytes(l2, g2), B.rms_norm_bwd_workspace_bytes(m, k), B.muon_workspace_bytes(mu)))

    def step(stream=None):
        B.rms_norm_fwd(x, y, gamma=gamma, residual=x, sum_out=s, rstd=rstd, stream=stream)
        B.linear_fwd(l1, ws, stream)
        B.linear_fwd(l2, ws, stream)
        B.linear_bwd(l2, g2, ws, stream)
        B.linear_bwd(l1, g1, ws, stream)
        B.rms_norm_bwd(s, rstd, dy, dx, gamma=gamma, dsum=out, dgamma=dg, workspace=ws, stream=stream)
        B.muon_step(mu, ws, stream)

    outs = (out, dh, dw2, db2, dw, db, dy, dx, dg, mom_out, wout)
    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    assert all(torch.isfinite(t.float()).all() for t in want)
    side = torch.cuda.Stream()
    for t in outs:
        t.zero_()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(torch.cuda.current_stream())
    for _ in range(3):
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
