"""GPU parity of group norm with an activation (gs_group_norm_fwd,
gs_group_norm_bwd) and of its 8-bit checkpoint against the fp64 oracle.

Tolerances.  u is the unit roundoff of the type (2^-24 fp32, 2^-11 fp16, 2^-8
bf16), e = 2^-24 and k = (m / 64 + 64) e for sums over m values in lane chains
and trees.  With X the group's largest magnitude and sd its spread, the mean is
off by k X, every deviation from it by as much, so the variance by
2 k (1 + X / sd) of itself and rstd by as much.  An output: h off by (k + 2 e) X rstd and
that part of itself, times gamma and a slope of at most 1.13; activations by
2e-7 (1 + |z|), 16-bit or not; u for its rounding.  Gradients take mean and rstd as
they were kept: z is off by 4 e (|h gamma| + |z|) + 2 e |x rstd gamma|, the slope by that and 2e-7 (1 + |z|), or
(relu) altogether where z is within it of 0.
"""

import numpy as np
import pytest
import torch

from gaussian_splatting_tile_amd import binding as B
from oracle import attention as A
from oracle import network as N
from tests.gpu_util import say
from tests.test_gpu_attention import E, T, TINY, U, _close, _guarded, _np, _untouched, _ws

pytestmark = pytest.mark.gpu


def _map(x, odd):
    """x [n][p][c] as a view into a buffer of 77s, images and pixels apart
    (`odd`: by odd numbers from an odd address)."""
    n, p, c = x.shape
    sp = c + (5 if odd else 0)
    si = p * sp + (11 if odd else 0)
    buf = torch.full((n * si + 16,), 77.0, device="cuda").to(x.dtype)
    v = buf.as_strided((n, p, c), (si, sp, 1), 3 if odd else 8)
    v.copy_(x)
    return v, buf


def _per_group(v, groups):
    n, p, c = v.shape
    return v.reshape(n, p, groups, c // groups)


def _case(n, p, c, groups, t, act, odd=False, kept=False, offset=1.0, affine=True, params=True, eps=1e-5):
    say(f"[gpu] group norm {n} x {p} x {c} / {groups} {t} {act} odd={odd} kept={kept}")
    rng = np.random.default_rng(n + 3 * p + 7 * c + 11 * groups)
    x = offset * rng.standard_normal((1, 1, c)) + np.exp(0.5 * rng.standard_normal((n, 1, c))) * rng.standard_normal((n, p, c))
    x = torch.from_numpy(x).to(T[t]).cuda()
    gamma, beta = (torch.from_numpy(v).float().cuda() for v in (1 + 0.2 * rng.standard_normal(c), 0.3 * rng.standard_normal(c)))
    if not affine:
        gamma = beta = None
    G, H = (None, None) if not affine else (_np(gamma), _np(beta))
    (xv, _), (yv, yb) = _map(x, odd), _map(torch.full_like(x, 5.0), odd)
    mean, rstd = torch.empty(n, groups, device="cuda"), torch.empty(n, groups, device="cuda")
    codes = scales = code_buf = None
    if kept:
        code_buf = torch.full((n, p, c + 7 * odd), 0x11, dtype=torch.uint8, device="cuda")
        codes = code_buf[..., :c].view(torch.float8_e4m3fn)
        scales = torch.zeros(n, p, c // 32, dtype=torch.uint8, device="cuda")
    nb = B.group_norm_fwd_workspace_bytes(n, p, c, groups)
    ws, whole = _ws(nb)
    B.group_norm_fwd(xv, yv, groups, gamma=gamma, beta=beta, act=act, mean=mean, rstd=rstd, kept=codes, kept_scales=scales, eps=eps, workspace=ws)
    torch.cuda.synchronize()
    _guarded(whole, nb)
    X = _np(x)
    mean64, rstd64, z64, y64 = A.group_norm(X, groups, G, H, act, eps)
    k = (p * c // groups / 64 + 64) * E
    big = np.abs(_per_group(X, groups)).max(axis=(1, 3))
    near = 2 * k * (1 + big * rstd64)
    _close(_np(mean), mean64, k * big + TINY["f32"], "mean")
    _close(_np(rstd), rstd64, near * rstd64, "rstd")
    wide = lambda v: np.repeat(v, c // groups, axis=1)[:, None]
    gam, bet = (np.ones(c), np.zeros(c)) if not affine else (np.abs(G), np.abs(H))
    h64 = (X - wide(mean64)) * wide(rstd64)
    z_off = gam * ((k + 2 * E) * wide(big * rstd64) + np.abs(h64) * (wide(near) + 4 * E)) + 4 * E * (np.abs(z64) + bet)
    soft = 0.0 if act in ("none", "relu") else 2e-7 * (1 + np.abs(z64))
    _close(_np(yv), y64, 1.13 * z_off + soft + U[t] * np.abs(y64) + TINY[t], "y")
    if kept:
        q64, s64 = N.mxfp8_quantize(X.reshape(n * p, c))
        np.testing.assert_array_equal(scales.cpu().numpy().reshape(n * p, -1), s64)
        got = code_buf[..., :c].cpu().numpy().reshape(n * p, c)
        zero = q64 & 127 == 0
        assert ((got == q64) | (zero & (got & 127 == 0))).all()
        assert (code_buf[..., c:] == 0x11).all()
        X = N.mxfp8_value(got, s64).reshape(n, p, c)
    assert _untouched(yv, yb)
    # nothing kept, in place
    again = xv if not kept else x.clone()
    B.group_norm_fwd(again, again, groups, gamma=gamma, beta=beta, act=act, eps=eps, workspace=ws)
    _close(_np(again), y64, 1.13 * z_off + soft + U[t] * np.abs(y64) + TINY[t], "y in place")

    # backward, twice: the second adds to the parameters' gradients
    dy = torch.from_numpy(rng.standard_normal((n, p, c)) * 0.1).to(T[t]).cuda()
    (xv, _), (dyv, _), (dxv, dxb) = _map(x, odd), _map(dy, odd), _map(torch.full_like(x, 5.0), odd)
    dg, db = (torch.full((c,), 9.0, device="cuda") for _ in range(2)) if params else (None, None)
    nb = B.group_norm_bwd_workspace_bytes(n, p, c, groups)
    ws, whole = _ws(nb)
    for acc in (False, True):
        B.group_norm_bwd(codes if kept else xv, mean, rstd, dyv, dxv, groups, gamma=gamma, beta=beta, act=act, dgamma=dg, dbeta=db, x_scales=scales,
                         workspace=ws, accumulate=acc)
    torch.cuda.synchronize()
    _guarded(whole, nb)
    M, R, D = mean.cpu().double().numpy(), rstd.cpu().double().numpy(), _np(dy)
    dx64, dg64, db64 = A.group_norm_grads(X, M, R, D, groups, G, H, act)
    h = (X - wide(M)) * wide(R)
    z = h * (1.0 if G is None else G) + (0.0 if H is None else H)
    zo = 4 * E * (np.abs(h) * gam + np.abs(z) + bet) + 2 * E * np.abs(X * wide(R)) * gam + 1e-30
    slope = A.act_slope(z, act)
    dz = D * slope
    dz_off = np.abs(D) * (np.where(np.abs(z) <= zo, 1.0, 0.0) if act == "relu" else 0.0 if act == "none" else zo + 2e-7 * (1 + np.abs(z))) + 4 * E * np.abs(dz)
    h_off = 4 * E * np.abs(h) + 2 * E * np.abs(X * wide(R))
    m = p * c // groups
    k = (m / 64 + 64) * E
    avg = lambda v: wide(_per_group(v, groups).sum(axis=(1, 3)) / m)
    u, u_off = np.abs(dz) * gam, dz_off * gam + 2 * E * np.abs(dz) * gam
    mgh = np.abs(avg(dz * gam * np.sign(1 if G is None else G) * h))
    mgh_off = avg(u_off * np.abs(h) + u * h_off) + k * avg(u * np.abs(h))
    tol = wide(R) * (u_off + avg(u_off) + k * avg(u) + np.abs(h) * mgh_off + h_off * mgh + 8 * E * (u + avg(u) + np.abs(h) * mgh))
    _close(_np(dxv), dx64, tol + U[t] * np.abs(dx64) + TINY[t], "dx")
    if params:
        k = (n * p / 64 + n + 64) * E
        _close(_np(dg), 2 * dg64, 2 * (dz_off * np.abs(h) + np.abs(dz) * h_off + 2 * k * np.abs(dz * h)).sum(axis=(0, 1)) + E, "dgamma, added twice")
        _close(_np(db), 2 * db64, 2 * (dz_off + 2 * k * np.abs(dz)).sum(axis=(0, 1)) + E, "dbeta, added twice")
    assert _untouched(dxv, dxb)


# one workgroup per image, and three launches; channels in and across eights, a group of one channel, of all, more than a block has
SIZES = [(1, 1, 1, 1), (2, 7, 8, 8), (3, 100, 30, 5), (1, 64, 64, 8), (2, 50, 100, 4), (1, 300, 90, 6), (5, 33, 1024, 1024), (2, 9, 1024, 1),
         (2, 5000, 24, 3), (3, 1200, 200, 25), (1, 40, 2056, 257), (2, 3, 3000, 600), (1, 9000, 12, 12), (2, 2000, 60, 1)]


@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("size", SIZES)
def test_group_norm(size, t):
    acts = ["none", "relu", "silu", "gelu"]
    i = sum(size)
    _case(*size, t, acts[i % 4])
    _case(*size, t, acts[(i + 1) % 4], odd=True)
    _case(*size, t, acts[(i + 2) % 4], affine=False, params=False)


@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("size", [(1, 1, 32, 1), (2, 37, 64, 16), (3, 90, 96, 3), (2, 3000, 32, 4), (1, 777, 320, 32), (1, 11, 2080, 65)])
def test_group_norm_with_an_8_bit_checkpoint(size, t):
    _case(*size, t, "silu", kept=True)
    _case(*size, t, "gelu", kept=True, odd=True)


@pytest.mark.parametrize("size", [(1, 200, 64, 4), (2, 6000, 48, 3)])
def test_group_norm_of_values_far_from_zero(size):
    """Offsets of thousands of spreads: a variance from a sum of squares would
    have lost all its bits."""
    n, p, c, groups = size
    rng = np.random.default_rng(1)
    x = torch.from_numpy(4096.0 + rng.standard_normal((n, p, c))).float().cuda()
    y, mean, rstd = torch.empty_like(x), torch.empty(n, groups, device="cuda"), torch.empty(n, groups, device="cuda")
    B.group_norm_fwd(x, y, groups, mean=mean, rstd=rstd, workspace=_ws(B.group_norm_fwd_workspace_bytes(n, p, c, groups))[0])
    m64, r64, _, y64 = A.group_norm(_np(x), groups)
    # deviations of channels' and blocks' means are exact to e 4096 each, squares of those are below 1e-7
    _close(_np(rstd), r64, 2e-6 * r64, "rstd")
    _close(_np(mean), m64, 4 * E * 4096, "mean")
    _close(_np(y), y64, 4 * E * 4096 + 1e-5 * np.abs(y64), "y")


def test_group_norm_of_nothing():
    x, dg, db = torch.empty(0, 5, 8, device="cuda"), torch.full((8,), 3.0, device="cuda"), torch.full((8,), 3.0, device="cuda")
    m = torch.empty(0, 2, device="cuda")
    B.group_norm_fwd(x, x, 2, mean=m, rstd=m)
    B.group_norm_bwd(x, m, m, x, x, 2, dgamma=dg, dbeta=db, accumulate=True)
    assert (dg == 3).all() and (db == 3).all()
    B.group_norm_bwd(x, m, m, x, x, 2, dgamma=dg, dbeta=db)
    assert (dg == 0).all() and (db == 0).all()
    x, m = torch.empty(3, 0, 8, device="cuda"), torch.empty(3, 2, device="cuda")
    B.group_norm_fwd(x, x, 2)
    B.group_norm_bwd(x, m, m, x, x, 2)


@pytest.mark.parametrize("p", [40, 9000])
def test_group_norm_keeps_infinities_and_nans_in_their_groups(p):
    x = torch.randn(2, p, 16, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    x[0, 3, 5] = float("nan")
    x[1, 7, 15] = float("inf")
    y = torch.empty_like(x)
    mean, rstd = torch.empty(2, 4, device="cuda"), torch.empty(2, 4, device="cuda")
    B.group_norm_fwd(x, y, 4, act="silu", mean=mean, rstd=rstd, workspace=_ws(B.group_norm_fwd_workspace_bytes(2, p, 16, 4))[0])
    assert torch.isnan(rstd[0, 1]) and torch.isnan(rstd[1, 3]) and int(torch.isfinite(rstd).sum()) == int(torch.isfinite(mean).sum()) == 6
    bad = ~torch.isfinite(y).cpu().numpy()
    want = np.zeros((2, p, 16), bool)
    want[0, :, 4:8] = want[1, :, 12:] = True
    np.testing.assert_array_equal(bad, want)
