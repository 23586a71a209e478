"""Network-head operators against the fp64 oracle by the bounds of
limb_model.py, which a kernel that lost a limb exceeds; the in-place forms,
bit by bit; and infinities in rows of any width."""

import numpy as np
import pytest
import torch

from gaussian_splatting_tile_amd import binding as B
from oracle import network as N
from tests import limb_model as M
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

T = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def _np(t):
    return None if t is None else t.detach().float().cpu().double().numpy()


def _make(rng, shape, t, scale=1.0):
    return torch.from_numpy(rng.standard_normal(shape) * scale).to(T[t]).cuda()


def _ws(n):
    return torch.full((max(int(n), 16),), 0xFF, dtype=torch.uint8, device="cuda")        # NaNs in any type


# ---- fp32 products -----------------------------------------------------------
# few rows by 4 and 16 waves; staged by 64 and 128 tiles, with and without splits of k; packed where the result is wide
@pytest.mark.parametrize("planes", [False, True])
@pytest.mark.parametrize("m,n,k", [(5, 700, 136), (16, 4100, 515), (70, 59, 333), (64, 96, 8200), (3000, 200, 700), (1500, 1100, 333), (2300, 1030, 64), (40, 33, 13001)])
def test_linear_f32_keeps_its_limbs(m, n, k, planes):
    say(f"[gpu] fp32 linear {m} {n} {k} planes={planes}")
    rng = np.random.default_rng(m + n + k)
    x, w = _make(rng, (m, k), "f32"), _make(rng, (n, k), "f32", k ** -0.5)
    y = torch.empty((n, m) if planes else (m, n), device="cuda")
    lin = B.linear_struct(x, w, y, planes=planes)
    B.linear_fwd(lin, _ws(B.linear_fwd_workspace_bytes(lin)))
    want = _np(x) @ _np(w).T
    err = M.error(y.cpu(), want.T.copy() if planes else want)
    say(f"[gpu]   error {err:.2e}")
    assert err < M.LINEAR_F32


@pytest.mark.parametrize("planes", [False, True])
@pytest.mark.parametrize("m,n,k", [(70, 59, 333), (900, 600, 58), (700, 640, 700), (2000, 300, 136), (9000, 47, 198), (3, 4099, 33)])
def test_linear_backward_f32_keeps_its_limbs(m, n, k, planes):
    say(f"[gpu] fp32 linear backward {m} {n} {k} planes={planes}")
    rng = np.random.default_rng(m + n + k)
    x, w = _make(rng, (m, k), "f32"), _make(rng, (n, k), "f32", k ** -0.5)
    dy = _make(rng, (n, m) if planes else (m, n), "f32")
    dx, dw, db = torch.empty(m, k, device="cuda"), torch.empty(n, k, device="cuda"), torch.empty(n, device="cuda")
    lin = B.linear_struct(x, w, None, planes=planes)
    gr = B.linear_grads_struct(lin, dy, dx=dx, dw=dw, db=db)
    B.linear_bwd(lin, gr, _ws(B.linear_bwd_workspace_bytes(lin, gr)))
    dz = _np(dy).T if planes else _np(dy)
    for got, want, what in ((dx, dz @ _np(w), "dx"), (dw, dz.T @ _np(x), "dw")):
        err = M.error(got.cpu(), want)
        say(f"[gpu]   {what} error {err:.2e}")
        assert err < M.LINEAR_F32, what


# ---- orthogonalised update ---------------------------------------------------
# one workgroup a matrix, products by 32, 64 and 128 tiles, sums of splits
@pytest.mark.parametrize("e,r,f", [(2, 17, 33), (3, 64, 40), (1, 128, 128), (2, 64, 384), (2, 100, 70), (1, 300, 130), (2, 129, 520), (1, 640, 512),
                                   (1, 58, 700), (2, 64, 1500), (1, 704, 64), (1, 260, 900), (1, 1000, 1030), (4, 256, 256)])
@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
def test_orthogonalize_keeps_its_limbs(e, r, f, t):
    say(f"[gpu] orthogonalize {e}x{r}x{f} {t}")
    rng = np.random.default_rng(r + f)
    g = (_make(rng, (e, r, f), "f32", 1e-3) + _make(rng, (e, r, 1), "f32", 1e-2) * _make(rng, (e, 1, f), "f32")).to(T[t])
    want = [N.orthogonalize(_np(g[i])) for i in range(e)]
    for to in ("f32", "f16", "bf16"):
        out = torch.empty((e, r, f), dtype=T[to], device="cuda")
        mu = B.muon_struct(g, out=out)
        B.orthogonalize(mu, _ws(B.muon_workspace_bytes(mu)))
        errs = [M.error(out[i].float().cpu(), want[i], T[to]) for i in range(e)]
        say(f"[gpu]   to {to}: {max(errs):.2e}")
        assert max(errs) < M.ORTHO[T[to]], to
        if to == t:                                        # over the gradient
            same = g.clone()
            mu = B.muon_struct(same, out=same)
            B.orthogonalize(mu, _ws(B.muon_workspace_bytes(mu)))
            assert torch.equal(same, out)


def test_orthogonalize_of_rank_1_and_small_scales():
    rng = np.random.default_rng(9)
    g = torch.zeros(4, 40, 24, device="cuda")
    g[0] = _make(rng, (40, 1), "f32") * _make(rng, (1, 24), "f32")
    g[1], g[2], g[3] = g[0] * 1e12, g[0] * 1e-6, g[0] * 1e-7
    out = torch.empty_like(g)
    mu = B.muon_struct(g, out=out)
    B.orthogonalize(mu, _ws(B.muon_workspace_bytes(mu)))
    for i in range(4):
        assert M.error(out[i].cpu(), N.orthogonalize(_np(g[i]))) < M.ORTHO_RANK_1, i


@pytest.mark.parametrize("tg,tw", [("f16", "f16"), ("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16"), ("bf16", "f32"), ("f16", "f32")])
@pytest.mark.parametrize("e,r,f", [(2, 64, 128), (1, 200, 100), (1, 300, 513)])
def test_muon_step_of_every_type(e, r, f, tg, tw):
    """w' = w (1 - lr wd) - L with |L| = lr scale |O|: the fp32 step is off by
    the bound of O times |L| and three roundings of w; a 16-bit one differs from
    the rounded w' where O's error d (two limbs: at most 1.5e-4 |L|) carries a value over a rounding boundary, in the mean square
    by d times an ulp (2 u |w'|), and here by no more than twice that."""
    say(f"[gpu] muon {e}x{r}x{f} grad {tg} weight {tw}")
    rng = np.random.default_rng(r)
    g, w, mom = _make(rng, (e, r, f), tg, 1e-2), _make(rng, (e, r, f), tw, 0.1), _make(rng, (e, r, f), "f32", 1e-2)
    h = dict(lr=0.03, beta=0.9, weight_decay=0.1, scale=1.5)
    mo, wo = torch.empty_like(mom), torch.empty_like(w)
    mu = B.muon_struct(g, momentum=mom, weight=w, momentum_out=mo, weight_out=wo, **h)
    B.muon_step(mu, _ws(B.muon_workspace_bytes(mu)))
    for i in range(e):
        m64, w64 = N.muon_step(_np(g[i]), _np(mom[i]), _np(w[i]), **h)
        assert np.linalg.norm(_np(mo[i]) - m64) <= 2.0 ** -23 * np.linalg.norm(m64)
        step, size = np.linalg.norm(w64 - _np(w[i]) * (1 - h["lr"] * h["weight_decay"])), np.linalg.norm(w64)
        if tw == "f32":
            err, bound = np.linalg.norm(_np(wo[i]) - w64), M.ORTHO[torch.float32] * step + 3 * 2.0 ** -24 * size
        else:
            u = 2.0 ** -11 if tw == "f16" else 2.0 ** -8
            err = np.linalg.norm(_np(wo[i]) - torch.from_numpy(w64).to(T[tw]).double().numpy())
            bound = 2 * np.sqrt(1.5e-4 * step * 2 * u * size + (1.5e-4 * step) ** 2)
        say(f"[gpu]   {err:.2e} of {bound:.2e}")
        assert err <= bound


# ---- norm --------------------------------------------------------------------
# widths of every group of lanes whose last vector overlaps the one before, and rows read twice
WIDTHS = [(9, 5), (40, 37), (33, 129), (17, 513), (9, 1027), (6, 2051), (5, 4099), (3, 8195)]


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("m,n", WIDTHS)
def test_norm_in_place(m, n, t):
    """Every form that may write over its inputs gives the bits of the one that
    does not."""
    rng = np.random.default_rng(n)
    x, r, g = _make(rng, (m, n), t), _make(rng, (m, n), t), 1 + _make(rng, (n,), "f32", 0.2)
    y, s = torch.empty_like(x), torch.empty_like(x)
    rstd = torch.empty(m, device="cuda")
    B.rms_norm_fwd(x, y, gamma=g, residual=r, sum_out=s, rstd=rstd)
    for y_in, s_in in (("x", "r"), ("r", "x"), ("x", None), ("r", None), (None, "x"), (None, "r")):
        xv, rv = x.clone(), r.clone()
        at = {"x": xv, "r": rv}
        yv, sv = at.get(y_in, torch.empty_like(x)), at.get(s_in, torch.empty_like(x))
        B.rms_norm_fwd(xv, yv, gamma=g, residual=rv, sum_out=sv)
        assert torch.equal(yv, y) and torch.equal(sv, s), (y_in, s_in)
    B.rms_norm_fwd(x, y)
    xv = x.clone()
    B.rms_norm_fwd(xv, xv)
    assert torch.equal(xv, y)

    dy, ds, dx, dg = _make(rng, (m, n), t), _make(rng, (m, n), t), torch.empty_like(x), torch.empty(n, device="cuda")
    ws = _ws(B.rms_norm_bwd_workspace_bytes(m, n))
    B.rms_norm_bwd(s, rstd, dy, dx, gamma=g, dsum=ds, dgamma=dg, workspace=ws)
    for over in ("dy", "dsum"):
        a, b, dg2 = dy.clone(), ds.clone(), torch.empty_like(dg)
        to = a if over == "dy" else b
        B.rms_norm_bwd(s, rstd, a, to, gamma=g, dsum=b, dgamma=dg2, workspace=ws)
        assert torch.equal(to, dx) and torch.equal(dg2, dg), over


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("m,n", WIDTHS)
def test_norm_of_infinities_anywhere(m, n, t):
    """rstd of a row with an infinity is 0: its values give 0 and the infinity
    itself 0 times infinity, wherever it stands."""
    at = torch.arange(max(0, n - 64), n, device="cuda")    # the row's last columns
    rows = torch.ones(len(at), n, dtype=T[t], device="cuda")
    rows[torch.arange(len(at), device="cuda"), at] = float("inf")
    y, rstd = torch.empty_like(rows), torch.empty(len(at), device="cuda")
    B.rms_norm_fwd(rows, y, rstd=rstd)
    assert (rstd == 0).all()
    inf = torch.isinf(rows)
    assert torch.isnan(y[inf]).all() and (y[~inf] == 0).all()
