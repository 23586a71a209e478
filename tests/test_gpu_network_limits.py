"""Network-head calls at the far end of the sizes that include/gs.h names:
more blocks than one dimension of a launch takes, and arrays whose elements lie
past 32-bit offsets on every way of the products.  Values are chosen so that
the results are exact, or are compared with fp64 at the far end."""

import numpy as np
import pytest
import torch

from gaussian_splatting_tile_amd import binding as B
from oracle import network as N
from tests.gpu_util import say

pytestmark = pytest.mark.gpu


def _ws(n):
    return torch.empty(max(int(n), 16), dtype=torch.uint8, device="cuda")


def _call(f):
    """f(); a refusal is reported without its arguments, gigabytes each."""
    try:
        f()
    except B.GsError as e:
        pytest.fail(str(e), pytrace=False)


def _all(t):
    return bool(t.all())


@pytest.fixture(autouse=True)
def _release():
    yield
    torch.cuda.empty_cache()


def test_norm_of_more_rows_than_a_launch_has_threads():
    """2^28 rows by 16 lanes each are 2^32 threads.  Rows of one magnitude norm
    to their signs."""
    m, n = (1 << 28) + 3, 8
    say(f"[gpu] norm {m}x{n}")
    x = torch.full((m, n), 2.0, dtype=torch.bfloat16, device="cuda")
    x[1::2] = -0.5
    rstd = torch.zeros(m, device="cuda")
    _call(lambda: B.rms_norm_fwd(x, x, rstd=rstd, eps=0.0))
    ok = _all(x[::2] == 1.0), _all(x[1::2] == -1.0), _all(rstd[::2] == 0.5), _all(rstd[1::2] == 2.0)
    assert all(ok), ok


def test_quantise_of_more_rows_than_a_launch_has_threads():
    m = (1 << 28) + 3
    say(f"[gpu] quantise {m}x32")
    x = torch.full((m, 32), 2.0, dtype=torch.bfloat16, device="cuda")
    x[1::2] = 1.0
    codes, scales = torch.zeros(m, 32, dtype=torch.float8_e4m3fn, device="cuda"), torch.zeros(m, 1, dtype=torch.uint8, device="cuda")
    _call(lambda: B.mxfp8_quantize(x, codes, scales))
    # 256 = 2 x 2^7 = 1 x 2^8
    ok = _all(codes.view(torch.uint8) == 0x78), _all(scales[::2] == 127 - 7), _all(scales[1::2] == 127 - 8)
    assert all(ok), ok


@pytest.mark.parametrize("planes", [False, True])
@pytest.mark.parametrize("t", [torch.bfloat16, torch.float32])
def test_linear_of_more_tiles_than_a_launch_takes(t, planes):
    """2^30 rows in tiles of 64 by 256 threads or of 128 by 512 are 2^32
    threads.  Small whole numbers, so every result is exact."""
    m = 1 << 30
    say(f"[gpu] linear {m} x 1 x 1 {t} planes={planes}")
    x = torch.arange(m, dtype=torch.int32, device="cuda").remainder_(63).to(t).view(m, 1)
    xs = x.view(1, m) if planes else x
    w, b, y, z = torch.full((1, 1), 2.0, dtype=t, device="cuda"), torch.ones(1, device="cuda"), torch.zeros_like(xs), torch.zeros_like(x)
    lin = B.linear_struct(x, w, y, bias=b, residual=xs, z=z, planes=planes)
    _call(lambda: B.linear_fwd(lin, _ws(B.linear_fwd_workspace_bytes(lin))))
    z -= 1
    y -= 1
    ok = _all(z == 2 * x), _all(y == 3 * xs)
    assert all(ok), ok
    lin = B.linear_struct(x, w, None, planes=planes)
    gr = B.linear_grads_struct(lin, xs, dx=z)
    z.zero_()
    _call(lambda: B.linear_bwd(lin, gr, _ws(B.linear_bwd_workspace_bytes(lin, gr))))
    ok = _all(z == 2 * x)
    assert ok, "dx"


def test_linear_backward_of_no_rows_into_a_large_dw():
    n = 1 << 16
    say(f"[gpu] dw of {n} x {n} over no rows")
    x, dy = torch.zeros(0, n, dtype=torch.bfloat16, device="cuda"), torch.zeros(0, n, dtype=torch.bfloat16, device="cuda")
    dw = torch.ones(n, n, dtype=torch.bfloat16, device="cuda")
    lin = B.linear_struct(x, dw, None)
    gr = B.linear_grads_struct(lin, dy, dw=dw)
    _call(lambda: B.linear_bwd(lin, gr))
    ok = not bool(dw.any())
    assert ok, "dw"


# ---- rows more than 2^31 elements into every array -----------------------------
STRIDE, ROWS = 60000, 40000


def _np(t):
    return t.detach().float().cpu().double().numpy()


def _views(t, *widths):
    buf = torch.empty(ROWS * STRIDE, dtype=t, device="cuda").view(ROWS, STRIDE)
    at, out = 0, []
    for w in widths:
        out.append(buf[:, at:at + w])
        at += (w + 127) // 128 * 128
    return out


def _near(got, want, tol):
    assert np.linalg.norm(_np(got) - want) <= tol * np.linalg.norm(want)


TAIL = slice(ROWS - 70, ROWS)


@pytest.mark.parametrize("n,k,shift", [(64, 72, 0), (1100, 40, 0), (300, 72, 1)])
@pytest.mark.parametrize("t,tol", [(torch.float32, 2e-6), (torch.bfloat16, 6e-3)])
def test_offsets_past_32_bits_converted_while_loading_and_packed(t, tol, n, k, shift):
    """The bounds: limb_model.py's for fp32, and bf16's rounding (rms below
    2^-8) of dz and of the result."""
    say(f"[gpu] far rows {n} {k} {t}")
    gen = torch.Generator(device="cuda").manual_seed(n)
    x, y, z, dy, dx = (v[:, shift:] for v in _views(t, k + shift, n + shift, n + shift, n + shift, k + shift))
    w = (torch.randn(n, k, generator=gen, device="cuda") * k ** -0.5).to(t)
    for v in (x, dy):
        v.copy_(torch.randn(v.shape, generator=gen, device="cuda"))
    lin = B.linear_struct(x, w, y, z=z, act="relu")
    B.linear_fwd(lin, _ws(B.linear_fwd_workspace_bytes(lin)))
    z64, y64 = N.linear(_np(x[TAIL]), _np(w), None, "relu")
    _near(y[TAIL], y64, tol)
    _near(z[TAIL], z64, tol)
    dw, db = torch.empty(n, k, device="cuda"), torch.empty(n, device="cuda")
    gr = B.linear_grads_struct(lin, dy, dx=dx, dw=dw, db=db)
    B.linear_bwd(lin, gr, _ws(B.linear_bwd_workspace_bytes(lin, gr)))
    dz = torch.where(z > 0, dy, torch.zeros((), dtype=t, device="cuda"))
    _near(dx[TAIL], _np(dz[TAIL]) @ _np(w), tol)
    _near(dw, _np(dz.double().t() @ x.double()), tol)
    _near(db, _np(dz.double().sum(0)), 1e-5)
    rstd, dg = torch.empty(ROWS, device="cuda"), torch.empty(n, device="cuda")
    B.rms_norm_fwd(y, z, residual=dy, sum_out=y, rstd=rstd)
    s64, r64, z64 = N.rms_norm(_np(y[TAIL]))
    _near(z[TAIL], z64, tol)
    B.rms_norm_bwd(y, rstd, dy, z, dgamma=dg, workspace=_ws(B.rms_norm_bwd_workspace_bytes(ROWS, n)))
    _near(z[TAIL], N.rms_norm_grads(s64, _np(rstd[TAIL]), _np(dy[TAIL]))[0], tol)


def test_offsets_past_32_bits_of_the_weights_of_few_rows():
    gen = torch.Generator(device="cuda").manual_seed(3)
    w, = _views(torch.bfloat16, 72)
    w.copy_(torch.randn(w.shape, generator=gen, device="cuda"))
    x = torch.randn(2, 72, generator=gen, device="cuda").bfloat16()
    y = torch.empty(2, ROWS, device="cuda")
    lin = B.linear_struct(x, w, y)
    B.linear_fwd(lin, _ws(B.linear_fwd_workspace_bytes(lin)))
    _near(y[:, TAIL], _np(x) @ _np(w[TAIL]).T, 1e-6)


@pytest.mark.parametrize("ty,tol", [(torch.bfloat16, 3e-3), (torch.float32, 1e-6)])
def test_offsets_past_32_bits_of_8_bit_rows(ty, tol):
    gen = torch.Generator(device="cuda").manual_seed(4)
    x, = _views(torch.bfloat16, 96)
    x.copy_(torch.randn(x.shape, generator=gen, device="cuda"))
    codes, scales = _views(torch.uint8, 96, 3)
    w = torch.randn(64, 96, generator=gen, device="cuda")
    wc, wsc = torch.empty(64, 96, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(64, 3, dtype=torch.uint8, device="cuda")
    B.mxfp8_quantize(w, wc, wsc)
    B.mxfp8_quantize(x, codes.view(torch.float8_e4m3fn), scales)
    c64, s64 = N.mxfp8_quantize(_np(x[TAIL]))
    assert (scales[TAIL].cpu().numpy() == s64).all()
    y = torch.empty(ROWS, 64, dtype=ty, device="cuda")
    lin = B.linear_struct(codes.view(torch.float8_e4m3fn), wc, y, x_scales=scales, w_scales=wsc)
    B.linear_fwd(lin, _ws(B.linear_fwd_workspace_bytes(lin)))
    want = N.mxfp8_value(c64, s64) @ N.mxfp8_value(wc.view(torch.uint8).cpu().numpy(), wsc.cpu().numpy()).T
    _near(y[TAIL], want, tol)


def test_offsets_past_32_bits_of_planes():
    m, n, k, stride = 70000, 60, 64, 40_000_000
    gen = torch.Generator(device="cuda").manual_seed(5)
    buf = torch.empty(n, stride, device="cuda")
    y, dy = buf[:, 8:8 + m], buf[:, 100_000:100_000 + m]
    x, w = torch.randn(m, k, generator=gen, device="cuda").bfloat16(), torch.randn(n, k, generator=gen, device="cuda").bfloat16()
    dy.copy_(torch.randn(n, m, generator=gen, device="cuda"))
    z = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    lin = B.linear_struct(x, w, y, z=z, act="relu", planes=True)
    B.linear_fwd(lin, _ws(B.linear_fwd_workspace_bytes(lin)))
    z64 = x.double() @ w.double().t()
    _near(y, _np(z64.clamp(min=0).t()), 2e-6)
    dx, dw, db = torch.empty_like(x), torch.empty(n, k, device="cuda"), torch.empty(n, device="cuda")
    gr = B.linear_grads_struct(lin, dy, dx=dx, dw=dw, db=db)
    B.linear_bwd(lin, gr, _ws(B.linear_bwd_workspace_bytes(lin, gr)))
    dz = torch.where(z.t() > 0, dy, torch.zeros((), device="cuda")).double()
    _near(dx, _np(dz.t() @ w.double()), 6e-3)
    _near(dw, _np(dz @ x.double()), 6e-3)
    _near(db, _np(dz.sum(1)), 1e-5)


def test_orthogonalize_of_a_batch_past_32_bit_offsets():
    e, r, f = 34000, 64, 1024
    say(f"[gpu] orthogonalize {e}x{r}x{f}")
    g = torch.randn(e, r, f, generator=torch.Generator(device="cuda").manual_seed(6), device="cuda", dtype=torch.bfloat16)
    mu = B.muon_struct(g, out=g)
    last = _np(g[-1])
    B.orthogonalize(mu, _ws(B.muon_workspace_bytes(mu)))
    want = torch.from_numpy(N.orthogonalize(last)).bfloat16().double().numpy()
    assert np.linalg.norm(_np(g[-1]) - want) <= 3e-3 * np.linalg.norm(want)
