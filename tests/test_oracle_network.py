"""Pins of the network-head oracle (oracle/network.py) to things other than
itself: torch's own layers and autograd in fp64, central differences, the
format's table, and closed forms of the Newton-Schulz iteration."""

import numpy as np
import pytest
import torch

from oracle import network as N


def _t(a):
    return torch.from_numpy(np.asarray(a, np.float64)).requires_grad_(True)


def test_norm_and_its_gradient_match_autograd():
    rng = np.random.default_rng(1)
    x, r, g, dy, ds = (rng.standard_normal(s) for s in ((5, 37), (5, 37), 37, (5, 37), (5, 37)))
    tx, tr, tg = _t(x), _t(r), _t(g)
    s = tx + tr
    y = torch.nn.functional.rms_norm(s, (37,), tg, 1e-6)
    (y * torch.from_numpy(dy)).sum().backward(retain_graph=True)
    (s * torch.from_numpy(ds)).sum().backward()
    so, rstd, yo = N.rms_norm(x, r, g, 1e-6)
    dx, dg = N.rms_norm_grads(so, rstd, dy, g, ds)
    np.testing.assert_allclose(yo, y.detach().numpy(), rtol=1e-12, atol=1e-13)
    np.testing.assert_allclose(dx, tx.grad.numpy(), rtol=1e-11, atol=1e-12)
    np.testing.assert_allclose(dx, tr.grad.numpy(), rtol=1e-11, atol=1e-12)
    np.testing.assert_allclose(dg, tg.grad.numpy(), rtol=1e-11, atol=1e-12)


def test_norm_gradient_matches_differences():
    rng = np.random.default_rng(2)
    x, g, dy = rng.standard_normal((3, 9)), rng.standard_normal(9), rng.standard_normal((3, 9))
    s, rstd, _ = N.rms_norm(x, None, g, 1e-3)
    dx, dg = N.rms_norm_grads(s, rstd, dy, g)
    f = lambda x, g: float((N.rms_norm(x, None, g, 1e-3)[2] * dy).sum())
    h = 1e-6
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = h
        assert abs((f(x + e, g) - f(x - e, g)) / (2 * h) - dx[i]) < 1e-7
    for j in range(9):
        e = np.zeros(9)
        e[j] = h
        assert abs((f(x, g + e) - f(x, g - e)) / (2 * h) - dg[j]) < 1e-7


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
def test_linear_and_its_gradient_match_autograd_and_differences(act):
    rng = np.random.default_rng(3)
    x, w, b, r, dy = (rng.standard_normal(s) for s in ((6, 5), (4, 5), 4, (6, 4), (6, 4)))
    tx, tw, tb, tr = _t(x), _t(w), _t(b), _t(r)
    F = torch.nn.functional
    z = F.linear(tx, tw, tb)
    y = {"none": lambda v: v, "relu": F.relu, "silu": F.silu, "gelu": F.gelu}[act](z) + tr
    (y * torch.from_numpy(dy)).sum().backward()
    zo, yo = N.linear(x, w, b, act, r)
    dx, dw, db, _ = N.linear_grads(x, w, zo, dy, act)
    for got, want in ((yo, y.detach()), (dx, tx.grad), (dw, tw.grad), (db, tb.grad)):
        np.testing.assert_allclose(got, want.numpy(), rtol=1e-11, atol=1e-12)
    np.testing.assert_allclose(dy, tr.grad.numpy())
    h = 1e-6
    f = lambda x: float((N.linear(x, w, b, act, r)[1] * dy).sum())
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = h
        assert abs((f(x + e) - f(x - e)) / (2 * h) - dx[i]) < 1e-6


def test_e4m3_table_and_rounding_match_torch():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(N.e4m3_table(), want)
    v = np.concatenate([np.linspace(-448, 448, 4099), np.ldexp(1.0, np.arange(-12, 9)) * 1.0625, [0.0]])
    v = np.concatenate([v, np.zeros(-len(v) % 32)])
    v[::32] = 448.0                                     # every block's scale is 1
    q, s = N.mxfp8_quantize(v[None])
    assert (s == 127).all()
    np.testing.assert_array_equal(N.mxfp8_value(q, s)[0], torch.from_numpy(v).to(torch.float8_e4m3fn).double().numpy())


def test_block_scale_is_the_smallest_that_fits():
    v = np.zeros((1, 32 * 6))
    tops = [448.0, 449.0, 1e-30, 0.0, 3.5, np.inf]
    for i, t in enumerate(tops):
        v[0, 32 * i + 5] = t
    q, s = N.mxfp8_quantize(v)
    assert list(s[0]) == [127, 128, 127 - 108, 0, 127 - 7, 255]
    back = N.mxfp8_value(q, s)[0]
    assert back[5] == 448.0 and back[32 + 5] == 448.0 and back[3 * 32 + 5] == 0.0 and back[4 * 32 + 5] == 3.5
    assert np.isnan(back[5 * 32:]).all() and 1e-30 / 2 ** -108 <= 448


def test_orthogonalize_matches_the_matrix_iteration():
    rng = np.random.default_rng(4)
    for shape in ((7, 11), (11, 7), (6, 6), (1, 5)):
        u = rng.standard_normal(shape)
        x = u / (np.linalg.norm(u) + 1e-7)
        x = x.T if shape[0] > shape[1] else x
        a, b, c = N.COEFFS
        for _ in range(5):
            g = x @ x.T
            x = a * x + (b * g + c * g @ g) @ x
        x = x.T if shape[0] > shape[1] else x
        np.testing.assert_allclose(N.orthogonalize(u), x, rtol=0, atol=1e-11)


def test_orthogonalize_closed_forms():
    # a multiple of an orthogonal matrix: every singular value is 1 / sqrt(n) at the start
    q = np.linalg.qr(np.random.default_rng(5).standard_normal((8, 8)))[0]
    s = 1 / np.sqrt(8.0)
    for _ in range(5):
        s = N.COEFFS[0] * s + N.COEFFS[1] * s ** 3 + N.COEFFS[2] * s ** 5
    np.testing.assert_allclose(N.orthogonalize(3.0 * q), s * q, rtol=0, atol=1e-7)
    np.testing.assert_array_equal(N.orthogonalize(np.zeros((3, 4))), np.zeros((3, 4)))
    # classical coefficients converge to the polar factor
    u = np.random.default_rng(6).standard_normal((5, 9))
    p, _, t = np.linalg.svd(u, full_matrices=False)
    np.testing.assert_allclose(N.orthogonalize(u, steps=40, coeffs=(1.5, -0.5, 0.0)), p @ t, rtol=0, atol=1e-10)
