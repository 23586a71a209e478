"""The attention oracle against closed forms and differences."""

import numpy as np
import pytest

from oracle import attention as A


def test_equal_scores_average_the_values():
    rng = np.random.default_rng(0)
    v = rng.standard_normal((2, 7, 1, 3))
    out, lse, p = A.attention(np.zeros((2, 4, 2, 3)), rng.standard_normal((2, 7, 1, 3)), v, 0.5, A.seen_keys(2, 7, [7, 3]))
    np.testing.assert_allclose(out[0], np.broadcast_to(v[0].mean(0), (4, 2, 3)), atol=1e-15)
    np.testing.assert_allclose(out[1], np.broadcast_to(v[1, :3].mean(0), (4, 2, 3)), atol=1e-15)
    np.testing.assert_allclose(lse, np.log([[[7.0]], [[3.0]]]) + np.zeros((2, 2, 4)), atol=1e-15)
    assert (p[1, ..., 3:] == 0).all()


def test_nothing_attended():
    z = np.ones((1, 2, 1, 3))
    out, lse, _ = A.attention(z, z, z, 1.0, A.seen_keys(1, 2, None, [[0, 0]]))
    assert (out == 0).all() and (lse == -np.inf).all()


@pytest.mark.parametrize("g", [1, 3])
def test_gradients_against_differences(g):
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((2, 4, 2 * g, 5)), rng.standard_normal((2, 6, 2, 5)), rng.standard_normal((2, 6, 2, 5))
    w, seen = rng.standard_normal(q.shape), A.seen_keys(2, 6, [6, 4], rng.random((2, 6)) < 0.8)
    f = lambda: float((A.attention(q, k, v, 0.4, seen)[0] * w).sum())
    out, lse, _ = A.attention(q, k, v, 0.4, seen)
    grads = A.attention_grads(q, k, v, 0.4, seen, out, lse, w)
    for x, dx in zip((q, k, v), grads):
        for at in zip(*(rng.integers(0, n, 12) for n in x.shape)):
            keep, h = x[at], 1e-5
            x[at] = keep + h
            up = f()
            x[at] = keep - h
            down = f()
            x[at] = keep
            assert abs((up - down) / (2 * h) - dx[at]) < 1e-8


@pytest.mark.parametrize("activation", ["none", "relu", "silu", "gelu"])
def test_group_norm_gradients_against_differences(activation):
    rng = np.random.default_rng(2)
    x, gamma, beta = rng.standard_normal((2, 3, 6)) + 1.0, 1 + 0.2 * rng.standard_normal(6), 0.3 * rng.standard_normal(6)
    w = rng.standard_normal(x.shape)
    f = lambda: float((A.group_norm(x, 2, gamma, beta, activation, 1e-3)[3] * w).sum())
    mean, rstd, z, _ = A.group_norm(x, 2, gamma, beta, activation, 1e-3)
    assert np.abs(z).min() > 1e-3                       # no kink within the differences
    for v, dv in zip((x, gamma, beta), A.group_norm_grads(x, mean, rstd, w, 2, gamma, beta, activation)):
        for at in np.ndindex(v.shape):
            keep, h = v[at], 1e-5
            v[at] = keep + h
            up = f()
            v[at] = keep - h
            down = f()
            v[at] = keep
            assert abs((up - down) / (2 * h) - dv[at]) < 1e-7


def test_group_norm_of_one_group_of_equal_values():
    mean, rstd, z, y = A.group_norm(np.full((1, 4, 2), 3.0), 1, eps=0.25)
    assert mean[0, 0] == 3.0 and rstd[0, 0] == 2.0 and (y == 0).all()
