"""The network head (gaussian_splatting_tile_amd/head.py): its operators run
together through the rasterizer's forward and backward."""

import numpy as np
import pytest
import torch

from gaussian_splatting_tile_amd import binding as B
from gaussian_splatting_tile_amd import head as H
from oracle import network as N
from tests.gpu_util import say

pytestmark = pytest.mark.gpu


def _np(t):
    return t.detach().float().cpu().double().numpy()


def _oracle(head, tokens):
    """The head's planes [rows][m] and what its backward needs, in fp64."""
    s, keep = _np(tokens), []
    for i in range(head.blocks):
        _, rstd, y = N.rms_norm(s, None, _np(head.gamma[i]))
        z, h = N.linear(y, _np(head.w1[i]), _np(head.b1[i]), head.act)
        keep.append((s, rstd, y, z, h))
        s = N.linear(h, _np(head.w2[i]), _np(head.b2[i]), "none", s)[1]
    _, rstd, y = N.rms_norm(s, None, _np(head.gamma[head.blocks]))
    keep.append((s, rstd, y))
    return N.linear(y, _np(head.w_out), _np(head.b_out))[1].T, keep


def _oracle_grads(head, keep, dplanes):
    g = {k: np.zeros(getattr(head, k).shape) for k in head.matrices + head.vectors}
    s, rstd, y = keep[-1]
    dy, g["w_out"], g["b_out"], _ = N.linear_grads(y, _np(head.w_out), None, dplanes.T)
    ds, g["gamma"][head.blocks] = N.rms_norm_grads(s, rstd, dy, _np(head.gamma[head.blocks]))
    for i in reversed(range(head.blocks)):
        s, rstd, y, z, h = keep[i]
        dh, g["w2"][i], g["b2"][i], _ = N.linear_grads(h, _np(head.w2[i]), None, ds)
        dy, g["w1"][i], g["b1"][i], _ = N.linear_grads(y, _np(head.w1[i]), z, dh, head.act)
        ds, g["gamma"][i] = N.rms_norm_grads(s, rstd, dy, _np(head.gamma[i]), ds)
    return g


@pytest.mark.parametrize("dtype,tol", [(torch.float32, 2e-5), (torch.float16, 1e-2), (torch.bfloat16, 6e-2)])
def test_head_forward_and_backward_match_the_oracle(dtype, tol):
    """Relative (Frobenius) errors: some ten roundings in a chain, each of at
    most u (2^-11, 2^-8) of values that the norms keep of one size, and for
    fp32 the sums' error bounds."""
    m, head = 333, H.GaussianHead(333, 64, 96, 3, sh_degree=1, dtype=dtype)
    rng = np.random.default_rng(1)
    for k in head.vectors:
        getattr(head, k).add_(torch.from_numpy(rng.standard_normal(getattr(head, k).shape) * 0.1).float().cuda())
    tokens = torch.from_numpy(rng.standard_normal((m, 64))).to(dtype).cuda()
    planes = head.forward(tokens)
    want, keep = _oracle(head, tokens)
    assert np.linalg.norm(_np(planes) - want) <= tol * np.linalg.norm(want)
    d = rng.standard_normal((head.rows, m))
    head.dplanes.copy_(torch.from_numpy(d))
    head.backward()
    for k, w in _oracle_grads(head, keep, d).items():
        err = np.linalg.norm(_np(head.grads[k]) - w) / np.linalg.norm(w)
        say(f"[gpu] head {dtype} d{k}: {err:.2e}")
        assert err <= tol, (k, err)


def test_head_trains_through_the_rasterizer_and_serves_in_8_bits():
    losses, head, tokens, image, served, target = H.fit(steps=60, say=say)
    assert all(np.isfinite(losses)) and losses[-1] < 0.5 * losses[0], (losses[0], losses[-1])
    assert torch.isfinite(served).all()
    # 8-bit values are within 2^-4 of their own (half a step of 2^-3), and the
    # image moves far less than training moved it
    assert float((served - image).square().mean()) < 0.2 * losses[0]
    planes, eight = _np(head.forward(tokens)), _np(head.serve(tokens))
    assert np.linalg.norm(planes - eight) <= 0.1 * np.linalg.norm(planes)
    one = _np(head.serve(tokens[:1]))
    np.testing.assert_allclose(one[:, 0], eight[:, 0], rtol=0, atol=2e-2 * np.abs(eight[:, 0]).max())
