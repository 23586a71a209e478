"""fp32 probabilities of the backward where scores are large: P = exp(S - lse) from
the lse that it is given.

Scores are exact here (multiples of 1/4, few bits), so is dout . v, and delta is 0.  E =
2^-24.  With x = S - lse the difference is rounded once (E |x|), taken to base 2 (E |x|
and the constant's 0.3 E |x|) and raised (two ulp: 4 E); P's limbs, a product with 1 and the
result's rounding add less than 4 E, a product with a small integer and the scale
3 E more.  A difference taken in units of log 2 from rounded products would be off by E (|S| + |lse|)
log2 e instead: S is 50 to 60 here, x -9 to 0."""

import math

import pytest
import torch

from gaussian_splatting_tile_amd import binding as B

pytestmark = pytest.mark.gpu

E = 2.0 ** -24


@pytest.mark.parametrize("scale", [0.7, 0.0883883461, 1.3])
@pytest.mark.parametrize("nk,d", [(1, 8), (40, 40), (1500, 64), (300, 128)])
def test_probabilities_of_large_scores(nk, d, scale):
    scale = float(torch.tensor(scale, dtype=torch.float32))
    k, q = torch.zeros(1, nk, 1, d), torch.zeros(1, 1, 1, d)
    near = torch.arange(nk) % 40                            # steps of a score
    top = round(60 / scale * 4) / 4
    q[..., 0], q[..., 1] = 1.0, 1.0
    k[0, :, 0, 0], k[0, :, 0, 1] = top, -torch.floor(near * 0.2 / scale * 4) / 4
    v, dout = torch.zeros(1, nk, 1, d), torch.zeros(1, 1, 1, d)
    v[0, :, 0, 2], dout[..., 2] = 3.0, 1.0
    q, k, v, dout = (t.cuda() for t in (q, k, v, dout))
    S = (k[0, :, 0, 0].double() + k[0, :, 0, 1].double()) * scale
    lse = torch.logsumexp(S, 0).float().view(1, 1, 1)
    x = S - lse.double().view(())
    P = torch.exp(x)
    out, dq, dk, dv = torch.zeros_like(q), torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    a = B.attention_struct(q, k, v, out, lse=lse, scale=scale)
    g = B.attention_grads_struct(a, dout, dq=dq, dk=dk, dv=dv)
    B.attention_bwd(a, g, torch.empty(max(16, B.attention_bwd_workspace_bytes(a, g)), dtype=torch.uint8, device="cuda"))
    off = E * (2.3 * x.abs() + 8)
    err = (dv[0, :, 0, 2].double() / P - 1).abs()
    assert bool((err <= off).all()), float((err / off).max())
    err = (dk[0, :, 0, :2].double() / (3 * scale * P)[:, None] - 1).abs()
    assert bool((err <= (off + 3 * E)[:, None]).all()), float((err / off[:, None]).max())
    want = scale * 3 * (P[:, None] * k[0, :, 0].double()).sum(0)
    bound = scale * 3 * ((P * (off + 3 * E))[:, None] * k[0, :, 0].double().abs()).sum(0) + (nk / 2 + 8) * E * want.abs()
    assert bool(((dq[0, 0, 0].double() - want).abs() <= bound + 1e-30).all())
    assert math.isfinite(float(dq.sum()))


@pytest.mark.parametrize("scale", [0.7, 0.0883883461, 1.3, 0.11, 0.4142])
@pytest.mark.parametrize("nq,nk", [(1, 1), (1, 40), (130, 64), (3, 4096), (40, 1500)])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_lse_of_large_scores_and_the_gradients_that_take_it(nq, nk, scale, sign):
    """lse is the largest score, rounded, which the differences from it take as it is, and the log of a
    sum: off by its own rounding, E |lse|, and what the sum is: E (2.3 x 9 + 4) for its terms, nk / 32 + 40
    additions of 32 a tile, of tiles and of splits, and 2 of the log and its product.  dv of what the forward kept
    is then off by as much of P, and by what it adds itself."""
    d, scale = 16, float(torch.tensor(scale, dtype=torch.float32))
    k, q = torch.zeros(1, nk, 1, d), torch.zeros(1, nq, 1, d)
    near = torch.arange(nk) % 40
    q[..., 0], q[..., 1] = 1.0, 1.0
    k[0, :, 0, 0], k[0, :, 0, 1] = sign * round(60 / scale * 4) / 4, -torch.floor(near * 0.2 / scale * 4) / 4
    v, dout = torch.zeros(1, nk, 1, d), torch.zeros(1, nq, 1, d)
    dout[0, 0, 0, 2] = 1.0
    q, k, v, dout = (t.cuda() for t in (q, k, v, dout))
    S = (k[0, :, 0, 0].double() + k[0, :, 0, 1].double()) * scale
    want = torch.logsumexp(S, 0)
    out, lse, dv = torch.empty_like(q), torch.empty(1, 1, nq, device="cuda"), torch.empty_like(k)
    a = B.attention_struct(q, k, v, out, lse=lse, scale=scale)
    B.attention_fwd(a, torch.empty(max(16, B.attention_fwd_workspace_bytes(a)), dtype=torch.uint8, device="cuda"))
    off = E * (float(want.abs()) + 26.7 + nk / 32 + 42)
    if nk == 1:
        off = E * float(want.abs())                        # the score itself, rounded
    assert float((lse.double() - want).abs().max()) <= off, float((lse.double() - want).abs().max()) / off
    g = B.attention_grads_struct(a, dout, dv=dv)
    B.attention_bwd(a, g, torch.empty(max(16, B.attention_bwd_workspace_bytes(a, g)), dtype=torch.uint8, device="cuda"))
    P = torch.exp(S - want)
    err = (dv[0, :, 0, 2].double() / P - 1).abs()
    bound = off + E * (2.3 * (S - want).abs() + 8)
    assert bool((err <= bound * 1.001).all()), float((err / bound).max())
