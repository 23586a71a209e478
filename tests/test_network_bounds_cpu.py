"""The bounds of limb_model.py tell a result from one that has lost a limb."""

import numpy as np
import pytest
import torch

from oracle import network as N
from tests import limb_model as M


@pytest.mark.parametrize("k", [32, 136, 700, 2048])
def test_product_bound(k):
    rng = np.random.default_rng(k)
    a, b = torch.from_numpy(rng.standard_normal((40, k))).float(), torch.from_numpy(rng.standard_normal((33, k)) * k ** -0.5).float()
    want = a.double() @ b.double().T
    assert M.error(M.product(a, b, 3), want) < M.LINEAR_F32 < M.error(M.product(a, b, 2), want)


@pytest.mark.parametrize("r,f", [(17, 33), (33, 20), (100, 70), (64, 384)])
def test_orthogonalize_bounds(r, f):
    rng = np.random.default_rng(r + f)
    g = torch.from_numpy(rng.standard_normal((r, f)) * 1e-3 + rng.standard_normal((r, 1)) * 1e-2 * rng.standard_normal((1, f))).float()
    want = N.orthogonalize(g.double().numpy())
    for t, nl in ((torch.float32, 3), (torch.bfloat16, 2), (torch.float16, 2)):
        good, bad = (M.error(M.orthogonalize(g, n).to(t), want, t) for n in (nl, nl - 1))
        assert good < M.ORTHO[t] < bad, (t, good, bad)


@pytest.mark.parametrize("scale", [1.0, 1e12, 1e-6])
def test_rank_1_bound(scale):
    """And from one without eps, where that matters (1e-7 beside 1e-6 |u v^T|)."""
    rng = np.random.default_rng(7)
    g = (torch.from_numpy(rng.standard_normal((40, 1))).float() * torch.from_numpy(rng.standard_normal((1, 24))).float() * scale).float()
    want = N.orthogonalize(g.double().numpy())
    assert M.error(M.orthogonalize(g, 3), want) < M.ORTHO_RANK_1 < M.error(M.orthogonalize(g, 2), want)
    if scale < 1e-3:
        assert M.error(M.orthogonalize(g, 3, eps=0.0), want) > M.ORTHO_RANK_1
