"""Infinities in rows of any width."""

import pytest
import torch

from gaussian_splatting_tile_amd import binding as B

pytestmark = pytest.mark.gpu

T = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ---- norm --------------------------------------------------------------------
# widths of every group of lanes whose last vector overlaps the one before, and rows read twice
WIDTHS = [(9, 5), (40, 37), (33, 129), (17, 513), (9, 1027), (6, 2051), (5, 4099), (3, 8195)]


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
