"""ViewReader's own checks (gaussian_splatting_tile_amd/head.py), before any kernel runs."""

import pytest
import torch

from gaussian_splatting_tile_amd.head import ViewReader


def test_reader_takes_maps_of_its_own_type():
    """Zeroing views that are not there would turn others into it without a word."""
    r = ViewReader(6, 32, 2, 5, 32, 2, 4, device="cpu")
    for seen in (None, torch.ones(2, dtype=torch.bool)):
        with pytest.raises(ValueError, match="features"):
            r.forward(torch.ones(6, 32), torch.ones(2, 5, 32), seen)


@pytest.mark.parametrize("width,channels,heads,groups", [(256, 32, 1, 4), (416, 32, 2, 4), (64, 96, 2, 5), (48, 32, 2, 4), (64, 48, 2, 4), (64, 32, 3, 4)])
def test_reader_refuses_what_its_operators_do(width, channels, heads, groups):
    """Before any buffer is made, not at the first forward."""
    with pytest.raises(AssertionError):
        ViewReader(6, width, 2, 5, channels, heads, groups, device="cpu")
    ViewReader(6, 256, 2, 5, 96, 2, 6, device="cpu")
