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
