"""The network head's own checks, before any kernel runs."""

import pytest
import torch

from gaussian_splatting_tile_amd.head import GaussianHead


def test_training_takes_all_tokens():
    """One token, or one column, would be repeated over the whole batch."""
    head = GaussianHead(6, 32, 64, 1, sh_degree=0, device="cpu")
    for shape in ((1, 32), (5, 32), (7, 32), (6, 1), (32,)):
        before = head.s[0].clone()
        with pytest.raises(ValueError, match="tokens"):
            head.forward(torch.ones(shape))
        assert torch.equal(head.s[0].nan_to_num(), before.nan_to_num())
