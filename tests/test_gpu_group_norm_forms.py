"""The group norm's forms that many images or wide groups take, against the fp64
oracle as tests/test_gpu_group_norm.py has it: an image per workgroup whose
values are read again, sums of a hundred images' gradients, groups of more
channels than a workgroup has threads."""

import pytest

from tests.test_gpu_group_norm import _case

pytestmark = pytest.mark.gpu

# more pixels than a workgroup's registers hold (4 x 512 / eights of channels), up to 8192 / eights
MANY = [(130, 700, 24, 3), (128, 270, 60, 5), (129, 2100, 8, 2), (128, 2060, 3, 1)]


@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("size", MANY)
def test_many_images_of_a_workgroup_each(size, t):
    _case(*size, t, "silu")
    _case(*size, t, "relu", odd=True)


@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("size", [(128, 140, 128, 8), (131, 600, 32, 1)])
def test_many_images_with_an_8_bit_checkpoint(size, t):
    _case(*size, t, "silu", kept=True)
    _case(*size, t, "none", kept=True, odd=True, params=False)


@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_many_images_held(t):
    _case(150, 60, 64, 8, t, "silu")                       # values in registers, gradients of 150 images summed
    _case(150, 60, 64, 8, t, "relu", kept=True)


@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("size", [(2, 40, 1800, 3), (1, 700, 2100, 5), (2, 33, 1290, 2)])
def test_wide_groups(size, t):
    """Channels of magnitudes of their own, so that one taken for another shows."""
    _case(*size, t, "silu", offset=3.0)
    _case(*size, t, "relu", odd=True, offset=3.0)


def test_wide_groups_with_an_8_bit_checkpoint():
    _case(2, 40, 1824, 3, "bf16", "silu", kept=True)
    _case(1, 300, 2080, 4, "f32", "gelu", kept=True, odd=True)


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("size", [(1, 9000, 130, 1), (2, 4000, 192, 2), (3, 2500, 400, 50)])
def test_many_blocks_of_pixels(size, t):
    """Sums joined by channels, and by groups, before the results."""
    _case(*size, t, "silu")
