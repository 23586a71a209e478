"""Group norm's statistics where a few pixels are unlike the others, as a
border, padding or dead pixels are, and where channels of a group lie far apart.

Tolerances.  e = 2^-24; x is fp32, D the largest difference of two of a
channel's values and sd the group's spread.  Values are taken as differences d from
one of a channel's values or a mean of some, so |d| <= D, each rounded by e D.
A sum of r terms one after the other is off by r / 2 e D at most of the mean
of its terms.  Up to eight values of a thread here (4.4 with the first addition),
threads four at a time (7), blocks of pixels eight at a time (5), rows of those (10)
and the reciprocals (1.6): a mean is off by 28 e D at most.
* variance: squares of differences of such means, every one a part of the spread,
  so 2 x 28 e D / sd of itself (what the mean in the middle is off by counts squared); sums
  of squares themselves 12 e for a thread's and less than 20 e for what joins them.
* rstd is off by half of what the variance is, and the mean by 28 e D and its own
  rounding.
"""

import numpy as np
import pytest
import torch

from gaussian_splatting_tile_amd import binding as B
from oracle import attention as A
from tests.test_gpu_attention import E, _close, _ws

pytestmark = pytest.mark.gpu


def _statistics(x, groups):
    n, p, c = x.shape
    y, mean, rstd = torch.empty_like(x), torch.empty(n, groups, device="cuda"), torch.empty(n, groups, device="cuda")
    B.group_norm_fwd(x, y, groups, mean=mean, rstd=rstd, workspace=_ws(B.group_norm_fwd_workspace_bytes(n, p, c, groups))[0])
    return y, mean, rstd


# one workgroup's (values held; read again), sums joined by the workgroups that write, by channels first, by groups
SHAPES = [(1, 64, 32, 8), (128, 1024, 24, 3), (2, 2048, 24, 3), (1, 65536, 16, 2), (2, 65536, 128, 32)]


@pytest.mark.parametrize("n,p,c,groups", SHAPES)
@pytest.mark.parametrize("kind", ["left column", "eight pixels", "first row", "one pixel", "none"])
def test_variance_of_maps_with_unlike_pixels(n, p, c, groups, kind):
    """4096 +- 1, and 0 in some pixels: maps of 8 rows or a multiple have an eighth of
    their pixels apart, in a column, the places that a sample spread evenly would take."""
    gen = torch.Generator("cuda").manual_seed(p + c)
    x = 4096.0 + torch.randn(n, p, c, generator=gen, device="cuda")
    rows = 8 if p < 65536 else 64
    if kind == "left column":
        x.view(n, rows, p // rows, c)[:, :, 0] = 0.0
    elif kind == "eight pixels":
        x[:, ::p // 8] = 0.0
    elif kind == "first row":
        x.view(n, rows, p // rows, c)[:, 0] = 0.0
    elif kind == "one pixel":
        x[:, 0] = 0.0
    y, mean, rstd = _statistics(x, groups)
    v = x.double().view(n, p, groups, c // groups)
    m64 = v.mean((1, 3))
    var = (v - m64[:, None, :, None]).square().mean((1, 3))
    far = (x.amax(1) - x.amin(1)).double().view(n, groups, -1).amax(2)
    r64 = 1 / (var + 1e-5).sqrt()
    tol = (32 + 56 * far / var.sqrt()) * E / 2 * r64
    host = lambda t: t.double().cpu().numpy()
    _close(host(rstd), host(r64), host(tol), "rstd")
    _close(host(mean), host(m64), host(28 * E * far + 2 * E * m64.abs()), "mean")


@pytest.mark.parametrize("n,p,c,groups", [(1, 64, 60, 4), (128, 1016, 24, 3), (2, 1000, 90, 6), (1, 9001, 24, 2), (2, 8008, 128, 32), (1, 200, 1800, 3)])
def test_mean_of_channels_that_lie_far_apart(n, p, c, groups):
    """Values on a grid of 2^-4 on which every channel's sums are exact (below 2^23
    steps of 2^-7, the grid of a mean of eight): what is left of the mean's error is the
    joining of the channels, and its own rounding, 2^-24 of itself."""
    rng = np.random.default_rng(p + c)
    x = rng.integers(-32, 33, (n, p, c)) / 16.0
    x += np.round(np.linspace(1000, -1000, c // groups))[np.arange(c) % (c // groups)] + 0.125
    x = torch.from_numpy(x).float().cuda()
    _, mean, rstd = _statistics(x, groups)
    m64, r64, _, _ = A.group_norm(x.double().cpu().numpy(), groups)
    _close(mean.double().cpu().numpy(), m64, 1.001 * E * np.abs(m64), "mean")
    _close(rstd.double().cpu().numpy(), r64, 16 * E * r64, "rstd")
