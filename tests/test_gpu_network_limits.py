"""Network-head calls at the far end of the sizes that include/gs.h names:
more blocks than one dimension of a launch takes, and arrays whose elements lie
past 32-bit offsets on every way of the products.  Values are chosen so that
the results are exact, or are compared with fp64 at the far end."""

import numpy as np
import pytest
import torch

from gaussian_splatting_tile_amd import binding as B
from oracle import network as N
from tests.gpu_util import say

pytestmark = pytest.mark.gpu


def _ws(n):
    return torch.empty(max(int(n), 16), dtype=torch.uint8, device="cuda")


def _call(f):
    """f(); a refusal is reported without its arguments, gigabytes each."""
    try:
        f()
    except B.GsError as e:
        pytest.fail(str(e), pytrace=False)


def _all(t):
    return bool(t.all())


@pytest.fixture(autouse=True)
def _release():
    yield
    torch.cuda.empty_cache()


def test_norm_of_more_rows_than_a_launch_has_threads():
    """2^28 rows by 16 lanes each are 2^32 threads.  Rows of one magnitude norm
    to their signs."""
    m, n = (1 << 28) + 3, 8
    say(f"[gpu] norm {m}x{n}")
    x = torch.full((m, n), 2.0, dtype=torch.bfloat16, device="cuda")
    x[1::2] = -0.5
    rstd = torch.zeros(m, device="cuda")
    _call(lambda: B.rms_norm_fwd(x, x, rstd=rstd, eps=0.0))
    ok = _all(x[::2] == 1.0), _all(x[1::2] == -1.0), _all(rstd[::2] == 0.5), _all(rstd[1::2] == 2.0)
    assert all(ok), ok


def test_quantise_of_more_rows_than_a_launch_has_threads():
    m = (1 << 28) + 3
    say(f"[gpu] quantise {m}x32")
    x = torch.full((m, 32), 2.0, dtype=torch.bfloat16, device="cuda")
    x[1::2] = 1.0
    codes, scales = torch.zeros(m, 32, dtype=torch.float8_e4m3fn, device="cuda"), torch.zeros(m, 1, dtype=torch.uint8, device="cuda")
    _call(lambda: B.mxfp8_quantize(x, codes, scales))
    # 256 = 2 x 2^7 = 1 x 2^8
    ok = _all(codes.view(torch.uint8) == 0x78), _all(scales[::2] == 127 - 7), _all(scales[1::2] == 127 - 8)
    assert all(ok), ok
