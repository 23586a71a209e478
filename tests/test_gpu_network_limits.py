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


@pytest.mark.parametrize("planes", [False, True])
@pytest.mark.parametrize("t", [torch.bfloat16, torch.float32])
def test_linear_of_more_tiles_than_a_launch_takes(t, planes):
    """2^30 rows in tiles of 64 by 256 threads or of 128 by 512 are 2^32
    threads.  Small whole numbers, so every result is exact."""
    m = 1 << 30
    say(f"[gpu] linear {m} x 1 x 1 {t} planes={planes}")
    x = torch.arange(m, dtype=torch.int32, device="cuda").remainder_(63).to(t).view(m, 1)
    xs = x.view(1, m) if planes else x
    w, b, y, z = torch.full((1, 1), 2.0, dtype=t, device="cuda"), torch.ones(1, device="cuda"), torch.zeros_like(xs), torch.zeros_like(x)
    lin = B.linear_struct(x, w, y, bias=b, residual=xs, z=z, planes=planes)
    _call(lambda: B.linear_fwd(lin, _ws(B.linear_fwd_workspace_bytes(lin))))
    z -= 1
    y -= 1
    ok = _all(z == 2 * x), _all(y == 3 * xs)
    assert all(ok), ok
    lin = B.linear_struct(x, w, None, planes=planes)
    gr = B.linear_grads_struct(lin, xs, dx=z)
    z.zero_()
    _call(lambda: B.linear_bwd(lin, gr, _ws(B.linear_bwd_workspace_bytes(lin, gr))))
    ok = _all(z == 2 * x)
    assert ok, "dx"


def test_linear_backward_of_no_rows_into_a_large_dw():
    n = 1 << 16
    say(f"[gpu] dw of {n} x {n} over no rows")
    x, dy = torch.zeros(0, n, dtype=torch.bfloat16, device="cuda"), torch.zeros(0, n, dtype=torch.bfloat16, device="cuda")
    dw = torch.ones(n, n, dtype=torch.bfloat16, device="cuda")
    lin = B.linear_struct(x, dw, None)
    gr = B.linear_grads_struct(lin, dy, dw=dw)
    _call(lambda: B.linear_bwd(lin, gr))
    ok = not bool(dw.any())
    assert ok, "dw"
