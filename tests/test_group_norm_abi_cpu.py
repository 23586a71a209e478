"""Argument checks and size queries of group norm (gs_group_norm_*): decided on
the host, nothing is launched."""

import ctypes as C

import pytest
import torch

from gaussian_splatting_tile_amd import binding as B
from tests.test_attention_abi_cpu import PTR, layouts_match


def test_struct_layouts_match_header():
    layouts_match([("gs_group_norm", B.GsGroupNorm), ("gs_group_norm_grads", B.GsGroupNormGrads)])


def _map(name, c=64, p=5000):
    return {name: PTR, f"{name}_image": p * c, f"{name}_pixel": c}


def _norm(**kw):
    a = dict(n=2, c=64, groups=8, dtype=B.GS_DTYPE_BF16, activation=2, eps=1e-5, p=5000, **_map("x"), gamma=PTR, beta=PTR, **_map("y"), mean=PTR, rstd=PTR,
             **_map("kept"), **_map("kept_scales", 2))
    a.update(kw)
    return B.GsGroupNorm(**a)


def _grads(**kw):
    a = dict(n=2, c=64, groups=8, dtype=B.GS_DTYPE_BF16, x_dtype=B.GS_DTYPE_MXFP8, activation=2, p=5000, **_map("x"), **_map("x_scales", 2), mean=PTR, rstd=PTR,
             gamma=PTR, beta=PTR, **_map("dy"), **_map("dx"), dgamma=PTR, dbeta=PTR)
    a.update(kw)
    return B.GsGroupNormGrads(**a)


SHAPES = [dict(n=-1), dict(n=65536), dict(p=-1), dict(p=(1 << 30) + 1), dict(c=0), dict(c=65544), dict(groups=0), dict(groups=7), dict(groups=128), dict(dtype=3),
          dict(dtype=-1), dict(activation=-1), dict(activation=4), dict(x=None), dict(x_pixel=-1), dict(x_image=-1), dict(gamma=PTR + 2), dict(beta=PTR + 2),
          dict(mean=PTR + 2), dict(rstd=PTR + 2)]


def test_argument_errors():
    L = B.lib()
    need = L.gs_group_norm_fwd_workspace_bytes(2, 5000, 64, 8)
    assert need > 0 and L.gs_group_norm_fwd_workspace_bytes(2, 5000, 64, 7) == L.gs_group_norm_fwd_workspace_bytes(0, 5000, 64, 8) == 0
    assert L.gs_group_norm_fwd(None, PTR, need, None) == B.GS_ERR_INVALID_ARG
    bad = SHAPES + [dict(x=PTR + 1), dict(y=None), dict(y=PTR + 1), dict(y_pixel=63), dict(y_pixel=0), dict(y_image=5000 * 64 - 1), dict(y_image=0), dict(y_image=-1),
                    dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(kept=None), dict(kept_scales=None), dict(c=48), dict(kept_pixel=63),
                    dict(kept_image=0), dict(kept_scales_pixel=1), dict(kept_scales_image=-1)]
    for kw in bad:
        assert L.gs_group_norm_fwd(C.byref(_norm(**kw)), PTR, 1 << 40, None) == B.GS_ERR_INVALID_ARG, kw
    assert L.gs_group_norm_fwd(C.byref(_norm()), PTR, need - 1, None) == B.GS_ERR_WORKSPACE
    assert L.gs_group_norm_fwd(C.byref(_norm()), None, need, None) == B.GS_ERR_INVALID_ARG
    assert L.gs_group_norm_fwd(C.byref(_norm()), PTR + 8, need, None) == B.GS_ERR_INVALID_ARG
    for kw in (dict(n=0, x=None, y=None), dict(p=0, x=None, y=None)):
        assert L.gs_group_norm_fwd(C.byref(_norm(**kw)), None, 0, None) == B.GS_OK, kw


def test_gradient_argument_errors():
    L = B.lib()
    need = L.gs_group_norm_bwd_workspace_bytes(2, 5000, 64, 8)
    assert need > 0 and L.gs_group_norm_bwd_workspace_bytes(2, 0, 64, 8) == L.gs_group_norm_bwd_workspace_bytes(1, 10, 64, 8) == 0
    assert L.gs_group_norm_bwd_workspace_bytes(2, 10, 64, 8) > 0            # sums of two images
    assert L.gs_group_norm_bwd(None, PTR, need, None) == B.GS_ERR_INVALID_ARG
    bad = SHAPES + [dict(x_dtype=4), dict(x_dtype=-1), dict(x_scales=None), dict(x_scales_pixel=-1), dict(c=48), dict(dy=None), dict(dy=PTR + 1), dict(dy_pixel=-1),
                    dict(dx=None), dict(dx=PTR + 1), dict(dx_pixel=63), dict(dx_image=0), dict(mean=None), dict(rstd=None), dict(dgamma=PTR + 2),
                    dict(dbeta=PTR + 2)]
    for kw in bad:
        assert L.gs_group_norm_bwd(C.byref(_grads(**kw)), PTR, 1 << 40, None) == B.GS_ERR_INVALID_ARG, kw
    assert L.gs_group_norm_bwd(C.byref(_grads(x_dtype=B.GS_DTYPE_BF16, x=PTR + 1)), PTR, need, None) == B.GS_ERR_INVALID_ARG
    assert L.gs_group_norm_bwd(C.byref(_grads(x_dtype=B.GS_DTYPE_F32)), PTR, need, None) == B.GS_ERR_UNSUPPORTED
    assert L.gs_group_norm_bwd(C.byref(_grads()), PTR, need - 1, None) == B.GS_ERR_WORKSPACE
    assert L.gs_group_norm_bwd(C.byref(_grads()), None, need, None) == B.GS_ERR_INVALID_ARG
    assert L.gs_group_norm_bwd(C.byref(_grads()), PTR + 8, need, None) == B.GS_ERR_INVALID_ARG
    assert L.gs_group_norm_bwd(C.byref(_grads(n=0, x=None, dy=None, dx=None, dgamma=None, dbeta=None)), None, 0, None) == B.GS_OK


def test_binding_refuses_tensors_that_do_not_fit(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    x, st, v = torch.zeros(2, 9, 64), torch.zeros(2, 8), torch.zeros(64)
    codes, scales = torch.zeros(2, 9, 64, dtype=torch.float8_e4m3fn), torch.zeros(2, 9, 2, dtype=torch.uint8)
    turned = torch.zeros(2, 64, 9).transpose(1, 2)
    bad = [dict(x=x[0]), dict(x=x.double()), dict(x=turned), dict(y=x[:, :8]), dict(y=x.half()), dict(y=turned), dict(y=x.to("meta")), dict(gamma=v[:63]),
           dict(gamma=v.half()), dict(beta=v.to("meta")), dict(mean=st[:1]), dict(rstd=st.double()), dict(kept=scales, kept_scales=scales),
           dict(kept=codes, kept_scales=scales[..., :1]), dict(kept=codes, kept_scales=scales.float()), dict(groups=1 << 32)]
    for kw in bad:
        with pytest.raises((ValueError, B.GsError)):
            B.group_norm_fwd(**{**dict(x=x, y=x, groups=8), **kw})
    ok = dict(x=x, mean=st, rstd=st, dy=x, dx=x, groups=8)
    bad = [dict(x=x.half()), dict(x=codes), dict(x_scales=scales), dict(x=codes, x_scales=scales[:, :8]), dict(dy=x[0]), dict(dy=x.half()), dict(dx=x.half()),
           dict(dx=x[:1]), dict(mean=st[:, :7]), dict(rstd=st.to("meta")), dict(dgamma=v[:3]), dict(dbeta=v.half())]
    for kw in bad:
        with pytest.raises(ValueError):
            B.group_norm_bwd(**{**ok, **kw})
    for call in (lambda: B.group_norm_fwd(x, x, 8), lambda: B.group_norm_bwd(**ok)):       # the host's memory
        with pytest.raises(ValueError, match="current GPU"):
            call()
    big = torch.empty(1, 1, (1 << 32) + 64, device="meta")
    with pytest.raises(ValueError, match="32 bits"):
        B.group_norm_fwd(big, big, 8)
