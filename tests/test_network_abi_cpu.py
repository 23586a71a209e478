"""Argument checks and size queries of the network-head calls (gs_rms_norm_*,
gs_mxfp8_quantize, gs_linear_*, gs_orthogonalize, gs_muon_step): decided on
the host, nothing is launched."""

import ctypes as C
import os
import shutil
import subprocess
import tempfile

import pytest
import torch

from gaussian_splatting_tile_amd import binding as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PTR = 0x10000        # never dereferenced


def test_struct_layouts_match_header():
    pairs = [("gs_rms_norm", B.GsRmsNorm), ("gs_rms_norm_grads", B.GsRmsNormGrads), ("gs_linear", B.GsLinear),
             ("gs_linear_grads", B.GsLinearGrads), ("gs_muon", B.GsMuon)]
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "gs.h"', "int main(void) {"]
    expect = []
    for cname, cls in pairs:
        lines.append(f'printf("%zu\\n", sizeof({cname}));')
        expect.append(C.sizeof(cls))
        for fname, _ in cls._fields_:
            lines.append(f'printf("%zu\\n", offsetof({cname}, {fname}));')
            expect.append(getattr(cls, fname).offset)
    lines.append("return 0; }")
    with tempfile.TemporaryDirectory() as d:
        src, exe = os.path.join(d, "layout.c"), os.path.join(d, "layout")
        open(src, "w").write("\n".join(lines) + "\n")
        subprocess.run([shutil.which("gcc") or "cc", "-I", os.path.join(ROOT, "include"), src, "-o", exe], check=True)
        got = [int(x) for x in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    assert got == expect


def _norm(**kw):
    a = B.GsRmsNorm(m=10, n=64, dtype=B.GS_DTYPE_BF16, y_dtype=B.GS_DTYPE_BF16, eps=1e-6, x=PTR, x_stride=64,
                    residual=PTR, residual_stride=64, gamma=PTR, sum=PTR, sum_stride=64, y=PTR, y_stride=64,
                    y_scales=PTR, y_scales_stride=2, rstd=PTR)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def test_norm_argument_errors():
    L = B.lib()
    assert L.gs_rms_norm_fwd(None, None) == B.GS_ERR_INVALID_ARG
    bad = [dict(m=-1), dict(m=(1 << 30) + 1), dict(n=0), dict(n=(1 << 20) + 1), dict(dtype=3), dict(dtype=-1), dict(eps=-1.0),
           dict(eps=float("nan")), dict(eps=float("inf")), dict(x=None), dict(y=None), dict(x_stride=63),
           dict(y_stride=63), dict(residual_stride=63), dict(sum_stride=1), dict(x=PTR + 1), dict(y=PTR + 1),
           dict(sum=PTR + 1), dict(gamma=PTR + 2), dict(rstd=PTR + 2),
           dict(y_dtype=3, n=40, y_stride=40), dict(y_dtype=3, y_scales=None), dict(y_dtype=3, y_scales_stride=1)]
    for kw in bad:
        assert L.gs_rms_norm_fwd(C.byref(_norm(**kw)), None) == B.GS_ERR_INVALID_ARG, kw
    assert L.gs_rms_norm_fwd(C.byref(_norm(y_dtype=B.GS_DTYPE_F32)), None) == B.GS_ERR_UNSUPPORTED
    assert L.gs_rms_norm_fwd(C.byref(_norm(m=0, x=None, y=None)), None) == B.GS_OK
    assert L.gs_mxfp8_quantize(PTR, 0, 10, 33, 64, PTR, 64, PTR, 2, None) == B.GS_ERR_INVALID_ARG
    assert L.gs_mxfp8_quantize(PTR, 3, 10, 32, 64, PTR, 64, PTR, 2, None) == B.GS_ERR_INVALID_ARG
    assert L.gs_mxfp8_quantize(None, 0, 0, 32, 64, None, 64, None, 2, None) == B.GS_OK


def _norm_grads(**kw):
    a = B.GsRmsNormGrads(m=10, n=64, dtype=B.GS_DTYPE_F16, sum=PTR, sum_stride=64, rstd=PTR, gamma=PTR, dy=PTR,
                         dy_stride=64, dsum=PTR, dsum_stride=64, dx=PTR, dx_stride=64, dgamma=PTR)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def test_norm_gradient_argument_errors():
    L = B.lib()
    need = L.gs_rms_norm_bwd_workspace_bytes(10, 64)
    assert need > 0 and L.gs_rms_norm_bwd_workspace_bytes(0, 64) == 0 and L.gs_rms_norm_bwd_workspace_bytes(10, 0) == 0
    assert L.gs_rms_norm_bwd(None, PTR, need, None) == B.GS_ERR_INVALID_ARG
    bad = [dict(m=-1), dict(n=0), dict(dtype=3), dict(sum=None), dict(rstd=None), dict(dy=None), dict(dx=None),
           dict(sum_stride=63), dict(dy_stride=63), dict(dsum_stride=63), dict(dx_stride=63), dict(dx=PTR + 1),
           dict(dgamma=PTR + 1)]
    for kw in bad:
        assert L.gs_rms_norm_bwd(C.byref(_norm_grads(**kw)), PTR, need, None) == B.GS_ERR_INVALID_ARG, kw
    assert L.gs_rms_norm_bwd(C.byref(_norm_grads()), PTR, need - 1, None) == B.GS_ERR_WORKSPACE
    assert L.gs_rms_norm_bwd(C.byref(_norm_grads()), None, need, None) == B.GS_ERR_INVALID_ARG
    assert L.gs_rms_norm_bwd(C.byref(_norm_grads()), PTR + 8, need, None) == B.GS_ERR_INVALID_ARG
    assert L.gs_rms_norm_bwd(C.byref(_norm_grads(m=0, dgamma=None)), None, 0, None) == B.GS_OK


def _linear(**kw):
    a = B.GsLinear(m=100, n=64, k=96, dtype=B.GS_DTYPE_BF16, y_dtype=B.GS_DTYPE_BF16, x=PTR, x_stride=96, w=PTR,
                   w_stride=96, x_scales=PTR, x_scales_stride=3, w_scales=PTR, w_scales_stride=3, bias=PTR,
                   residual=PTR, residual_stride=64, y=PTR, y_stride=64, z=PTR, z_stride=64)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def test_linear_argument_errors():
    L = B.lib()
    assert L.gs_linear_fwd(None, None, 0, None) == B.GS_ERR_INVALID_ARG
    mx = dict(dtype=B.GS_DTYPE_MXFP8, z=None)
    bad = [dict(m=-1), dict(n=0), dict(k=0), dict(n=(1 << 20) + 1), dict(dtype=4), dict(dtype=-1), dict(y_dtype=7), dict(activation=-1),
           dict(activation=4), dict(x=None), dict(w=None), dict(y=None), dict(x_stride=95), dict(w_stride=95),
           dict(y_stride=63), dict(residual_stride=63), dict(z_stride=63), dict(x=PTR + 1), dict(w=PTR + 1),
           dict(y=PTR + 1), dict(z=PTR + 1), dict(bias=PTR + 2), dict(residual=PTR + 1), dict(planes=1),
           dict(mx, x_scales=None), dict(mx, w_scales=None), dict(mx, x_scales_stride=2), dict(mx, w_scales_stride=2)]
    for kw in bad:
        assert L.gs_linear_fwd(C.byref(_linear(**kw)), None, 0, None) == B.GS_ERR_INVALID_ARG, kw
        assert L.gs_linear_fwd_workspace_bytes(C.byref(_linear(**kw))) == 0
    for kw in (dict(y_dtype=B.GS_DTYPE_MXFP8), dict(dtype=B.GS_DTYPE_MXFP8), dict(mx, k=90)):
        assert L.gs_linear_fwd(C.byref(_linear(**kw)), None, 0, None) == B.GS_ERR_UNSUPPORTED, kw
    assert L.gs_linear_fwd(C.byref(_linear(m=0, x=None, w=None, y=None)), None, 0, None) == B.GS_OK
    # a long contraction over few outputs is split and needs room
    deep = dict(m=64, k=1 << 16, x_stride=1 << 16, w_stride=1 << 16)
    need = L.gs_linear_fwd_workspace_bytes(C.byref(_linear(**deep)))
    assert need > 0
    assert L.gs_linear_fwd(C.byref(_linear(**deep)), PTR, need - 1, None) == B.GS_ERR_WORKSPACE
    assert L.gs_linear_fwd(C.byref(_linear(**deep)), None, need, None) == B.GS_ERR_INVALID_ARG
    assert L.gs_linear_fwd(C.byref(_linear(**deep)), PTR + 4, need, None) == B.GS_ERR_INVALID_ARG


def _grads(**kw):
    g = B.GsLinearGrads(dy=PTR, dy_stride=64, dx=PTR, dx_stride=96, dw=PTR, dw_stride=96, dw_dtype=B.GS_DTYPE_F32, db=PTR)
    for k, v in kw.items():
        setattr(g, k, v)
    return g


def test_linear_gradient_argument_errors():
    L = B.lib()
    lin = _linear(activation=B.GS_ACT["gelu"])
    need = L.gs_linear_bwd_workspace_bytes(C.byref(lin), C.byref(_grads()))
    assert need > 0
    assert L.gs_linear_bwd(C.byref(lin), None, PTR, need, None) == B.GS_ERR_INVALID_ARG
    assert L.gs_linear_bwd(None, C.byref(_grads()), PTR, need, None) == B.GS_ERR_INVALID_ARG
    bad = [dict(dy=None), dict(dy_stride=63), dict(dy=PTR + 1), dict(dx_stride=95), dict(dx=PTR + 1), dict(dw_stride=95),
           dict(dw=PTR + 2), dict(dw_dtype=B.GS_DTYPE_F16), dict(db=PTR + 2)]
    for kw in bad:
        assert L.gs_linear_bwd(C.byref(lin), C.byref(_grads(**kw)), PTR, need, None) == B.GS_ERR_INVALID_ARG, kw
    assert L.gs_linear_bwd(C.byref(_linear(activation=3, z=None)), C.byref(_grads()), PTR, need, None) == B.GS_ERR_INVALID_ARG
    assert L.gs_linear_bwd(C.byref(_linear(dtype=B.GS_DTYPE_MXFP8, z=None)), C.byref(_grads()), PTR, need, None) == B.GS_ERR_UNSUPPORTED
    assert L.gs_linear_bwd(C.byref(lin), C.byref(_grads()), PTR, need - 1, None) == B.GS_ERR_WORKSPACE
    assert L.gs_linear_bwd(C.byref(lin), C.byref(_grads()), None, need, None) == B.GS_ERR_INVALID_ARG
    empty = _linear(m=0)
    assert L.gs_linear_bwd(C.byref(empty), C.byref(_grads(dw=None, db=None)), None, 0, None) == B.GS_OK


def _muon(**kw):
    a = B.GsMuon(batch=2, rows=64, cols=48, grad_dtype=B.GS_DTYPE_F32, out_dtype=B.GS_DTYPE_F32, steps=5, a=3.4445, b=-4.775,
                 c=2.0315, eps=1e-7, lr=0.02, beta=0.95, scale=1.0, nesterov=1, grad=PTR, out=PTR, momentum=PTR,
                 momentum_out=PTR, weight=PTR, weight_out=PTR)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def test_muon_argument_errors():
    L = B.lib()
    need = L.gs_muon_workspace_bytes(C.byref(_muon()))
    assert need > 0 and L.gs_muon_workspace_bytes(C.byref(_muon(batch=0))) == 0
    nan, inf = float("nan"), float("inf")
    both = [dict(batch=-1), dict(batch=65536), dict(rows=0), dict(cols=0), dict(rows=16385), dict(grad_dtype=3), dict(out_dtype=3),
            dict(steps=0), dict(steps=65), dict(a=nan), dict(b=inf), dict(c=nan), dict(eps=0.0), dict(eps=nan), dict(grad=None),
            dict(grad=PTR + 2)]
    for kw in both + [dict(out=None), dict(out=PTR + 1)]:
        assert L.gs_orthogonalize(C.byref(_muon(**kw)), PTR, need, None) == B.GS_ERR_INVALID_ARG, kw
    for kw in both + [dict(momentum=None), dict(momentum_out=None), dict(weight=None), dict(weight_out=None), dict(momentum=PTR + 2),
                      dict(weight_out=PTR + 1), dict(lr=nan), dict(beta=inf), dict(weight_decay=nan), dict(scale=inf)]:
        assert L.gs_muon_step(C.byref(_muon(**kw)), PTR, need, None) == B.GS_ERR_INVALID_ARG, kw
    for f in (L.gs_orthogonalize, L.gs_muon_step):
        assert f(None, PTR, need, None) == B.GS_ERR_INVALID_ARG
        assert f(C.byref(_muon()), PTR, need - 1, None) == B.GS_ERR_WORKSPACE
        assert f(C.byref(_muon()), None, need, None) == B.GS_ERR_INVALID_ARG
        assert f(C.byref(_muon()), PTR + 4, need, None) == B.GS_ERR_INVALID_ARG
        assert f(C.byref(_muon(batch=0, grad=None)), None, 0, None) == B.GS_OK


def test_binding_refuses_tensors_that_do_not_fit():
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(8, 64, dtype=torch.bfloat16)
    y = torch.zeros(4, 8, dtype=torch.bfloat16)
    B.linear_struct(x, w, y)
    for kw in (dict(y=torch.zeros(8, 4, dtype=torch.bfloat16)), dict(w=w[:, :32]), dict(w=w.float()), dict(x=x.double()),
               dict(bias=torch.zeros(7)), dict(bias=torch.zeros(8, dtype=torch.float16)), dict(residual=y.float()),
               dict(y=torch.zeros(8, 4, dtype=torch.bfloat16).t()), dict(z=y.float()), dict(x=x[:1].expand(4, 64)),
               dict(y=y.to("meta"))):
        with pytest.raises(ValueError):
            B.linear_struct(**{**dict(x=x, w=w, y=y), **kw})
    with pytest.raises(KeyError):
        B.linear_struct(x, w, y, act="tanh")
    with pytest.raises(ValueError):
        B.rms_norm_fwd(x, torch.zeros(4, 64))
    with pytest.raises(ValueError):
        B.mxfp8_quantize(x, torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8))
    with pytest.raises(ValueError):
        B.muon_struct(x, momentum=torch.zeros(4, 64, dtype=torch.bfloat16), weight=x)
    with pytest.raises(ValueError):
        B.muon_struct(x, out=x[:2])
    lin = B.linear_struct(x, w, y)
    with pytest.raises(ValueError):
        B.linear_grads_struct(lin, y, dw=torch.zeros(8, 64, dtype=torch.float16))


def test_gradients_leave_the_forward_descriptor_as_it_is():
    """A y of one type and a dy of another in one descriptor would have the
    next forward write dy's type into y."""
    x, w = torch.zeros(40, 64, dtype=torch.bfloat16), torch.zeros(8, 64, dtype=torch.bfloat16)
    dy, dw = torch.zeros(40, 8, dtype=torch.bfloat16), torch.zeros(8, 64)
    lin = B.linear_struct(x, w, dy.clone())
    with pytest.raises(ValueError):
        B.linear_grads_struct(lin, dy.float(), dw=dw)
    assert lin.y_dtype == B.GS_DTYPE_BF16
    B.linear_grads_struct(lin, dy, dw=dw)
    assert lin.y_dtype == B.GS_DTYPE_BF16


def test_a_descriptor_without_y_takes_gradients_of_any_type():
    """Each of them is used with its own type, whichever was made last: an
    fp32 dy of bf16 operands has to be converted first, a bf16 one is read as
    it is."""
    x, w = torch.zeros(40, 64, dtype=torch.bfloat16), torch.zeros(8, 64, dtype=torch.bfloat16)
    dy, dw = torch.zeros(40, 8, dtype=torch.bfloat16), torch.zeros(8, 64)
    size = lambda d: (lambda a: B.linear_bwd_workspace_bytes(a, B.linear_grads_struct(a, d, dw=dw)))(B.linear_struct(x, w, None))
    assert size(dy) != size(dy.float())
    lin = B.linear_struct(x, w, None)
    kept = [B.linear_grads_struct(lin, d, dw=dw) for d in (dy, dy.float(), dy)]
    assert [B.linear_bwd_workspace_bytes(lin, g) for g in kept] == [size(dy), size(dy.float()), size(dy)]


def test_muon_results_have_one_type():
    """One type describes out and weight: of two the other would be written in
    elements of the wrong size."""
    g = torch.zeros(4, 64)
    for out, weight in ((torch.bfloat16, torch.float32), (torch.float32, torch.float16)):
        with pytest.raises(ValueError):
            B.muon_struct(g, out=g.to(out), momentum=g, weight=g.to(weight))
    with pytest.raises(ValueError):
        B.muon_struct(g, out=g.half(), momentum=g, weight_out=g)
    a = B.muon_struct(g, out=g.half(), momentum=g, weight=g.half())
    assert a.out_dtype == B.GS_DTYPE_F16 and B.muon_struct(g, out=g.bfloat16()).out_dtype == B.GS_DTYPE_BF16


def test_calls_refuse_memory_that_the_gpu_must_not_touch(monkeypatch):
    """Tensors of the host or of another GPU than the current one, and
    workspaces that are not so many bytes of that GPU's memory."""
    x, w, v = torch.zeros(4, 64), torch.zeros(8, 64), torch.zeros(4)
    codes, scales = torch.zeros(4, 64, dtype=torch.float8_e4m3fn), torch.zeros(4, 2, dtype=torch.uint8)
    lin = B.linear_struct(x, w, torch.zeros(4, 8))
    gr = B.linear_grads_struct(lin, torch.zeros(4, 8), dx=torch.zeros(4, 64))
    mu = B.muon_struct(x, out=x, momentum=x, weight=x)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    calls = [lambda: B.rms_norm_fwd(x, x), lambda: B.rms_norm_bwd(x, v, x, x), lambda: B.mxfp8_quantize(x, codes, scales),
             lambda: B.linear_fwd(lin, ws), lambda: B.linear_bwd(lin, gr, ws), lambda: B.orthogonalize(mu, ws),
             lambda: B.muon_step(mu, ws)]
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    for call in calls:
        with pytest.raises(ValueError):
            call()
    gpu, ok = torch.device("cuda", 0), ws.to("meta")
    for device, workspace, stream in ((torch.device("cuda", 1), None, None), (gpu, ws, None), (gpu, ws[::2], None)):
        with pytest.raises(ValueError):
            B._stream_for(device, workspace, stream)

    class Side:
        device, cuda_stream = gpu, 64

    class Shared(torch.Tensor):                     # a workspace's properties, without one
        def get_device(self):
            return 0

    whole = torch.zeros(16, dtype=torch.uint8).as_subclass(Shared)
    assert B._stream_for(gpu, whole, Side).value == 64 and B._stream_for(None, ok, Side).value == 64
    Side.device = torch.device("cuda", 1)
    with pytest.raises(ValueError):
        B._stream_for(gpu, whole, Side)
    Side.device = gpu
    for bad in (whole[::2], whole[:1].expand(16)):
        with pytest.raises(ValueError):
            B._stream_for(gpu, bad, Side)
    with pytest.raises(ValueError):
        B.linear_grads_struct(lin, torch.zeros(4, 8, device="meta"))


def test_sizes_that_the_descriptors_cannot_hold():
    """A size of 2^32 + 64 in a 32-bit field would read as 64."""
    big = (1 << 32) + 64
    e = lambda *s, t=torch.bfloat16: torch.empty(s, dtype=t, device="meta")
    too_large = lambda: pytest.raises(ValueError, match="32 bits")
    with too_large():
        B.linear_struct(e(1, big), e(8, big), e(1, 8))
    with too_large():
        B.linear_struct(e(1, 8), e(big, 8), e(1, big))
    with too_large():
        B.rms_norm_fwd(e(1, big), e(1, big))
    with too_large():
        B.rms_norm_bwd(e(1, big), e(1, t=torch.float32), e(1, big), e(1, big))
    with too_large():
        B.rms_norm_bwd_workspace_bytes(1, big)
    with too_large():
        B.mxfp8_quantize(e(1, big), e(1, big, t=torch.float8_e4m3fn), e(1, big // 32, t=torch.uint8))
    for shape in ((big, 8), (8, big), (big, 1, 8)):
        with too_large():
            B.muon_struct(e(*shape), out=e(*shape))
