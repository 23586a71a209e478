"""Argument checks and size queries of cross attention (gs_attention_*):
decided on the host, nothing is launched."""

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


def layouts_match(pairs):
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


def test_struct_layouts_match_header():
    layouts_match([("gs_attention", B.GsAttention), ("gs_attention_grads", B.GsAttentionGrads)])


def _fields(name, rows, heads, d=64):
    return {name: PTR, f"{name}_batch": rows * heads * d, f"{name}_row": heads * d, f"{name}_head": d}


def _attention(**kw):
    a = dict(batch=2, heads=8, kv_heads=4, nq=100, nk=300, d=64, dtype=B.GS_DTYPE_BF16, scale=0.125, lse=PTR, kv_lengths=PTR, kv_mask=PTR,
             kv_mask_stride=300, **_fields("q", 100, 8), **_fields("k", 300, 4), **_fields("v", 300, 4), **_fields("out", 100, 8))
    a.update(kw)
    return B.GsAttention(**a)


def _grads(**kw):
    g = dict(**_fields("dout", 100, 8), **_fields("dq", 100, 8), **_fields("dk", 300, 4), **_fields("dv", 300, 4))
    g.update(kw)
    return B.GsAttentionGrads(**g)


BAD = [dict(batch=-1), dict(batch=65536), dict(heads=0), dict(heads=7), dict(kv_heads=0), dict(kv_heads=3), dict(nq=-1), dict(nk=-1), dict(nq=(1 << 30) + 1),
       dict(nk=(1 << 30) + 1), dict(d=0), dict(dtype=3), dict(dtype=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
       dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(q=PTR + 1), dict(k=PTR + 1), dict(v=PTR + 1), dict(out=PTR + 1), dict(q_row=-64),
       dict(k_batch=-1), dict(v_head=-1), dict(out_row=-1), dict(lse=PTR + 2), dict(kv_lengths=PTR + 2), dict(kv_mask_stride=-1)]


def test_attention_argument_errors():
    L = B.lib()
    assert L.gs_attention_fwd(None, None, 0, None) == B.GS_ERR_INVALID_ARG and L.gs_attention_fwd_workspace_bytes(None) == 0
    for kw in BAD:
        assert L.gs_attention_fwd(C.byref(_attention(**kw)), PTR, 1 << 40, None) == B.GS_ERR_INVALID_ARG, kw
        assert L.gs_attention_fwd_workspace_bytes(C.byref(_attention(**kw))) == 0, kw
    # elements of out that share a place
    for kw in (dict(out_row=0), dict(out_row=511), dict(out_head=63), dict(out_batch=100 * 512 - 1), dict(out_batch=0)):
        assert L.gs_attention_fwd(C.byref(_attention(**kw)), PTR, 1 << 40, None) == B.GS_ERR_INVALID_ARG, kw
    for kw in (dict(d=129), dict(nq=1 << 30, batch=1, heads=8, kv_heads=4, out_batch=1 << 60), dict(batch=65535, nk=1 << 29)):
        assert L.gs_attention_fwd(C.byref(_attention(**kw)), PTR, 1 << 40, None) == B.GS_ERR_UNSUPPORTED, kw
    for kw in (dict(batch=0, q=None, k=None, v=None, out=None), dict(nq=0, q=None, out=None)):
        assert L.gs_attention_fwd(C.byref(_attention(**kw)), None, 0, None) == B.GS_OK, kw
    # many states and few queries are split and need room
    long = dict(nq=1, nk=100000)
    need = L.gs_attention_fwd_workspace_bytes(C.byref(_attention(**long)))
    assert need > 0
    assert L.gs_attention_fwd(C.byref(_attention(**long)), PTR, need - 1, None) == B.GS_ERR_WORKSPACE
    assert L.gs_attention_fwd(C.byref(_attention(**long)), None, need, None) == B.GS_ERR_INVALID_ARG
    assert L.gs_attention_fwd(C.byref(_attention(**long)), PTR + 8, need, None) == B.GS_ERR_INVALID_ARG


def test_attention_gradient_argument_errors():
    L = B.lib()
    a = _attention()
    need = L.gs_attention_bwd_workspace_bytes(C.byref(a), C.byref(_grads()))
    assert need > 0
    assert L.gs_attention_bwd(C.byref(a), None, PTR, need, None) == B.GS_ERR_INVALID_ARG
    assert L.gs_attention_bwd(None, C.byref(_grads()), PTR, need, None) == B.GS_ERR_INVALID_ARG
    for kw in BAD + [dict(lse=None)]:
        assert L.gs_attention_bwd(C.byref(_attention(**kw)), C.byref(_grads()), PTR, 1 << 40, None) == B.GS_ERR_INVALID_ARG, kw
    bad = [dict(dout=None), dict(dout=PTR + 1), dict(dout_row=-1), dict(dq=PTR + 1), dict(dk=PTR + 1), dict(dv=PTR + 1), dict(dq_row=0), dict(dq_head=32),
           dict(dk_row=255), dict(dv_batch=0), dict(dk_head=-64)]
    for kw in bad:
        assert L.gs_attention_bwd(C.byref(a), C.byref(_grads(**kw)), PTR, 1 << 40, None) == B.GS_ERR_INVALID_ARG, kw
    assert L.gs_attention_bwd(C.byref(a), C.byref(_grads()), PTR, need - 1, None) == B.GS_ERR_WORKSPACE
    assert L.gs_attention_bwd(C.byref(a), C.byref(_grads()), None, need, None) == B.GS_ERR_INVALID_ARG
    assert L.gs_attention_bwd(C.byref(a), C.byref(_grads()), PTR + 8, need, None) == B.GS_ERR_INVALID_ARG
    assert L.gs_attention_bwd(C.byref(_attention(batch=0)), C.byref(_grads()), None, 0, None) == B.GS_OK


def _tensors(b=2, nq=5, nk=7, h=4, kv=2, d=16, t=torch.bfloat16):
    z = lambda *s: torch.zeros(s, dtype=t)
    return z(b, nq, h, d), z(b, nk, kv, d), z(b, nk, kv, d), z(b, nq, h, d)


def test_binding_refuses_tensors_that_do_not_fit():
    q, k, v, out = _tensors()
    a = B.attention_struct(q, k, v, out, lse=torch.zeros(2, 4, 5))
    assert (a.batch, a.heads, a.kv_heads, a.nq, a.nk, a.d) == (2, 4, 2, 5, 7, 16) and a.scale == 0.25
    f, ok = torch.zeros(2, 4, 5), torch.ones(2, 7, dtype=torch.uint8)
    bad = [dict(q=q[0]), dict(k=k[0]), dict(k=k[:1]), dict(v=v[:, :6]), dict(v=v[..., :8]), dict(out=out[:, :4]), dict(k=k.half()), dict(v=v.float()),
           dict(out=out.float()), dict(q=q.transpose(2, 3).contiguous().transpose(2, 3)), dict(q=q.double(), k=k.double(), v=v.double(), out=out.double()),
           dict(lse=f[:, :3]), dict(lse=f.double()), dict(lse=f.transpose(1, 2).contiguous().transpose(1, 2)), dict(lse=f.reshape(2, 20)),
           dict(kv_lengths=torch.ones(2)), dict(kv_lengths=torch.ones(3, dtype=torch.int32)), dict(kv_lengths=torch.ones(4, dtype=torch.int32)[::2]),
           dict(kv_lengths=torch.ones(2, dtype=torch.int32, device="meta")), dict(kv_mask=ok.float()), dict(kv_mask=ok[:, :6]), dict(kv_mask=ok[:1]),
           dict(kv_mask=torch.ones(2, 14, dtype=torch.uint8)[:, ::2]), dict(kv_mask=ok.to("meta")), dict(k=k.to("meta")), dict(out=out.to("meta"))]
    for kw in bad:
        with pytest.raises(ValueError):
            B.attention_struct(**{**dict(q=q, k=k, v=v, out=out), **kw})
    for kw in (dict(dout=out.float()), dict(dout=out[:, :4]), dict(dout=out, dq=out.float()), dict(dout=out, dk=out), dict(dout=out, dv=v[..., :8]),
               dict(dout=out.to("meta")), dict(dout=out, dq=out.to("meta"))):
        with pytest.raises(ValueError):
            B.attention_grads_struct(a, **kw)
    with pytest.raises(B.GsError):                      # heads that k's do not divide
        B.attention_fwd(_attention(heads=6, kv_heads=4), stream=type("S", (), {"cuda_stream": 0})())


def test_binding_refuses_memory_that_the_gpu_must_not_touch(monkeypatch):
    q, k, v, out = _tensors()
    a = B.attention_struct(q, k, v, out, lse=torch.zeros(2, 4, 5))
    g = B.attention_grads_struct(a, out, dq=out, dk=k, dv=v)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    for call in (lambda: B.attention_fwd(a), lambda: B.attention_bwd(a, g)):
        with pytest.raises(ValueError, match="current GPU"):
            call()


def test_sizes_that_the_descriptors_cannot_hold():
    big = (1 << 32) + 64
    e = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="meta")
    for b, nq, nk, h, kv in ((big, 1, 1, 1, 1), (1, big, 1, 1, 1), (1, 1, big, 1, 1), (1, 1, 1, big, 1), (1, 1, 1, 1, big)):
        with pytest.raises(ValueError, match="32 bits"):
            B.attention_struct(e(b, nq, h, 8), e(b, nk, kv, 8), e(b, nk, kv, 8), e(b, nq, h, 8))
