"""ctypes binding of libgs_hip.so (C ABI in include/gs.h).

Argument marshalling only: torch tensors supply device memory and the
stream, every step of the rasterizer runs in the HIP library.  There is no
fallback: if the library is missing or a call fails, an exception is raised.
"""

from __future__ import annotations

import ctypes as C
import os
from typing import Dict, Optional, Sequence

import torch

from . import build as _build

GS_OK, GS_ERR_INVALID_ARG, GS_ERR_UNSUPPORTED, GS_ERR_WORKSPACE, GS_ERR_HIP = range(5)
GS_SH_F32, GS_SH_F16, GS_SH_Q8 = 0, 1, 2
GS_ADAM_F32, GS_ADAM_Q8LOG = 0, 1
GS_ADAM_DENSE, GS_ADAM_LAZY = 0, 1
GS_DTYPE_F32, GS_DTYPE_F16, GS_DTYPE_BF16, GS_DTYPE_MXFP8 = 0, 1, 2, 3
GS_ACT = {"none": 0, "relu": 1, "silu": 2, "gelu": 3}
SPLAT_FLOATS = 12          # gs_splat is 48 bytes


class GsCamera(C.Structure):
    _fields_ = [("width", C.c_int32), ("height", C.c_int32), ("fx", C.c_float), ("fy", C.c_float),
                ("cx", C.c_float), ("cy", C.c_float), ("viewmat", C.c_float * 12),
                ("znear", C.c_float), ("guard", C.c_float), ("lod_min_radius_px", C.c_float),
                ("time", C.c_float)]


class GsFwdView(C.Structure):
    _fields_ = [("camera", GsCamera), ("splats", C.c_void_p), ("vals", C.c_void_p),
                ("tile_ranges", C.c_void_p), ("schedule", C.c_void_p), ("image", C.c_void_p),
                ("final_T", C.c_void_p), ("n_contrib", C.c_void_p), ("weight", C.c_void_p),
                ("reached_lists", C.c_int32)]


class GsSortView(C.Structure):
    _fields_ = [("camera", GsCamera), ("splats", C.c_void_p), ("n", C.c_int64), ("k_capacity", C.c_int64),
                ("vals", C.c_void_p), ("tile_ranges", C.c_void_p), ("schedule", C.c_void_p),
                ("bwd_index", C.c_void_p), ("keys", C.c_void_p), ("k_total", C.c_void_p),
                ("workspace", C.c_void_p), ("workspace_bytes", C.c_size_t),
                ("depth_keys", C.c_void_p), ("tile_rects", C.c_void_p), ("reach_tiles", C.c_int32)]


class GsBinKeys(C.Structure):
    _fields_ = [("depth_keys", C.c_void_p), ("tile_rects", C.c_void_p)]


class GsBwdView(C.Structure):
    _fields_ = [("camera", GsCamera), ("n", C.c_int64), ("splats", C.c_void_p), ("vals", C.c_void_p),
                ("tile_ranges", C.c_void_p), ("schedule", C.c_void_p), ("bwd_index", C.c_void_p),
                ("k_capacity", C.c_int64), ("final_T", C.c_void_p), ("n_contrib", C.c_void_p),
                ("dL_dimage", C.c_void_p), ("g2", C.c_void_p), ("workspace", C.c_void_p),
                ("workspace_bytes", C.c_size_t), ("reached_lists", C.c_int32)]


class GsGaussians(C.Structure):
    _fields_ = [("n", C.c_int64), ("sh_degree", C.c_int32), ("sh_dtype", C.c_int32),
                ("means", C.c_void_p), ("scales", C.c_void_p), ("quats", C.c_void_p),
                ("opacities", C.c_void_p), ("sh", C.c_void_p), ("active", C.c_void_p),
                ("sh_bounds", C.c_void_p), ("velocity", C.c_void_p), ("t_offset", C.c_void_p)]


class GsGrads(C.Structure):
    _fields_ = [("means", C.c_void_p), ("log_scales", C.c_void_p), ("quats", C.c_void_p),
                ("opacity_logits", C.c_void_p), ("sh", C.c_void_p), ("velocity", C.c_void_p),
                ("t_offset", C.c_void_p)]


class GsShAdam(C.Structure):
    _fields_ = [("n", C.c_int64), ("rows", C.c_int32), ("value_dtype", C.c_int32),
                ("state_dtype", C.c_int32), ("step", C.c_int32), ("lr", C.c_float),
                ("beta1", C.c_float), ("beta2", C.c_float), ("eps", C.c_float), ("update", C.c_int32),
                ("grad", C.c_void_p), ("value", C.c_void_p), ("m", C.c_void_p), ("v", C.c_void_p),
                ("m_bounds", C.c_void_p), ("v_bounds", C.c_void_p)]


class GsRmsNorm(C.Structure):
    _fields_ = [("m", C.c_int64), ("n", C.c_int32), ("dtype", C.c_int32), ("y_dtype", C.c_int32), ("eps", C.c_float),
                ("x", C.c_void_p), ("x_stride", C.c_int64), ("residual", C.c_void_p), ("residual_stride", C.c_int64),
                ("gamma", C.c_void_p), ("sum", C.c_void_p), ("sum_stride", C.c_int64), ("y", C.c_void_p),
                ("y_stride", C.c_int64), ("y_scales", C.c_void_p), ("y_scales_stride", C.c_int64),
                ("rstd", C.c_void_p)]


class GsRmsNormGrads(C.Structure):
    _fields_ = [("m", C.c_int64), ("n", C.c_int32), ("dtype", C.c_int32), ("sum", C.c_void_p),
                ("sum_stride", C.c_int64), ("rstd", C.c_void_p), ("gamma", C.c_void_p), ("dy", C.c_void_p),
                ("dy_stride", C.c_int64), ("dsum", C.c_void_p), ("dsum_stride", C.c_int64), ("dx", C.c_void_p),
                ("dx_stride", C.c_int64), ("dgamma", C.c_void_p), ("accumulate", C.c_int32)]


class GsLinear(C.Structure):
    _fields_ = [("m", C.c_int64), ("n", C.c_int32), ("k", C.c_int32), ("dtype", C.c_int32), ("y_dtype", C.c_int32),
                ("activation", C.c_int32), ("planes", C.c_int32), ("x", C.c_void_p), ("x_stride", C.c_int64),
                ("w", C.c_void_p), ("w_stride", C.c_int64), ("x_scales", C.c_void_p), ("x_scales_stride", C.c_int64),
                ("w_scales", C.c_void_p), ("w_scales_stride", C.c_int64), ("bias", C.c_void_p),
                ("residual", C.c_void_p), ("residual_stride", C.c_int64), ("y", C.c_void_p), ("y_stride", C.c_int64),
                ("z", C.c_void_p), ("z_stride", C.c_int64)]
    device = None              # of the tensors (linear_struct)


class GsLinearGrads(C.Structure):
    _fields_ = [("dy", C.c_void_p), ("dy_stride", C.c_int64), ("dx", C.c_void_p), ("dx_stride", C.c_int64),
                ("dw", C.c_void_p), ("dw_stride", C.c_int64), ("dw_dtype", C.c_int32), ("accumulate", C.c_int32),
                ("db", C.c_void_p)]
    dy_dtype = None            # gs_dtype of dy (linear_grads_struct)


class GsMuon(C.Structure):
    _fields_ = [("batch", C.c_int32), ("rows", C.c_int32), ("cols", C.c_int32), ("grad_dtype", C.c_int32),
                ("out_dtype", C.c_int32), ("steps", C.c_int32), ("a", C.c_float), ("b", C.c_float), ("c", C.c_float),
                ("eps", C.c_float), ("lr", C.c_float), ("beta", C.c_float), ("weight_decay", C.c_float),
                ("scale", C.c_float), ("nesterov", C.c_int32), ("grad", C.c_void_p), ("out", C.c_void_p),
                ("momentum", C.c_void_p), ("momentum_out", C.c_void_p), ("weight", C.c_void_p),
                ("weight_out", C.c_void_p)]
    device = None              # of the tensors (muon_struct)


def _tensor_fields(name):
    return [(name, C.c_void_p)] + [(f"{name}_{dim}", C.c_int64) for dim in ("batch", "row", "head")]


class GsAttention(C.Structure):
    _fields_ = [("batch", C.c_int32), ("heads", C.c_int32), ("kv_heads", C.c_int32), ("nq", C.c_int32), ("nk", C.c_int32),
                ("d", C.c_int32), ("dtype", C.c_int32), ("scale", C.c_float), *_tensor_fields("q"), *_tensor_fields("k"),
                *_tensor_fields("v"), *_tensor_fields("out"), ("lse", C.c_void_p), ("kv_lengths", C.c_void_p),
                ("kv_mask", C.c_void_p), ("kv_mask_stride", C.c_int64)]
    device = None              # of the tensors (attention_struct)


class GsAttentionGrads(C.Structure):
    _fields_ = [*_tensor_fields("dout"), *_tensor_fields("dq"), *_tensor_fields("dk"), *_tensor_fields("dv")]


class GsGroupNorm(C.Structure):
    _fields_ = [("n", C.c_int32), ("c", C.c_int32), ("groups", C.c_int32), ("dtype", C.c_int32), ("activation", C.c_int32),
                ("eps", C.c_float), ("p", C.c_int64), ("x", C.c_void_p), ("x_image", C.c_int64), ("x_pixel", C.c_int64),
                ("gamma", C.c_void_p), ("beta", C.c_void_p), ("y", C.c_void_p), ("y_image", C.c_int64),
                ("y_pixel", C.c_int64), ("mean", C.c_void_p), ("rstd", C.c_void_p), ("kept", C.c_void_p),
                ("kept_image", C.c_int64), ("kept_pixel", C.c_int64), ("kept_scales", C.c_void_p),
                ("kept_scales_image", C.c_int64), ("kept_scales_pixel", C.c_int64)]


class GsGroupNormGrads(C.Structure):
    _fields_ = [("n", C.c_int32), ("c", C.c_int32), ("groups", C.c_int32), ("dtype", C.c_int32), ("x_dtype", C.c_int32),
                ("activation", C.c_int32), ("accumulate", C.c_int32), ("p", C.c_int64), ("x", C.c_void_p),
                ("x_image", C.c_int64), ("x_pixel", C.c_int64), ("x_scales", C.c_void_p), ("x_scales_image", C.c_int64),
                ("x_scales_pixel", C.c_int64), ("mean", C.c_void_p), ("rstd", C.c_void_p), ("gamma", C.c_void_p),
                ("beta", C.c_void_p), ("dy", C.c_void_p), ("dy_image", C.c_int64), ("dy_pixel", C.c_int64),
                ("dx", C.c_void_p), ("dx_image", C.c_int64), ("dx_pixel", C.c_int64), ("dgamma", C.c_void_p),
                ("dbeta", C.c_void_p)]


class GsError(RuntimeError):
    pass


_lib = None
SYMBOLS = ("gs_project", "gs_bin_sort_workspace_bytes", "gs_schedule_words", "gs_bwd_index_words", "gs_bin_sort",
           "gs_bin_sort_views",
           "gs_render_fwd_views", "gs_render_bwd_screen_views", "gs_project_views", "gs_project_views_binned",
           "gs_render_fwd",
           "gs_render_bwd_workspace_bytes", "gs_render_bwd", "gs_render_bwd_screen_workspace_bytes",
           "gs_render_bwd_screen", "gs_project_bwd", "gs_project_bwd_binned", "gs_active_mask_workspace_bytes",
           "gs_active_mask", "gs_active_mask_static", "gs_active_mask_static_scratch_bytes",
           "gs_sh_q8_bounds_floats", "gs_sh_quantize8", "gs_sh_adam_step", "gs_rms_norm_fwd",
           "gs_rms_norm_bwd_workspace_bytes", "gs_rms_norm_bwd", "gs_mxfp8_quantize", "gs_linear_fwd_workspace_bytes",
           "gs_linear_fwd", "gs_linear_bwd_workspace_bytes", "gs_linear_bwd", "gs_muon_workspace_bytes",
           "gs_orthogonalize", "gs_muon_step", "gs_attention_fwd_workspace_bytes", "gs_attention_fwd",
           "gs_attention_bwd_workspace_bytes", "gs_attention_bwd", "gs_group_norm_fwd_workspace_bytes", "gs_group_norm_fwd",
           "gs_group_norm_bwd_workspace_bytes", "gs_group_norm_bwd", "gs_status_string",
           "gs_version")


def lib_path() -> str:
    return _build.LIB


def lib():
    """Load the HIP library (built in tree by build.py); raise if absent."""
    global _lib
    if _lib is not None:
        return _lib
    path = lib_path()
    if not os.path.exists(path):
        raise GsError(f"HIP library not built: {path} (run python -m gaussian_splatting_tile_amd.build)")
    L = C.CDLL(path)
    for name in SYMBOLS:
        getattr(L, name)
    vp, i64, sz = C.c_void_p, C.c_int64, C.c_size_t
    L.gs_project.argtypes = [C.POINTER(GsGaussians), C.POINTER(GsCamera), vp, vp]
    L.gs_bin_sort_workspace_bytes.argtypes = [i64, i64, C.c_int32]
    L.gs_bin_sort_workspace_bytes.restype = sz
    L.gs_schedule_words.argtypes = [C.c_int32, C.c_int32]
    L.gs_schedule_words.restype = sz
    L.gs_bwd_index_words.argtypes = [i64, i64]
    L.gs_bwd_index_words.restype = sz
    L.gs_bin_sort.argtypes = [vp, i64, C.POINTER(GsCamera), i64, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.gs_bin_sort_views.argtypes = [C.c_int32, C.POINTER(GsSortView), vp]
    L.gs_render_fwd.argtypes = [vp, vp, vp, vp, C.POINTER(GsCamera), vp, vp, vp, vp, vp]
    L.gs_render_fwd_views.argtypes = [C.c_int32, C.POINTER(GsFwdView), vp, vp]
    L.gs_project_views.argtypes = [C.POINTER(GsGaussians), C.c_int32, C.POINTER(GsCamera), C.POINTER(vp), vp]
    L.gs_project_views_binned.argtypes = [C.POINTER(GsGaussians), C.c_int32, C.POINTER(GsCamera), C.POINTER(vp),
                                          C.POINTER(GsBinKeys), vp]
    L.gs_render_bwd_screen_views.argtypes = [C.c_int32, C.POINTER(GsBwdView), vp, vp]
    L.gs_render_bwd_workspace_bytes.argtypes = [i64, i64]
    L.gs_render_bwd_workspace_bytes.restype = sz
    L.gs_render_bwd.argtypes = [C.POINTER(GsGaussians), C.POINTER(GsCamera), vp, vp, vp, vp, vp, i64, vp, vp,
                                vp, vp, C.POINTER(GsGrads), vp, sz, vp]
    L.gs_render_bwd_screen_workspace_bytes.argtypes = [i64]
    L.gs_render_bwd_screen_workspace_bytes.restype = sz
    L.gs_render_bwd_screen.argtypes = [C.POINTER(GsCamera), i64, vp, vp, vp, vp, vp, i64, vp, vp, vp, vp, vp,
                                       vp, sz, vp]
    L.gs_project_bwd.argtypes = [C.POINTER(GsGaussians), C.c_int32, C.POINTER(GsCamera), C.POINTER(vp),
                                 C.POINTER(vp), C.POINTER(GsGrads), vp]
    L.gs_project_bwd_binned.argtypes = [C.POINTER(GsGaussians), C.c_int32, C.POINTER(GsCamera), C.POINTER(vp),
                                        C.POINTER(vp), C.POINTER(vp), C.POINTER(GsGrads), vp]
    L.gs_active_mask_workspace_bytes.argtypes = [i64]
    L.gs_active_mask_workspace_bytes.restype = sz
    L.gs_active_mask.argtypes = [vp, i64, i64, vp, vp, sz, vp]
    L.gs_active_mask_static.argtypes = [vp, i64, i64, vp, vp]
    L.gs_active_mask_static_scratch_bytes.argtypes = []
    L.gs_active_mask_static_scratch_bytes.restype = sz
    L.gs_sh_q8_bounds_floats.argtypes = [i64, C.c_int32]
    L.gs_sh_q8_bounds_floats.restype = sz
    L.gs_sh_quantize8.argtypes = [vp, i64, C.c_int32, vp, vp, vp]
    L.gs_sh_adam_step.argtypes = [C.POINTER(GsShAdam), vp]
    L.gs_rms_norm_fwd.argtypes = [C.POINTER(GsRmsNorm), vp]
    L.gs_rms_norm_bwd_workspace_bytes.argtypes = [i64, C.c_int32]
    L.gs_rms_norm_bwd_workspace_bytes.restype = sz
    L.gs_rms_norm_bwd.argtypes = [C.POINTER(GsRmsNormGrads), vp, sz, vp]
    L.gs_mxfp8_quantize.argtypes = [vp, C.c_int32, i64, C.c_int32, i64, vp, i64, vp, i64, vp]
    L.gs_linear_fwd_workspace_bytes.argtypes = [C.POINTER(GsLinear)]
    L.gs_linear_fwd_workspace_bytes.restype = sz
    L.gs_linear_fwd.argtypes = [C.POINTER(GsLinear), vp, sz, vp]
    L.gs_linear_bwd_workspace_bytes.argtypes = [C.POINTER(GsLinear), C.POINTER(GsLinearGrads)]
    L.gs_linear_bwd_workspace_bytes.restype = sz
    L.gs_linear_bwd.argtypes = [C.POINTER(GsLinear), C.POINTER(GsLinearGrads), vp, sz, vp]
    L.gs_muon_workspace_bytes.argtypes = [C.POINTER(GsMuon)]
    L.gs_muon_workspace_bytes.restype = sz
    L.gs_orthogonalize.argtypes = [C.POINTER(GsMuon), vp, sz, vp]
    L.gs_muon_step.argtypes = [C.POINTER(GsMuon), vp, sz, vp]
    L.gs_attention_fwd_workspace_bytes.argtypes = [C.POINTER(GsAttention)]
    L.gs_attention_fwd_workspace_bytes.restype = sz
    L.gs_attention_fwd.argtypes = [C.POINTER(GsAttention), vp, sz, vp]
    L.gs_attention_bwd_workspace_bytes.argtypes = [C.POINTER(GsAttention), C.POINTER(GsAttentionGrads)]
    L.gs_attention_bwd_workspace_bytes.restype = sz
    L.gs_attention_bwd.argtypes = [C.POINTER(GsAttention), C.POINTER(GsAttentionGrads), vp, sz, vp]
    for name in ("gs_group_norm_fwd_workspace_bytes", "gs_group_norm_bwd_workspace_bytes"):
        getattr(L, name).argtypes = [i64, i64, C.c_int32, C.c_int32]
        getattr(L, name).restype = sz
    L.gs_group_norm_fwd.argtypes = [C.POINTER(GsGroupNorm), vp, sz, vp]
    L.gs_group_norm_bwd.argtypes = [C.POINTER(GsGroupNormGrads), vp, sz, vp]
    L.gs_status_string.restype = C.c_char_p
    L.gs_status_string.argtypes = [C.c_int]
    L.gs_version.restype = C.c_int32
    for name in ("gs_project", "gs_project_views", "gs_project_views_binned", "gs_bin_sort", "gs_bin_sort_views", "gs_render_fwd",
                 "gs_render_fwd_views",
                 "gs_render_bwd",
                 "gs_render_bwd_screen", "gs_render_bwd_screen_views",
                 "gs_project_bwd", "gs_project_bwd_binned", "gs_active_mask", "gs_active_mask_static",
                 "gs_sh_quantize8", "gs_rms_norm_fwd", "gs_rms_norm_bwd", "gs_mxfp8_quantize", "gs_linear_fwd",
                 "gs_linear_bwd", "gs_orthogonalize", "gs_muon_step", "gs_attention_fwd", "gs_attention_bwd",
                 "gs_group_norm_fwd", "gs_group_norm_bwd"):
        getattr(L, name).restype = C.c_int
    _lib = L
    return L


def _check(status: int, what: str):
    if status != GS_OK:
        msg = lib().gs_status_string(status).decode()
        raise GsError(f"{what} failed: {msg} (status {status})")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream(stream=None):
    if stream is None:
        # the handle alone: making a Stream object of it takes 1.3 us, a tenth of a small call
        return C.c_void_p(torch._C._cuda_getCurrentRawStream(torch.cuda.current_device()))
    return C.c_void_p(stream.cuda_stream)


def _stream_for(device: Optional[torch.device], workspace: Optional[torch.Tensor], stream=None):
    """The stream of a call whose tensors are on `device` (None: not known).
    Kernels get bare addresses: the host's memory or another GPU's is refused
    here."""
    if device is None:
        return _stream(stream)
    index = device.index                                # None: the host; else the GPU is in use and its number at hand
    if index is None or index != torch._C._cuda_getDevice():
        raise ValueError(f"tensors on {device}: expected the current GPU")
    if workspace is not None and (workspace.get_device() != index or not workspace.is_contiguous()):
        raise ValueError("workspace: expected contiguous memory on the tensors' device")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(index)
    if stream.device != device:
        raise ValueError(f"stream of {stream.device} for tensors on {device}")
    return _stream(stream)


def camera_struct(cam) -> GsCamera:
    """From an object with width, height, fx, fy, cx, cy, viewmat[3][4],
    znear, guard, lod_min_radius_px (see scenes.Camera)."""
    c = GsCamera()
    c.width, c.height = int(cam.width), int(cam.height)
    c.fx, c.fy, c.cx, c.cy = float(cam.fx), float(cam.fy), float(cam.cx), float(cam.cy)
    vm = [float(x) for x in __import__("numpy").asarray(cam.viewmat, dtype="float32").reshape(-1)]
    for i in range(12):
        c.viewmat[i] = vm[i]
    c.znear, c.guard = float(cam.znear), float(cam.guard)
    c.lod_min_radius_px = float(getattr(cam, "lod_min_radius_px", 0.0))
    c.time = float(getattr(cam, "time", 0.0))
    return c


def grads_struct(grads: Dict[str, torch.Tensor]) -> GsGrads:
    """fp32 gradient arrays by name; "velocity" and "t_offset" only with
    moving Gaussians."""
    return GsGrads(_ptr(grads["means"]), _ptr(grads["log_scales"]), _ptr(grads["quats"]),
                   _ptr(grads["opacity_logits"]), _ptr(grads["sh"]), _ptr(grads.get("velocity")),
                   _ptr(grads.get("t_offset")))


def gaussians_struct(g: Dict[str, torch.Tensor], sh_degree: int, active: Optional[torch.Tensor] = None
                     ) -> GsGaussians:
    s = GsGaussians()
    s.n = int(g["means"].shape[1])
    s.sh_degree = int(sh_degree)
    s.sh_dtype = {torch.float16: GS_SH_F16, torch.uint8: GS_SH_Q8}.get(g["sh"].dtype, GS_SH_F32)
    for k in ("means", "scales", "quats", "opacities"):
        t = g[k]
        assert t.is_cuda and t.dtype == torch.float32 and t.is_contiguous(), k
    assert g["sh"].is_cuda and g["sh"].is_contiguous()
    s.means, s.scales, s.quats = g["means"].data_ptr(), g["scales"].data_ptr(), g["quats"].data_ptr()
    s.opacities, s.sh = g["opacities"].data_ptr(), g["sh"].data_ptr()
    if active is not None:
        assert active.is_cuda and active.dtype == torch.uint8 and active.is_contiguous()
        s.active = active.data_ptr()
    if s.sh_dtype == GS_SH_Q8:
        b = g["sh_bounds"]
        assert b.is_cuda and b.dtype == torch.float32 and b.is_contiguous()
        s.sh_bounds = b.data_ptr()
    if g.get("velocity") is not None:
        v, t = g["velocity"], g["t_offset"]
        assert v.is_cuda and v.dtype == torch.float32 and v.is_contiguous() and tuple(v.shape) == (3, s.n)
        assert t.is_cuda and t.dtype == torch.float32 and t.is_contiguous() and t.numel() == s.n
        s.velocity, s.t_offset = v.data_ptr(), t.data_ptr()
    return s


def sh_q8_bounds_floats(n: int, rows: int) -> int:
    return int(lib().gs_sh_q8_bounds_floats(n, rows))


def sh_quantize8(sh: torch.Tensor, codes: torch.Tensor, bounds: torch.Tensor, stream=None):
    """gs_sh_quantize8: sh float32 [K][3][n] -> codes uint8 [K][3][n], bounds
    float32 [K*3][ceil(n/256)][2]."""
    K, c3, n = sh.shape
    assert sh.dtype == torch.float32 and sh.is_contiguous() and codes.dtype == torch.uint8
    assert bounds.numel() >= sh_q8_bounds_floats(n, K * c3)
    _check(lib().gs_sh_quantize8(_ptr(sh), int(n), int(K * c3), _ptr(codes), _ptr(bounds), _stream(stream)),
           "gs_sh_quantize8")


def sh_adam_struct(grad: torch.Tensor, value: torch.Tensor, m: torch.Tensor, v: torch.Tensor,
                   m_bounds: Optional[torch.Tensor] = None, v_bounds: Optional[torch.Tensor] = None,
                   step: int = 1, lr: float = 1e-3, beta1: float = 0.9, beta2: float = 0.999,
                   eps: float = 1e-15, lazy: bool = True) -> GsShAdam:
    """Descriptor of gs_sh_adam_step over [rows][n] (or [K][3][n]) arrays:
    grad float32; value float32 or float16; m, v float32 (full-precision
    state) or uint8 codes with float32 bounds [rows][ceil(n/256)][2];
    lazy: units with a zero gradient keep their state (else every unit
    moves)."""
    n = grad.shape[-1]
    rows = grad.numel() // n if n else grad.shape[0]
    for t in (grad, value, m, v):
        assert t.is_contiguous() and t.shape == grad.shape, "arrays must be contiguous and of one shape"
    assert grad.dtype == torch.float32 and value.dtype in (torch.float32, torch.float16)
    a = GsShAdam()
    a.n, a.rows, a.step = int(n), int(rows), int(step)
    a.value_dtype = GS_SH_F16 if value.dtype == torch.float16 else GS_SH_F32
    a.lr, a.beta1, a.beta2, a.eps = float(lr), float(beta1), float(beta2), float(eps)
    a.update = GS_ADAM_LAZY if lazy else GS_ADAM_DENSE
    a.grad, a.value, a.m, a.v = _ptr(grad), _ptr(value), _ptr(m), _ptr(v)
    if m.dtype == torch.uint8:
        assert v.dtype == torch.uint8 and m_bounds is not None and v_bounds is not None
        nbf = sh_q8_bounds_floats(n, rows)
        assert m_bounds.dtype == torch.float32 and m_bounds.numel() >= nbf and m_bounds.is_contiguous()
        assert v_bounds.dtype == torch.float32 and v_bounds.numel() >= nbf and v_bounds.is_contiguous()
        a.state_dtype = GS_ADAM_Q8LOG
        a.m_bounds, a.v_bounds = _ptr(m_bounds), _ptr(v_bounds)
    else:
        assert m.dtype == torch.float32 and v.dtype == torch.float32
        a.state_dtype = GS_ADAM_F32
    return a


def sh_adam_step(grad, value, m, v, m_bounds=None, v_bounds=None, step=1, lr=1e-3, beta1=0.9,
                 beta2=0.999, eps=1e-15, stream=None, lazy=True):
    """gs_sh_adam_step: one fused Adam update of value, m, v (and the bounds)
    in place; lazy (SparseAdam's rule) or dense (every unit)."""
    a = sh_adam_struct(grad, value, m, v, m_bounds, v_bounds, step, lr, beta1, beta2, eps, lazy)
    _check(lib().gs_sh_adam_step(C.byref(a), _stream(stream)), "gs_sh_adam_step")


# ---- the four calls ---------------------------------------------------------
def project(gs: GsGaussians, cam: GsCamera, splats: torch.Tensor, stream=None):
    _check(lib().gs_project(C.byref(gs), C.byref(cam), _ptr(splats), _stream(stream)), "gs_project")


def bin_sort_workspace_bytes(n: int, k_capacity: int, n_tiles: int) -> int:
    return int(lib().gs_bin_sort_workspace_bytes(n, k_capacity, n_tiles))


def _nbytes(t):
    return 0 if t is None else t.nbytes


def schedule_words(width: int, height: int) -> int:
    return int(lib().gs_schedule_words(width, height))


def bwd_index_words(n: int, k_capacity: int) -> int:
    return int(lib().gs_bwd_index_words(n, k_capacity))


def bin_sort(splats, n, cam: GsCamera, k_capacity, vals, tile_ranges, schedule, bwd_index, keys, k_total,
             workspace, stream=None):
    _check(lib().gs_bin_sort(_ptr(splats), int(n), C.byref(cam), int(k_capacity), _ptr(vals),
                             _ptr(tile_ranges), _ptr(schedule), _ptr(bwd_index), _ptr(keys), _ptr(k_total),
                             _ptr(workspace), _nbytes(workspace), _stream(stream)), "gs_bin_sort")


def bin_sort_views(bufs, with_bwd: bool = True, stream=None, prebinned=False, reach=False):
    """gs_bin_sort_views over ViewBuffers objects (their splats must be
    current): one launch per sort step for up to 8 views.  prebinned: take
    the depth keys and tile rects that project_views(..., binned=True) wrote
    into the buffers with those splats (one flag for all views, or one per
    view).  reach: list each Gaussian only in the tiles it reaches (one flag
    for all views, or one per view)."""
    nv = len(bufs)
    pre = list(prebinned) if isinstance(prebinned, (list, tuple)) else [prebinned] * nv
    rch = list(reach) if isinstance(reach, (list, tuple)) else [reach] * nv
    arr = (GsSortView * max(nv, 1))()
    for i, b in enumerate(bufs):
        b.reached = bool(rch[i])
        arr[i] = GsSortView(b.camc, _ptr(b.splats), int(b.n), int(b.k_capacity), _ptr(b.vals), _ptr(b.ranges),
                            _ptr(b.schedule), _ptr(b.bwd_index) if with_bwd else None, _ptr(b.keys),
                            _ptr(b.k_total),
                            _ptr(b.ws), _nbytes(b.ws),
                            _ptr(b.depth_keys) if pre[i] else None,
                            _ptr(b.tile_rects) if pre[i] and not rch[i] else None, 1 if rch[i] else 0)
    _check(lib().gs_bin_sort_views(nv, arr, _stream(stream)), "gs_bin_sort_views")


def render_fwd(splats, vals, tile_ranges, schedule, cam: GsCamera, bg: Sequence[float], image, final_T,
               n_contrib, stream=None):
    bgv = (C.c_float * 3)(*[float(x) for x in bg])
    _check(lib().gs_render_fwd(_ptr(splats), _ptr(vals), _ptr(tile_ranges), _ptr(schedule), C.byref(cam),
                               C.cast(bgv, C.c_void_p), _ptr(image), _ptr(final_T), _ptr(n_contrib),
                               _stream(stream)), "gs_render_fwd")


def project_views(gs: GsGaussians, cams, splats_list, stream=None, bin_keys=None):
    """gs_project_views: records for every camera of the list in one pass.
    bin_keys: None, or one (depth_keys uint32/int32 [n], tile_rects
    uint32/int32 [2n] or None) pair (or None) per camera, for
    gs_project_views_binned (rects may be left out for views sorted with
    reach=True)."""
    nv = len(cams)
    cam_arr = (GsCamera * max(nv, 1))(*cams)
    sp_arr = (C.c_void_p * max(nv, 1))(*[_ptr(t) for t in splats_list])
    if bin_keys is None:
        _check(lib().gs_project_views(C.byref(gs), nv, cam_arr, sp_arr, _stream(stream)), "gs_project_views")
        return
    bk = (GsBinKeys * max(nv, 1))()
    for i, pair in enumerate(bin_keys):
        if pair is not None:
            bk[i] = GsBinKeys(_ptr(pair[0]), None if pair[1] is None else _ptr(pair[1]))
    _check(lib().gs_project_views_binned(C.byref(gs), nv, cam_arr, sp_arr, bk, _stream(stream)),
           "gs_project_views_binned")


def render_fwd_views(bufs, bg: Sequence[float] = (0.0, 0.0, 0.0), stream=None, weights=None):
    """gs_render_fwd_views over ViewBuffers objects (their splats, bins and
    schedules must be current).  weights: None, one float32 [n] tensor shared
    by all views, or a list with one tensor (or None) per view; the
    per-Gaussian blending weights are added to it."""
    nv = len(bufs)
    if weights is None or isinstance(weights, torch.Tensor):
        weights = [weights] * nv
    arr = (GsFwdView * max(nv, 1))()
    for i, b in enumerate(bufs):
        arr[i] = GsFwdView(b.camc, _ptr(b.splats), _ptr(b.vals), _ptr(b.ranges), _ptr(b.schedule),
                           _ptr(b.image), _ptr(b.final_T), _ptr(b.n_contrib), _ptr(weights[i]),
                           1 if getattr(b, "reached", False) else 0)
    bgv = (C.c_float * 3)(*[float(x) for x in bg])
    _check(lib().gs_render_fwd_views(nv, arr, C.cast(bgv, C.c_void_p), _stream(stream)), "gs_render_fwd_views")


def render_bwd_workspace_bytes(n: int, k_capacity: int) -> int:
    return int(lib().gs_render_bwd_workspace_bytes(n, k_capacity))


def render_bwd(gs: GsGaussians, cam: GsCamera, splats, vals, tile_ranges, schedule, bwd_index, k_capacity, bg,
               final_T, n_contrib, dL_dimage, grads: Dict[str, torch.Tensor], workspace, stream=None):
    bgv = (C.c_float * 3)(*[float(x) for x in bg])
    gr = grads_struct(grads)
    _check(lib().gs_render_bwd(C.byref(gs), C.byref(cam), _ptr(splats), _ptr(vals), _ptr(tile_ranges),
                               _ptr(schedule), _ptr(bwd_index), int(k_capacity), C.cast(bgv, C.c_void_p), _ptr(final_T), _ptr(n_contrib), _ptr(dL_dimage),
                               C.byref(gr), _ptr(workspace),
                               workspace.numel() * workspace.element_size(), _stream(stream)),
           "gs_render_bwd")


def render_bwd_screen_workspace_bytes(k_capacity: int) -> int:
    return int(lib().gs_render_bwd_screen_workspace_bytes(k_capacity))


def render_bwd_screen(cam: GsCamera, n, splats, vals, tile_ranges, schedule, bwd_index, k_capacity, bg, final_T,
                      n_contrib, dL_dimage, g2, workspace, stream=None):
    bgv = (C.c_float * 3)(*[float(x) for x in bg])
    _check(lib().gs_render_bwd_screen(C.byref(cam), int(n), _ptr(splats), _ptr(vals), _ptr(tile_ranges),
                                      _ptr(schedule), _ptr(bwd_index), int(k_capacity), C.cast(bgv, C.c_void_p),
                                      _ptr(final_T), _ptr(n_contrib), _ptr(dL_dimage), _ptr(g2), _ptr(workspace),
                                      _nbytes(workspace), _stream(stream)), "gs_render_bwd_screen")


def render_bwd_screen_views(bufs, dLs, g2s, workspaces, bg: Sequence[float] = (0.0, 0.0, 0.0), stream=None):
    """gs_render_bwd_screen_views over ViewBuffers objects with their upstream
    gradients, g2 outputs [n][9] and workspaces."""
    nv = len(bufs)
    arr = (GsBwdView * max(nv, 1))()
    for i, (b, dL, g2, ws) in enumerate(zip(bufs, dLs, g2s, workspaces)):
        arr[i] = GsBwdView(b.camc, b.n, _ptr(b.splats), _ptr(b.vals), _ptr(b.ranges), _ptr(b.schedule),
                           _ptr(b.bwd_index), b.k_capacity, _ptr(b.final_T), _ptr(b.n_contrib), _ptr(dL),
                           _ptr(g2), _ptr(ws), _nbytes(ws), 1 if getattr(b, "reached", False) else 0)
    bgv = (C.c_float * 3)(*[float(x) for x in bg])
    _check(lib().gs_render_bwd_screen_views(nv, arr, C.cast(bgv, C.c_void_p), _stream(stream)),
           "gs_render_bwd_screen_views")


def project_bwd(gs: GsGaussians, cams, splats_list, g2_list, grads: Dict[str, torch.Tensor], stream=None,
                depth_keys=None):
    """Chain rule of a batch of views: cams is a list of GsCamera, splats_list
    and g2_list the matching device tensors.  depth_keys (a list of the views'
    depth-key tensors from project_views(bin_keys=...), None entries allowed)
    selects gs_project_bwd_binned, which takes visibility from the keys."""
    nv = len(cams)
    cam_arr = (GsCamera * max(nv, 1))(*cams)
    sp_arr = (C.c_void_p * max(nv, 1))(*[_ptr(t) for t in splats_list])
    g2_arr = (C.c_void_p * max(nv, 1))(*[_ptr(t) for t in g2_list])
    gr = grads_struct(grads)
    if depth_keys is None:
        _check(lib().gs_project_bwd(C.byref(gs), nv, cam_arr, sp_arr, g2_arr, C.byref(gr), _stream(stream)),
               "gs_project_bwd")
        return
    if len(depth_keys) != nv:
        raise ValueError("project_bwd: one depth-key tensor (or None) per view")
    dk_arr = (C.c_void_p * max(nv, 1))(*[None if t is None else _ptr(t) for t in depth_keys])
    _check(lib().gs_project_bwd_binned(C.byref(gs), nv, cam_arr, sp_arr, g2_arr, dk_arr, C.byref(gr),
                                       _stream(stream)), "gs_project_bwd_binned")


def active_mask_workspace_bytes(n: int) -> int:
    return int(lib().gs_active_mask_workspace_bytes(n))


def active_mask(scores, n, keep, mask, workspace, stream=None):
    _check(lib().gs_active_mask(_ptr(scores), int(n), int(keep), _ptr(mask), _ptr(workspace),
                                0 if workspace is None else workspace.numel() * workspace.element_size(),
                                _stream(stream)), "gs_active_mask")


def active_mask_static(scores, n, keep, mask, stream=None):
    """gs_active_mask with the library's fixed scratch array: no workspace,
    nothing allocated (n up to 2^30)."""
    _check(lib().gs_active_mask_static(_ptr(scores), int(n), int(keep), _ptr(mask), _stream(stream)),
           "gs_active_mask_static")


# ---- a network head that predicts Gaussians ---------------------------------
_DTYPES = {torch.float32: GS_DTYPE_F32, torch.float16: GS_DTYPE_F16, torch.bfloat16: GS_DTYPE_BF16,
           torch.float8_e4m3fn: GS_DTYPE_MXFP8}
_BY_CODE = {code: t for t, code in _DTYPES.items()}
_SCALES = (torch.uint8, torch.float8_e8m0fnu)


def _dtype(t: torch.Tensor) -> int:
    try:
        return _DTYPES[t.dtype]
    except KeyError:
        raise ValueError(f"unsupported element type {t.dtype}") from None


def _int32(*sizes: int):
    """ctypes cuts larger values to their low bits."""
    for size in sizes:
        if size >> 31:
            raise ValueError(f"sizes {sizes}: more than 32 bits hold")


def _rows(t: Optional[torch.Tensor], rows: int, cols: int, what: str, dtypes=None, device=None):
    """(address, row stride) of a [rows][cols] tensor whose rows are
    contiguous; (None, cols) for None."""
    if t is None:
        return None, cols
    if t.shape != (rows, cols):
        raise ValueError(f"{what}: expected [{rows}][{cols}], got {tuple(t.shape)}")
    if dtypes is not None and t.dtype not in dtypes:
        raise ValueError(f"{what}: unexpected element type {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{what}: on {t.device}, another device than the others")
    stride, step = t.stride()
    if rows <= 1:
        stride = cols
    if (step != 1 and cols > 1) or stride < cols:
        raise ValueError(f"{what}: rows must be contiguous and must not overlap (strides {t.stride()})")
    return t.data_ptr(), stride


def _vector(t: Optional[torch.Tensor], n: int, what: str, device=None):
    if t is None:
        return None
    if t.dtype is not torch.float32 or t.numel() != n or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{what}: expected {n} contiguous float32 values on the others' device")
    return t.data_ptr()


def rms_norm_fwd(x: torch.Tensor, y: torch.Tensor, gamma: Optional[torch.Tensor] = None,
                 residual: Optional[torch.Tensor] = None, sum_out: Optional[torch.Tensor] = None,
                 rstd: Optional[torch.Tensor] = None, y_scales: Optional[torch.Tensor] = None, eps: float = 1e-6,
                 stream=None):
    """gs_rms_norm_fwd over the rows of x [m][n] (float32, float16 or
    bfloat16): y = (x + residual) * rstd * gamma in x's type, or
    torch.float8_e4m3fn with y_scales [m][n / 32] (uint8 or float8_e8m0fnu)."""
    m, n = x.shape
    _int32(n)
    own, dev = (x.dtype,), x.device
    a = GsRmsNorm(m, n, _dtype(x), _dtype(y), eps, *_rows(x, m, n, "x"), *_rows(residual, m, n, "residual", own, dev),
                  _vector(gamma, n, "gamma", dev), *_rows(sum_out, m, n, "sum_out", own, dev),
                  *_rows(y, m, n, "y", (x.dtype, torch.float8_e4m3fn), dev),
                  *_rows(y_scales, m, n // 32, "y_scales", _SCALES, dev), _vector(rstd, m, "rstd", dev))
    _check(lib().gs_rms_norm_fwd(C.byref(a), _stream_for(dev, None, stream)), "gs_rms_norm_fwd")


def rms_norm_bwd_workspace_bytes(m: int, n: int) -> int:
    _int32(n)
    return int(lib().gs_rms_norm_bwd_workspace_bytes(m, n))


def rms_norm_bwd(sum_in: torch.Tensor, rstd: torch.Tensor, dy: torch.Tensor, dx: torch.Tensor,
                 gamma: Optional[torch.Tensor] = None, dsum: Optional[torch.Tensor] = None,
                 dgamma: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                 accumulate: bool = False, stream=None):
    """gs_rms_norm_bwd: from the kept sum (x without a residual) and rstd, the
    gradient dx of x and residual and, with dgamma and a workspace of
    rms_norm_bwd_workspace_bytes(m, n), that of gamma."""
    m, n = sum_in.shape
    _int32(n)
    own, dev = (sum_in.dtype,), sum_in.device
    a = GsRmsNormGrads(m, n, _dtype(sum_in), *_rows(sum_in, m, n, "sum_in"), _vector(rstd, m, "rstd", dev),
                       _vector(gamma, n, "gamma", dev), *_rows(dy, m, n, "dy", own, dev),
                       *_rows(dsum, m, n, "dsum", own, dev), *_rows(dx, m, n, "dx", own, dev),
                       _vector(dgamma, n, "dgamma", dev), 1 if accumulate else 0)
    _check(lib().gs_rms_norm_bwd(C.byref(a), _ptr(workspace), _nbytes(workspace), _stream_for(dev, workspace, stream)),
           "gs_rms_norm_bwd")


def mxfp8_quantize(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, stream=None):
    """gs_mxfp8_quantize: x [m][n] -> codes float8_e4m3fn [m][n] and scales
    [m][n / 32] (uint8 or float8_e8m0fnu)."""
    m, n = x.shape
    _int32(n)
    dev = x.device
    xp, xs = _rows(x, m, n, "x")
    cp, cs = _rows(codes, m, n, "codes", (torch.float8_e4m3fn,), dev)
    sp, ss = _rows(scales, m, n // 32, "scales", _SCALES, dev)
    _check(lib().gs_mxfp8_quantize(xp, _dtype(x), m, n, xs, cp, cs, sp, ss, _stream_for(dev, None, stream)),
           "gs_mxfp8_quantize")


def linear_struct(x: torch.Tensor, w: torch.Tensor, y: Optional[torch.Tensor],
                  bias: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
                  z: Optional[torch.Tensor] = None, act: str = "none", planes: bool = False,
                  x_scales: Optional[torch.Tensor] = None, w_scales: Optional[torch.Tensor] = None) -> GsLinear:
    """Descriptor of y = act(x w^T + bias) + residual: x [m][k] and w [n][k] of
    one type; y [m][n], or with planes [n][m] (None for the backward alone);
    z: the pre-activation kept for the backward, [m][n] of x's type."""
    m, k = x.shape
    n = w.shape[0]
    _int32(n, k)
    own, dev = (x.dtype,), x.device
    rows, cols = (n, m) if planes else (m, n)
    yt = None if y is None else (y.dtype,)
    block = x.dtype is torch.float8_e4m3fn
    a = GsLinear(m, n, k, _dtype(x), _dtype(x if y is None else y), GS_ACT[act], 1 if planes else 0,
                 *_rows(x, m, k, "x"), *_rows(w, n, k, "w", own, dev),
                 *(_rows(x_scales, m, k // 32, "x_scales", _SCALES, dev) if block else (None, 0)),
                 *(_rows(w_scales, n, k // 32, "w_scales", _SCALES, dev) if block else (None, 0)),
                 _vector(bias, n, "bias", dev), *_rows(residual, rows, cols, "residual", yt, dev),
                 *_rows(y, rows, cols, "y", None, dev), *_rows(z, m, n, "z", own, dev))
    a.device = dev
    return a


def linear_fwd_workspace_bytes(a: GsLinear) -> int:
    return int(lib().gs_linear_fwd_workspace_bytes(C.byref(a)))


def linear_fwd(a: GsLinear, workspace: Optional[torch.Tensor] = None, stream=None):
    """gs_linear_fwd of a linear_struct; the tensors it was made from must be
    alive."""
    _check(lib().gs_linear_fwd(C.byref(a), _ptr(workspace), _nbytes(workspace), _stream_for(a.device, workspace, stream)),
           "gs_linear_fwd")


def linear_grads_struct(a: GsLinear, dy: torch.Tensor, dx: Optional[torch.Tensor] = None,
                        dw: Optional[torch.Tensor] = None, db: Optional[torch.Tensor] = None,
                        accumulate: bool = False) -> GsLinearGrads:
    """Descriptor of the gradients of a linear_struct: dy in y's layout; dx
    [m][k] of x's type, dw [n][k] of float32 or x's type, db [n] float32, each
    optional; accumulate adds to dw and db.  dy is of y's type; a descriptor
    without y takes dy's."""
    rows, cols = (a.n, a.m) if a.planes else (a.m, a.n)
    dy_dtype = _dtype(dy)
    if a.y and a.y_dtype != dy_dtype:
        raise ValueError(f"dy: expected y's type, got {dy.dtype}")
    a.y_dtype = dy_dtype
    own, dev = _BY_CODE[a.dtype], dy.device if a.device is None else a.device
    g = GsLinearGrads(*_rows(dy, rows, cols, "dy", None, dev), *_rows(dx, a.m, a.k, "dx", (own,), dev),
                      *_rows(dw, a.n, a.k, "dw", (own, torch.float32), dev),
                      GS_DTYPE_F32 if dw is None else _dtype(dw), 1 if accumulate else 0,
                      _vector(db, a.n, "db", dev))
    g.dy_dtype = dy_dtype
    return g


def _for_dy(a: GsLinear, g: GsLinearGrads) -> GsLinear:
    """The descriptor with dy's type, which another dy may have changed since."""
    if g.dy_dtype in (None, a.y_dtype):
        return a
    b = GsLinear.from_buffer_copy(a)
    b.y_dtype = g.dy_dtype
    return b


def linear_bwd_workspace_bytes(a: GsLinear, g: GsLinearGrads) -> int:
    return int(lib().gs_linear_bwd_workspace_bytes(C.byref(_for_dy(a, g)), C.byref(g)))


def linear_bwd(a: GsLinear, g: GsLinearGrads, workspace: Optional[torch.Tensor] = None, stream=None):
    """gs_linear_bwd of a linear_struct and its linear_grads_struct."""
    _check(lib().gs_linear_bwd(C.byref(_for_dy(a, g)), C.byref(g), _ptr(workspace), _nbytes(workspace),
                               _stream_for(a.device, workspace, stream)), "gs_linear_bwd")


def muon_struct(grad: torch.Tensor, out: Optional[torch.Tensor] = None, momentum: Optional[torch.Tensor] = None,
                weight: Optional[torch.Tensor] = None, momentum_out: Optional[torch.Tensor] = None,
                weight_out: Optional[torch.Tensor] = None, lr: float = 0.02, beta: float = 0.95,
                weight_decay: float = 0.0, scale: float = 1.0, nesterov: bool = True, steps: int = 5,
                coeffs: Sequence[float] = (3.4445, -4.7750, 2.0315), eps: float = 1e-7) -> GsMuon:
    """Descriptor of gs_orthogonalize (grad and out) and gs_muon_step (grad,
    momentum, weight; momentum_out and weight_out default to updating in
    place): contiguous [rows][cols] or [batch][rows][cols] arrays, momentum
    float32, the others float32, float16 or bfloat16."""
    shape = grad.shape
    if len(shape) not in (2, 3):
        raise ValueError("grad: expected [rows][cols] or [batch][rows][cols]")
    _int32(*shape)
    momentum_out = momentum if momentum_out is None else momentum_out
    weight_out = weight if weight_out is None else weight_out
    for t, what in ((grad, "grad"), (out, "out"), (momentum, "momentum"), (weight, "weight"),
                    (momentum_out, "momentum_out"), (weight_out, "weight_out")):
        if t is not None and (t.shape != shape or not t.is_contiguous() or t.device != grad.device):
            raise ValueError(f"{what}: arrays must be contiguous, of one shape and on one device")
    for t, what in ((momentum, "momentum"), (momentum_out, "momentum_out")):
        if t is not None and t.dtype != torch.float32:
            raise ValueError(f"{what}: expected float32")
    results = [t for t in (weight, weight_out, out) if t is not None] or [grad]
    to = results[0]
    if any(t.dtype != to.dtype for t in results):
        raise ValueError("weight, weight_out, out: expected one type")
    a = GsMuon(shape[0] if len(shape) == 3 else 1, shape[-2], shape[-1], _dtype(grad), _dtype(to), steps, *coeffs, eps,
               lr, beta, weight_decay, scale, 1 if nesterov else 0, _ptr(grad), _ptr(out), _ptr(momentum),
               _ptr(momentum_out), _ptr(weight), _ptr(weight_out))
    a.device = grad.device
    return a


def muon_workspace_bytes(a: GsMuon) -> int:
    return int(lib().gs_muon_workspace_bytes(C.byref(a)))


def orthogonalize(a: GsMuon, workspace: torch.Tensor, stream=None):
    """gs_orthogonalize: a's out receives the orthogonalised grad."""
    _check(lib().gs_orthogonalize(C.byref(a), _ptr(workspace), _nbytes(workspace), _stream_for(a.device, workspace, stream)),
           "gs_orthogonalize")


def muon_step(a: GsMuon, workspace: torch.Tensor, stream=None):
    """gs_muon_step: momentum, orthogonalised update and weight decay."""
    _check(lib().gs_muon_step(C.byref(a), _ptr(workspace), _nbytes(workspace), _stream_for(a.device, workspace, stream)),
           "gs_muon_step")


# ---- tokens that read an encoder's states ----------------------------------
def _heads(t: Optional[torch.Tensor], shape, what: str, like: Optional[torch.Tensor] = None):
    """(address, strides of batch, row and head) of a [batch][rows][heads][d]
    tensor whose d is contiguous."""
    if t is None:
        return None, 0, 0, 0
    if t.shape != shape:
        raise ValueError(f"{what}: expected {list(shape)}, got {list(t.shape)}")
    if like is not None and (t.dtype is not like.dtype or t.device != like.device):
        raise ValueError(f"{what}: expected {like.dtype} on {like.device}, got {t.dtype} on {t.device}")
    sb, sr, sh, sd = t.stride()
    if sd != 1 and shape[3] > 1:
        raise ValueError(f"{what}: the last dimension must be contiguous (strides {t.stride()})")
    return t.data_ptr(), sb, sr, sh


def attention_struct(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
                     lse: Optional[torch.Tensor] = None, kv_lengths: Optional[torch.Tensor] = None,
                     kv_mask: Optional[torch.Tensor] = None, scale: Optional[float] = None) -> GsAttention:
    """Descriptor of cross attention: q and out [batch][nq][heads][d], k and v
    [batch][nk][kv_heads][d] of one type (float32, float16 or bfloat16; views of
    any strides but for d), lse [batch][heads][nq] float32 for the backward,
    kv_lengths [batch] int32, kv_mask [batch][nk] uint8 or bool (0: not
    attended), scale d^-1/2 unless given."""
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q, k: expected [batch][rows][heads][d]")
    (b, nq, h, d), (_, nk, kv, _) = q.shape, k.shape
    _int32(b, nq, h, d, nk, kv)
    dev, states = q.device, (b, nk, kv, d)
    if kv_lengths is not None and (kv_lengths.dtype is not torch.int32 or kv_lengths.shape != (b,) or not kv_lengths.is_contiguous()
                                   or kv_lengths.device != dev):
        raise ValueError(f"kv_lengths: expected {b} contiguous int32 values on the others' device")
    mask, stride = None, 0
    if kv_mask is not None:
        if kv_mask.dtype not in (torch.uint8, torch.bool) or kv_mask.shape != (b, nk) or kv_mask.device != dev or (nk > 1 and kv_mask.stride(1) != 1):
            raise ValueError(f"kv_mask: expected uint8 or bool [{b}][{nk}] with contiguous rows on the others' device")
        mask, stride = kv_mask.data_ptr(), kv_mask.stride(0)
    if lse is not None and lse.shape != (b, h, nq):
        raise ValueError(f"lse: expected [{b}][{h}][{nq}], got {list(lse.shape)}")
    a = GsAttention(b, h, kv, nq, nk, d, _dtype(q), d ** -0.5 if scale is None else scale, *_heads(q, q.shape, "q"),
                    *_heads(k, states, "k", q), *_heads(v, states, "v", q), *_heads(out, q.shape, "out", q),
                    _vector(lse, b * h * nq, "lse", dev), None if kv_lengths is None else kv_lengths.data_ptr(), mask, stride)
    a.device = dev
    return a


def attention_fwd_workspace_bytes(a: GsAttention) -> int:
    return int(lib().gs_attention_fwd_workspace_bytes(C.byref(a)))


def attention_fwd(a: GsAttention, workspace: Optional[torch.Tensor] = None, stream=None):
    """gs_attention_fwd of an attention_struct; the tensors it was made from
    must be alive."""
    _check(lib().gs_attention_fwd(C.byref(a), _ptr(workspace), _nbytes(workspace), _stream_for(a.device, workspace, stream)),
           "gs_attention_fwd")


def attention_grads_struct(a: GsAttention, dout: torch.Tensor, dq: Optional[torch.Tensor] = None,
                           dk: Optional[torch.Tensor] = None, dv: Optional[torch.Tensor] = None) -> GsAttentionGrads:
    """Descriptor of the gradients of an attention_struct (whose out and lse the
    forward has written): dout of out's shape and type, and any of dq, dk, dv of
    q's, k's and v's shapes and type."""
    if dout.dtype is not _BY_CODE[a.dtype] or (a.device is not None and dout.device != a.device):
        raise ValueError(f"dout: expected {_BY_CODE[a.dtype]} on {a.device}, got {dout.dtype} on {dout.device}")
    rows, states = (a.batch, a.nq, a.heads, a.d), (a.batch, a.nk, a.kv_heads, a.d)
    return GsAttentionGrads(*_heads(dout, rows, "dout"), *_heads(dq, rows, "dq", dout), *_heads(dk, states, "dk", dout),
                            *_heads(dv, states, "dv", dout))


def attention_bwd_workspace_bytes(a: GsAttention, g: GsAttentionGrads) -> int:
    return int(lib().gs_attention_bwd_workspace_bytes(C.byref(a), C.byref(g)))


def attention_bwd(a: GsAttention, g: GsAttentionGrads, workspace: Optional[torch.Tensor] = None, stream=None):
    """gs_attention_bwd of an attention_struct and its attention_grads_struct."""
    _check(lib().gs_attention_bwd(C.byref(a), C.byref(g), _ptr(workspace), _nbytes(workspace),
                                  _stream_for(a.device, workspace, stream)), "gs_attention_bwd")


def _maps(t: Optional[torch.Tensor], shape, what: str, dtypes=None, device=None):
    """(address, strides of image and pixel) of a [n][p][c] tensor whose c is
    contiguous."""
    if t is None:
        return None, 0, 0
    if t.shape != shape:
        raise ValueError(f"{what}: expected {list(shape)}, got {list(t.shape)}")
    if (dtypes is not None and t.dtype not in dtypes) or (device is not None and t.device != device):
        raise ValueError(f"{what}: unexpected {t.dtype} on {t.device}")
    image, pixel, step = t.stride()
    if step != 1 and shape[2] > 1:
        raise ValueError(f"{what}: the last dimension must be contiguous (strides {t.stride()})")
    return t.data_ptr(), image, pixel


def group_norm_fwd_workspace_bytes(n: int, p: int, c: int, groups: int) -> int:
    _int32(c, groups)
    return int(lib().gs_group_norm_fwd_workspace_bytes(n, p, c, groups))


def group_norm_fwd(x: torch.Tensor, y: torch.Tensor, groups: int, gamma: Optional[torch.Tensor] = None,
                   beta: Optional[torch.Tensor] = None, act: str = "none", mean: Optional[torch.Tensor] = None,
                   rstd: Optional[torch.Tensor] = None, kept: Optional[torch.Tensor] = None,
                   kept_scales: Optional[torch.Tensor] = None, eps: float = 1e-5,
                   workspace: Optional[torch.Tensor] = None, stream=None):
    """gs_group_norm_fwd over x [n][p][c] (images, pixels, channels; float32,
    float16 or bfloat16): y = act(gamma h + beta) of x's type.  mean and rstd
    [n][groups] are kept for the backward, and x itself in 8-bit blocks where
    kept [n][p][c] (float8_e4m3fn) and kept_scales [n][p][c / 32] (uint8 or
    float8_e8m0fnu) are given."""
    if x.dim() != 3:
        raise ValueError("x: expected [n][p][c]")
    n, p, c = x.shape
    _int32(n, c, groups)
    dev = x.device
    a = GsGroupNorm(n, c, groups, _dtype(x), GS_ACT[act], eps, p, *_maps(x, x.shape, "x"), _vector(gamma, c, "gamma", dev),
                    _vector(beta, c, "beta", dev), *_maps(y, x.shape, "y", (x.dtype,), dev),
                    _vector(mean, n * groups, "mean", dev), _vector(rstd, n * groups, "rstd", dev),
                    *_maps(kept, x.shape, "kept", (torch.float8_e4m3fn,), dev),
                    *_maps(kept_scales, (n, p, c // 32), "kept_scales", _SCALES, dev))
    _check(lib().gs_group_norm_fwd(C.byref(a), _ptr(workspace), _nbytes(workspace), _stream_for(dev, workspace, stream)),
           "gs_group_norm_fwd")


def group_norm_bwd_workspace_bytes(n: int, p: int, c: int, groups: int) -> int:
    _int32(c, groups)
    return int(lib().gs_group_norm_bwd_workspace_bytes(n, p, c, groups))


def group_norm_bwd(x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor, dy: torch.Tensor, dx: torch.Tensor, groups: int,
                   gamma: Optional[torch.Tensor] = None, beta: Optional[torch.Tensor] = None, act: str = "none",
                   dgamma: Optional[torch.Tensor] = None, dbeta: Optional[torch.Tensor] = None,
                   x_scales: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                   accumulate: bool = False, stream=None):
    """gs_group_norm_bwd: from x of dy's type, or the checkpoint (kept and, as
    x_scales, kept_scales) in its place, and the kept mean and rstd, the gradient
    dx and, if given, dgamma and dbeta [c]; accumulate adds to these two."""
    if dy.dim() != 3:
        raise ValueError("dy: expected [n][p][c]")
    n, p, c = dy.shape
    _int32(n, c, groups)
    dev, own = dy.device, (dy.dtype,)
    block = x.dtype is torch.float8_e4m3fn
    if block != (x_scales is not None):
        raise ValueError("x_scales: expected with an 8-bit x alone")
    a = GsGroupNormGrads(n, c, groups, _dtype(dy), _dtype(x), GS_ACT[act], 1 if accumulate else 0, p,
                         *_maps(x, dy.shape, "x", (dy.dtype, torch.float8_e4m3fn), dev),
                         *_maps(x_scales, (n, p, c // 32), "x_scales", _SCALES, dev), _vector(mean, n * groups, "mean", dev),
                         _vector(rstd, n * groups, "rstd", dev), _vector(gamma, c, "gamma", dev), _vector(beta, c, "beta", dev),
                         *_maps(dy, dy.shape, "dy"), *_maps(dx, dy.shape, "dx", own, dev), _vector(dgamma, c, "dgamma", dev),
                         _vector(dbeta, c, "dbeta", dev))
    _check(lib().gs_group_norm_bwd(C.byref(a), _ptr(workspace), _nbytes(workspace), _stream_for(dev, workspace, stream)),
           "gs_group_norm_bwd")


# ---- buffers for one view ---------------------------------------------------
class ViewBuffers:
    """Device buffers for rendering one camera with a fixed key capacity."""

    def __init__(self, n: int, cam, k_capacity: int, device="cuda", with_keys: bool = False,
                 with_backward: bool = True):
        self.n = n
        self.cam = cam
        self.camc = camera_struct(cam)
        self.n_tiles = ((cam.width + 15) // 16) * ((cam.height + 15) // 16)
        self.k_capacity = int(k_capacity)
        kc = max(self.k_capacity, 1)
        self.splats = torch.empty((max(n, 1), SPLAT_FLOATS), dtype=torch.float32, device=device)
        self.vals = torch.empty(kc, dtype=torch.int32, device=device)
        self.keys = torch.empty(kc, dtype=torch.int64, device=device) if with_keys else None
        self.ranges = torch.empty((self.n_tiles, 2), dtype=torch.int32, device=device)
        self.k_total = torch.zeros(1, dtype=torch.int64, device=device)
        wsb = bin_sort_workspace_bytes(n, self.k_capacity, self.n_tiles)
        self.ws = torch.empty(wsb, dtype=torch.uint8, device=device)
        H, W = cam.height, cam.width
        self.image = torch.empty((3, H, W), dtype=torch.float32, device=device)
        self.final_T = torch.empty((H, W), dtype=torch.float32, device=device)
        self.n_contrib = torch.empty((H, W), dtype=torch.int32, device=device)
        self.schedule = torch.empty(schedule_words(W, H), dtype=torch.int32, device=device)
        self.bwd_index = (torch.empty(bwd_index_words(n, self.k_capacity), dtype=torch.int32, device=device)
                          if with_backward else None)
        # the sort's per-Gaussian inputs when the projection writes them
        # set by bin_sort_views: the lists hold only reached tiles (a hint
        # passed on to the blend kernels)
        self.reached = False
        self.depth_keys = torch.empty(max(n, 1), dtype=torch.int32, device=device)
        self.tile_rects = torch.empty(2 * max(n, 1), dtype=torch.int32, device=device)

    @property
    def bin_keys(self):
        return (self.depth_keys, self.tile_rects)

    def forward(self, gs: GsGaussians, bg=(0.0, 0.0, 0.0), stream=None):
        self.reached = False
        project(gs, self.camc, self.splats, stream)
        bin_sort(self.splats, self.n, self.camc, self.k_capacity, self.vals, self.ranges, self.schedule,
                 self.bwd_index, self.keys, self.k_total, self.ws, stream)
        render_fwd(self.splats, self.vals, self.ranges, self.schedule, self.camc, bg, self.image, self.final_T,
                   self.n_contrib, stream)

    def backward_workspace(self, device="cuda"):
        return torch.empty(render_bwd_workspace_bytes(self.n, self.k_capacity), dtype=torch.uint8, device=device)

    def backward_screen(self, dL_dimage, g2, workspace, bg=(0.0, 0.0, 0.0), stream=None):
        """Screen-space backward of this view into g2 [n][9] (for project_bwd)."""
        render_bwd_screen(self.camc, self.n, self.splats, self.vals, self.ranges, self.schedule, self.bwd_index,
                          self.k_capacity, bg, self.final_T, self.n_contrib, dL_dimage, g2, workspace, stream)

    def backward(self, gs: GsGaussians, dL_dimage, grads, workspace, bg=(0.0, 0.0, 0.0), stream=None):
        render_bwd(gs, self.camc, self.splats, self.vals, self.ranges, self.schedule, self.bwd_index,
                   self.k_capacity, bg, self.final_T, self.n_contrib, dL_dimage, grads, workspace, stream)
