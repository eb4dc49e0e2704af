"""ctypes binding of libdcn_b200.so (argument marshalling only).

Every function here checks devices, dtypes, shapes and contiguity, allocates
outputs with torch when the caller passes none, and forwards raw device
pointers plus torch's current CUDA stream to the C ABI declared in
include/dcn_b200.h.  All arithmetic runs in the library's CUDA kernels; there
is no CPU path.  If the shared library is missing the first call raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading
from typing import NamedTuple, Optional, Sequence, Tuple

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libdcn_b200.so")

DCN_OK, DCN_ERR_NULL, DCN_ERR_SHAPE, DCN_ERR_UNSUPPORTED, DCN_ERR_ALIGN, DCN_ERR_CUDA = range(6)
DCN_F32, DCN_F16, DCN_BF16 = 0, 1, 2
DCN_MASK_RAW, DCN_MASK_SOFTMAX = 0, 1
_DTYPE_CODE = {torch.float32: DCN_F32, torch.float16: DCN_F16, torch.bfloat16: DCN_BF16}

# Every entry point include/dcn_b200.h declares.
EXPORTS = ("dcn_core_output_hw", "dcn_core_forward", "dcn_core_backward", "deform_agg_forward",
           "deform_agg_backward", "dcn_status_string", "dcn_last_error_detail", "dcn_abi_version",
           "dcn_take_device_error", "deform_roi_pool_forward", "dcn_core_forward_proj",
           "dcn_selftest_bounded_wait", "dcn_deform_conv_forward", "dcn_probe_rate",
           "dcn_core_forward_proj_workspace_bytes", "dcn_core_forward_proj_noalloc",
           "dcn_add_rms_norm_forward", "dcn_add_rms_norm_backward", "dcn_add_rms_norm_backward_workspace_bytes",
           "dcn_add_rms_norm_backward_input",
           "dcn_grad_norm", "dcn_clip_grads", "dcn_grad_norm_workspace_bytes",
           "dcn_proj_adapters_forward", "dcn_proj_adapters_workspace_bytes", "dcn_proj_adapters_workspace_full_bytes")
ABI_VERSION = 2


class DcnParams(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "H", "W", "G", "C", "kh", "kw", "stride_h", "stride_w",
                                              "pad_h", "pad_w", "dil_h", "dil_w")] + \
               [("offset_scale", ctypes.c_float), ("mask_mode", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class DaggParams(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "num_cams", "num_scales", "num_rows", "num_anchors",
                                              "num_pts", "G", "C", "dtype")]


class DroiParams(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "H", "W", "C", "num_rois", "pooled_h", "pooled_w",
                                              "sampling")] + \
               [("spatial_scale", ctypes.c_float), ("gamma", ctypes.c_float), ("dtype", ctypes.c_int32)]


class DnormParams(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int32), ("eps", ctypes.c_float)] + \
               [(n, ctypes.c_int32) for n in ("dtype", "quant", "group")]


class DadaptParams(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64)] + \
               [(n, ctypes.c_int32) for n in ("cin", "cout", "rank", "num_adapters", "num_requests", "dtype")]


class DclipParams(ctypes.Structure):
    _fields_ = [("num_tensors", ctypes.c_int32), ("kind", ctypes.c_int32), ("max_norm", ctypes.c_float),
                ("eps", ctypes.c_float)]


class DcnError(RuntimeError):
    def __init__(self, status: int, detail: str):
        super().__init__(detail)
        self.status = status


_lock = threading.Lock()
_lib = None


def _declare(lib):
    vp, st = ctypes.c_void_p, ctypes.c_int
    P = ctypes.POINTER(DcnParams)
    A = ctypes.POINTER(DaggParams)
    i32p = ctypes.POINTER(ctypes.c_int32)
    lib.dcn_core_output_hw.argtypes = [P, i32p, i32p]
    lib.dcn_core_forward.argtypes = [P, vp, vp, vp, vp, vp]
    lib.dcn_core_backward.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.deform_agg_forward.argtypes = [A, vp, vp, vp, vp, vp, vp, vp]
    lib.deform_agg_backward.argtypes = [A, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    for f in ("dcn_core_output_hw", "dcn_core_forward", "dcn_core_backward", "deform_agg_forward",
              "deform_agg_backward"):
        getattr(lib, f).restype = st
    lib.dcn_status_string.argtypes = [st]
    lib.dcn_status_string.restype = ctypes.c_char_p
    lib.dcn_last_error_detail.argtypes = []
    lib.dcn_last_error_detail.restype = ctypes.c_char_p
    lib.dcn_abi_version.argtypes = []
    lib.dcn_abi_version.restype = ctypes.c_int32
    lib.deform_roi_pool_forward.argtypes = [ctypes.POINTER(DroiParams), vp, vp, vp, vp, vp]
    lib.deform_roi_pool_forward.restype = st
    lib.dcn_core_forward_proj.argtypes = [P, ctypes.c_int32, vp, vp, vp, vp, vp, vp, vp, ctypes.c_int64, vp]
    lib.dcn_core_forward_proj.restype = st
    lib.dcn_core_forward_proj_workspace_bytes.argtypes = [P]
    lib.dcn_core_forward_proj_workspace_bytes.restype = ctypes.c_int64
    lib.dcn_core_forward_proj_noalloc.argtypes = [P, ctypes.c_int32, vp, vp, vp, vp, vp, vp, vp]
    lib.dcn_core_forward_proj_noalloc.restype = st
    lib.dcn_deform_conv_forward.argtypes = [P, ctypes.c_int32, vp, vp, vp, vp, vp, vp, vp]
    lib.dcn_deform_conv_forward.restype = st
    lib.dcn_selftest_bounded_wait.argtypes = [ctypes.c_int32, vp]
    lib.dcn_selftest_bounded_wait.restype = st
    lib.dcn_take_device_error.argtypes = []
    lib.dcn_take_device_error.restype = ctypes.c_int32
    lib.dcn_probe_rate.argtypes = [ctypes.c_int32, ctypes.c_int32, vp, ctypes.c_int64,
                                   ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_char_p), vp]
    lib.dcn_probe_rate.restype = st
    N, L = ctypes.POINTER(DnormParams), ctypes.POINTER(DclipParams)
    lib.dcn_add_rms_norm_forward.argtypes = [N, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.dcn_add_rms_norm_backward.argtypes = [N, vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_int64, vp]
    lib.dcn_add_rms_norm_backward_input.argtypes = [N, vp, vp, vp, vp, vp, vp, vp]
    lib.dcn_add_rms_norm_backward_workspace_bytes.argtypes = [N]
    lib.dcn_grad_norm.argtypes = [L, vp, vp, vp, vp, vp, ctypes.c_int64, vp]
    lib.dcn_clip_grads.argtypes = [L, vp, vp, vp, vp, vp, vp, vp, ctypes.c_int64, vp]
    lib.dcn_grad_norm_workspace_bytes.argtypes = [ctypes.c_int32]
    for f in ("dcn_add_rms_norm_forward", "dcn_add_rms_norm_backward", "dcn_add_rms_norm_backward_input",
              "dcn_grad_norm", "dcn_clip_grads"):
        getattr(lib, f).restype = st
    for f in ("dcn_add_rms_norm_backward_workspace_bytes", "dcn_grad_norm_workspace_bytes"):
        getattr(lib, f).restype = ctypes.c_int64
    R = ctypes.POINTER(DadaptParams)
    lib.dcn_proj_adapters_forward.argtypes = [R, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_int64, vp]
    lib.dcn_proj_adapters_forward.restype = st
    for f in ("dcn_proj_adapters_workspace_bytes", "dcn_proj_adapters_workspace_full_bytes"):
        getattr(lib, f).argtypes = [R]
        getattr(lib, f).restype = ctypes.c_int64
    return lib


def lib(path: Optional[str] = None):
    """The loaded library (declared argtypes).  Raises if it is not built."""
    global _lib
    if path is not None:
        return _declare(ctypes.CDLL(path))
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                                   "`python -m deformable_convolution_sampling_dcn_b200.build`")
            l = _declare(ctypes.CDLL(LIB_PATH))
            if l.dcn_abi_version() != ABI_VERSION:
                raise RuntimeError("libdcn_b200.so ABI version mismatch; rebuild it")
            _lib = l
    return _lib


def check(status: int) -> None:
    if status != DCN_OK:
        L = lib()
        raise DcnError(status, f"{L.dcn_status_string(status).decode()}: {L.dcn_last_error_detail().decode()}")


def _pair(v) -> Tuple[int, int]:
    if isinstance(v, (tuple, list)):
        return int(v[0]), int(v[1])
    return int(v), int(v)


def _cuda_tensor(name, t: torch.Tensor, dtype=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    return t


def _stream(t: torch.Tensor) -> int:
    return torch.cuda.current_stream(t.device).cuda_stream


def core_params(x: torch.Tensor, G: int, kernel=(3, 3), stride=(1, 1), pad=(1, 1), dil=(1, 1),
                offset_scale: float = 1.0, softmax: bool = False) -> DcnParams:
    if x.dtype not in _DTYPE_CODE:
        raise TypeError(f"unsupported dtype {x.dtype}")
    B, H, W, GC = x.shape
    if GC % G:
        raise ValueError(f"channels {GC} not divisible by G={G}")
    kh, kw = _pair(kernel)
    sh, sw = _pair(stride)
    ph, pw = _pair(pad)
    dh, dw = _pair(dil)
    return DcnParams(B, H, W, G, GC // G, kh, kw, sh, sw, ph, pw, dh, dw, float(offset_scale),
                     DCN_MASK_SOFTMAX if softmax else DCN_MASK_RAW, _DTYPE_CODE[x.dtype])


def take_device_error() -> int:
    """Read and clear the device error word (0 = no bounded wait ran out)."""
    return int(lib().dcn_take_device_error())


PROBES = ("lds128", "chunk_f32_ffma2", "ffma", "ffma2", "chunk_f16_ffma", "chunk_f16_ffma2", "chunk_bf16_ffma2",
          "chunk_f16_mixed", "ldg128_l1", "gather4", "gather8", "gather8_ffma", "alu", "ldg256_l1",
          "atoms_f32")


def probe_rate(name: str, reps: int, device=None) -> Tuple[float, str]:
    """Run one on-chip rate probe; returns (units per SM per clock, unit)."""
    dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
    buf = torch.zeros(65536, dtype=torch.uint8, device=dev)
    units = ctypes.c_double()
    unit = ctypes.c_char_p()
    check(lib().dcn_probe_rate(PROBES.index(name), int(reps), buf.data_ptr(), buf.numel(), ctypes.byref(units),
                               ctypes.byref(unit), torch.cuda.current_stream(dev).cuda_stream))
    torch.cuda.synchronize(dev)
    words = buf[:16].view(torch.int64).cpu().tolist()
    return units.value * words[1] / words[0], unit.value.decode()


def selftest_bounded_wait(limit_us: int = 2000, device=None) -> None:
    """Enqueue the bounded-wait self-test on the current stream (see dcn_b200.h)."""
    check(lib().dcn_selftest_bounded_wait(int(limit_us), torch.cuda.current_stream(device).cuda_stream))


def dcn_core_output_hw(p: DcnParams) -> Tuple[int, int]:
    ho, wo = ctypes.c_int32(), ctypes.c_int32()
    check(lib().dcn_core_output_hw(ctypes.byref(p), ctypes.byref(ho), ctypes.byref(wo)))
    return ho.value, wo.value


def dcn_core_forward(x: torch.Tensor, offset: torch.Tensor, mask: torch.Tensor, *, group: int,
                     kernel=(3, 3), stride=(1, 1), pad=(1, 1), dil=(1, 1), offset_scale: float = 1.0,
                     softmax: bool = False, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out [B,Ho,Wo,G*C] = sum_k m_k bilinear(x, p_k) per (pixel, group); see dcn_b200.h."""
    _cuda_tensor("x", x)
    p = core_params(x, group, kernel, stride, pad, dil, offset_scale, softmax)
    Ho, Wo = dcn_core_output_hw(p)
    K = p.kh * p.kw
    _cuda_tensor("offset", offset, x.dtype)
    _cuda_tensor("mask", mask, x.dtype)
    if tuple(offset.shape) != (p.B, Ho, Wo, p.G, K, 2):
        raise ValueError(f"offset shape {tuple(offset.shape)} != {(p.B, Ho, Wo, p.G, K, 2)}")
    if tuple(mask.shape) != (p.B, Ho, Wo, p.G, K):
        raise ValueError(f"mask shape {tuple(mask.shape)} != {(p.B, Ho, Wo, p.G, K)}")
    if out is None:
        out = torch.empty((p.B, Ho, Wo, p.G * p.C), dtype=x.dtype, device=x.device)
    else:
        _cuda_tensor("out", out, x.dtype)
        if tuple(out.shape) != (p.B, Ho, Wo, p.G * p.C):
            raise ValueError("out has the wrong shape")
    check(lib().dcn_core_forward(ctypes.byref(p), x.data_ptr(), offset.data_ptr(), mask.data_ptr(),
                                 out.data_ptr(), _stream(x)))
    return out


def dcn_core_forward_proj(x: torch.Tensor, offset: torch.Tensor, mask: torch.Tensor, weight: torch.Tensor,
                          bias: Optional[torch.Tensor] = None, *, group: int, kernel=(3, 3), stride=(1, 1),
                          pad=(1, 1), dil=(1, 1), offset_scale: float = 1.0, softmax: bool = False,
                          out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                          fused: bool = False) -> torch.Tensor:
    """out [B,Ho,Wo,Cout] = bias + core(x, offset, mask) . weight[Cout, G*C]^T; see dcn_b200.h.

    By default the core goes through a workspace (`workspace`, or one torch
    allocates here) and a tensor-core GEMM projects it; fused=True runs the one
    fused kernel with no workspace."""
    _cuda_tensor("x", x)
    p = core_params(x, group, kernel, stride, pad, dil, offset_scale, softmax)
    Ho, Wo = dcn_core_output_hw(p)
    K = p.kh * p.kw
    _cuda_tensor("offset", offset, x.dtype)
    _cuda_tensor("mask", mask, x.dtype)
    _cuda_tensor("weight", weight, x.dtype)
    if tuple(offset.shape) != (p.B, Ho, Wo, p.G, K, 2):
        raise ValueError(f"offset shape {tuple(offset.shape)} != {(p.B, Ho, Wo, p.G, K, 2)}")
    if tuple(mask.shape) != (p.B, Ho, Wo, p.G, K):
        raise ValueError(f"mask shape {tuple(mask.shape)} != {(p.B, Ho, Wo, p.G, K)}")
    if weight.dim() != 2 or weight.shape[1] != p.G * p.C:
        raise ValueError(f"weight shape {tuple(weight.shape)} != (Cout, {p.G * p.C})")
    cout = int(weight.shape[0])
    if bias is not None:
        _cuda_tensor("bias", bias, x.dtype)
        if tuple(bias.shape) != (cout,):
            raise ValueError(f"bias shape {tuple(bias.shape)} != ({cout},)")
    if out is None:
        out = torch.empty((p.B, Ho, Wo, cout), dtype=x.dtype, device=x.device)
    else:
        _cuda_tensor("out", out, x.dtype)
        if tuple(out.shape) != (p.B, Ho, Wo, cout):
            raise ValueError("out has the wrong shape")
    ws_ptr, ws_bytes = None, 0
    if not fused:
        need = int(lib().dcn_core_forward_proj_workspace_bytes(ctypes.byref(p)))
        if workspace is None:
            workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=x.device)
        else:
            _cuda_tensor("workspace", workspace)
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    check(lib().dcn_core_forward_proj(ctypes.byref(p), cout, x.data_ptr(), offset.data_ptr(), mask.data_ptr(),
                                      weight.data_ptr(), None if bias is None else bias.data_ptr(),
                                      out.data_ptr(), ws_ptr, ws_bytes, _stream(x)))
    return out


def dcn_deform_conv_forward(x: torch.Tensor, offset: torch.Tensor, mask: torch.Tensor, weight: torch.Tensor,
                            bias: Optional[torch.Tensor] = None, *, group: int, kernel=(3, 3), stride=(1, 1),
                            pad=(1, 1), dil=(1, 1), offset_scale: float = 1.0, softmax: bool = False,
                            out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out [B,Ho,Wo,Cout] = bias + sum_k weight[:, k, :] . (m_k x(p_k)): modulated deformable convolution
    with weight [Cout, K, G*C] in one kernel; see dcn_b200.h."""
    _cuda_tensor("x", x)
    p = core_params(x, group, kernel, stride, pad, dil, offset_scale, softmax)
    Ho, Wo = dcn_core_output_hw(p)
    K = p.kh * p.kw
    _cuda_tensor("offset", offset, x.dtype)
    _cuda_tensor("mask", mask, x.dtype)
    _cuda_tensor("weight", weight, x.dtype)
    if tuple(offset.shape) != (p.B, Ho, Wo, p.G, K, 2):
        raise ValueError(f"offset shape {tuple(offset.shape)} != {(p.B, Ho, Wo, p.G, K, 2)}")
    if tuple(mask.shape) != (p.B, Ho, Wo, p.G, K):
        raise ValueError(f"mask shape {tuple(mask.shape)} != {(p.B, Ho, Wo, p.G, K)}")
    if weight.dim() != 3 or tuple(weight.shape[1:]) != (K, p.G * p.C):
        raise ValueError(f"weight shape {tuple(weight.shape)} != (Cout, {K}, {p.G * p.C})")
    cout = int(weight.shape[0])
    if bias is not None:
        _cuda_tensor("bias", bias, x.dtype)
        if tuple(bias.shape) != (cout,):
            raise ValueError(f"bias shape {tuple(bias.shape)} != ({cout},)")
    if out is None:
        out = torch.empty((p.B, Ho, Wo, cout), dtype=x.dtype, device=x.device)
    else:
        _cuda_tensor("out", out, x.dtype)
        if tuple(out.shape) != (p.B, Ho, Wo, cout):
            raise ValueError("out has the wrong shape")
    check(lib().dcn_deform_conv_forward(ctypes.byref(p), cout, x.data_ptr(), offset.data_ptr(), mask.data_ptr(),
                                        weight.data_ptr(), None if bias is None else bias.data_ptr(),
                                        out.data_ptr(), _stream(x)))
    return out


def dcn_core_backward(x, offset, mask, grad_out, *, group: int, kernel=(3, 3), stride=(1, 1), pad=(1, 1),
                      dil=(1, 1), offset_scale: float = 1.0, softmax: bool = False, grad_x=None,
                      grad_offset=None, grad_mask=None):
    """(grad_x, grad_offset, grad_mask) of <grad_out, dcn_core_forward(...)>; see dcn_b200.h."""
    _cuda_tensor("x", x)
    p = core_params(x, group, kernel, stride, pad, dil, offset_scale, softmax)
    Ho, Wo = dcn_core_output_hw(p)
    K = p.kh * p.kw
    for n, t in (("offset", offset), ("mask", mask), ("grad_out", grad_out)):
        _cuda_tensor(n, t, x.dtype)
    if tuple(offset.shape) != (p.B, Ho, Wo, p.G, K, 2) or tuple(mask.shape) != (p.B, Ho, Wo, p.G, K):
        raise ValueError("offset/mask shape mismatch")
    if tuple(grad_out.shape) != (p.B, Ho, Wo, p.G * p.C):
        raise ValueError("grad_out shape mismatch")
    grad_x = torch.empty_like(x) if grad_x is None else _cuda_tensor("grad_x", grad_x, x.dtype)
    grad_offset = torch.empty_like(offset) if grad_offset is None else _cuda_tensor("grad_offset", grad_offset, x.dtype)
    grad_mask = torch.empty_like(mask) if grad_mask is None else _cuda_tensor("grad_mask", grad_mask, x.dtype)
    if grad_x.shape != x.shape or grad_offset.shape != offset.shape or grad_mask.shape != mask.shape:
        raise ValueError("gradient buffer shape mismatch")
    check(lib().dcn_core_backward(ctypes.byref(p), x.data_ptr(), offset.data_ptr(), mask.data_ptr(),
                                  grad_out.data_ptr(), grad_x.data_ptr(), grad_offset.data_ptr(),
                                  grad_mask.data_ptr(), _stream(x)))
    return grad_x, grad_offset, grad_mask


def agg_params(feat: torch.Tensor, weights: torch.Tensor) -> DaggParams:
    if feat.dtype not in _DTYPE_CODE:
        raise TypeError(f"unsupported dtype {feat.dtype}")
    B, rows, GC = feat.shape
    Bw, A, P, cams, S, G = weights.shape
    if Bw != B or GC % G:
        raise ValueError("feat/weights shape mismatch")
    return DaggParams(B, cams, S, rows, A, P, G, GC // G, _DTYPE_CODE[feat.dtype])


def _agg_inputs(feat, spatial_shape, scale_start_index, sampling_location, weights):
    _cuda_tensor("feat", feat)
    _cuda_tensor("weights", weights, feat.dtype)
    p = agg_params(feat, weights)
    _cuda_tensor("spatial_shape", spatial_shape, torch.int32)
    _cuda_tensor("scale_start_index", scale_start_index, torch.int32)
    _cuda_tensor("sampling_location", sampling_location, torch.float32)
    if tuple(spatial_shape.shape) != (p.num_cams, p.num_scales, 2):
        raise ValueError("spatial_shape must be [cams, scales, 2]")
    if tuple(scale_start_index.shape) != (p.num_cams, p.num_scales):
        raise ValueError("scale_start_index must be [cams, scales]")
    if tuple(sampling_location.shape) != (p.B, p.num_anchors, p.num_pts, p.num_cams, 2):
        raise ValueError("sampling_location must be [B, A, P, cams, 2]")
    return p


def deform_agg_forward(feat, spatial_shape, scale_start_index, sampling_location, weights, *, out=None):
    """out [B, A, G*C]: weighted multi-camera multi-scale bilinear aggregation; see dcn_b200.h."""
    p = _agg_inputs(feat, spatial_shape, scale_start_index, sampling_location, weights)
    if out is None:
        out = torch.empty((p.B, p.num_anchors, p.G * p.C), dtype=feat.dtype, device=feat.device)
    else:
        _cuda_tensor("out", out, feat.dtype)
    check(lib().deform_agg_forward(ctypes.byref(p), feat.data_ptr(), spatial_shape.data_ptr(),
                                   scale_start_index.data_ptr(), sampling_location.data_ptr(),
                                   weights.data_ptr(), out.data_ptr(), _stream(feat)))
    return out


def deform_agg_backward(feat, spatial_shape, scale_start_index, sampling_location, weights, grad_out, *,
                        grad_feat=None, grad_loc=None, grad_weights=None):
    """(grad_feat, grad_loc, grad_weights) of <grad_out, deform_agg_forward(...)>."""
    p = _agg_inputs(feat, spatial_shape, scale_start_index, sampling_location, weights)
    _cuda_tensor("grad_out", grad_out, feat.dtype)
    grad_feat = torch.empty_like(feat) if grad_feat is None else _cuda_tensor("grad_feat", grad_feat, feat.dtype)
    grad_loc = torch.empty_like(sampling_location) if grad_loc is None else \
        _cuda_tensor("grad_loc", grad_loc, torch.float32)
    grad_weights = torch.empty_like(weights) if grad_weights is None else \
        _cuda_tensor("grad_weights", grad_weights, feat.dtype)
    check(lib().deform_agg_backward(ctypes.byref(p), feat.data_ptr(), spatial_shape.data_ptr(),
                                    scale_start_index.data_ptr(), sampling_location.data_ptr(),
                                    weights.data_ptr(), grad_out.data_ptr(), grad_feat.data_ptr(),
                                    grad_loc.data_ptr(), grad_weights.data_ptr(), _stream(feat)))
    return grad_feat, grad_loc, grad_weights


def deform_roi_pool_forward(x, rois, offset, *, pooled=(7, 7), sampling: int = 2, spatial_scale: float = 1.0,
                            gamma: float = 0.1, out=None):
    """out [N, PH, PW, C]: deformable RoI pooling of x [B, H, W, C]; see dcn_b200.h."""
    _cuda_tensor("x", x)
    if x.dtype not in _DTYPE_CODE:
        raise TypeError(f"unsupported dtype {x.dtype}")
    _cuda_tensor("rois", rois, torch.float32)
    _cuda_tensor("offset", offset, torch.float32)
    B, H, W, C = x.shape
    PH, PW = _pair(pooled)
    N = rois.shape[0]
    if tuple(rois.shape) != (N, 5) or tuple(offset.shape) != (N, PH, PW, 2):
        raise ValueError("rois must be [N, 5] and offset [N, PH, PW, 2]")
    p = DroiParams(B, H, W, C, N, PH, PW, int(sampling), float(spatial_scale), float(gamma), _DTYPE_CODE[x.dtype])
    if out is None:
        out = torch.empty((N, PH, PW, C), dtype=x.dtype, device=x.device)
    else:
        _cuda_tensor("out", out, x.dtype)
    check(lib().deform_roi_pool_forward(ctypes.byref(p), x.data_ptr(), rois.data_ptr(), offset.data_ptr(),
                                        out.data_ptr(), _stream(x)))
    return out


_INT32_MAX = 2 ** 31 - 1  # sizes go to the library in 32 bits


def _launch(index: int, fn, *args) -> None:
    """fn(*args, stream) on CUDA device `index` and its current stream; raises on a non-OK status.

    The small calls of this section are host-bound (a launch takes 3 us), so the
    device and stream are read through torch's own C accessors: 0.2 us against
    2.5 us for torch.cuda.current_stream(device).cuda_stream."""
    if index == torch._C._cuda_getDevice():
        status = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if status != DCN_OK:
        check(status)


def _like(name: str, t: torch.Tensor, shape, dtype: torch.dtype, index: int) -> torch.Tensor:
    """Checks an argument that has to have this shape and type, on CUDA device `index`."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == index and t.shape == shape and \
            t.is_contiguous():
        return t
    _cuda_tensor(name, t, dtype)
    if t.shape != shape:
        raise ValueError(f"{name} shape {tuple(t.shape)} != {tuple(shape)}")
    raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")


def _rows(x: torch.Tensor) -> Tuple[int, int]:
    shape = x.shape
    if not shape or shape[-1] < 1:
        raise ValueError("x must be [..., cols] with at least one column")
    if shape[-1] > _INT32_MAX:
        raise ValueError(f"{shape[-1]} columns exceed 32 bits")
    return x.numel() // shape[-1], shape[-1]


def _workspace(t: torch.Tensor, index: int) -> Tuple[int, int]:
    """Address and bytes of a caller's workspace, which has to be on CUDA device `index`."""
    _cuda_tensor("workspace", t)
    if t.get_device() != index:
        raise ValueError(f"workspace is on {t.device}, expected cuda:{index}")
    return t.data_ptr(), t.numel() * t.element_size()


class AddRmsNorm(NamedTuple):
    """Outputs of dcn_add_rms_norm_forward; None where a call does not ask for one."""
    out: Optional[torch.Tensor]
    residual_out: Optional[torch.Tensor]
    out8: Optional[torch.Tensor]
    scale: Optional[torch.Tensor]
    rstd: Optional[torch.Tensor]


_QUANT = {None: (0, None), "e4m3": (1, torch.float8_e4m3fn), "int8": (2, torch.int8)}


def dcn_add_rms_norm_forward(x: torch.Tensor, residual: Optional[torch.Tensor] = None,
                             weight: Optional[torch.Tensor] = None, *, eps: float = 1e-6,
                             quant: Optional[str] = None, group: int = 0, keep_out: Optional[bool] = None,
                             save_rstd: bool = False, out=None, residual_out=None, out8=None, scale=None,
                             rstd=None) -> AddRmsNorm:
    """Residual addition and root-mean-square norm over the last dimension; see dcn_b200.h.

    quant "e4m3" or "int8" gives the output in 8 bits (out8, out8 * scale is the
    norm's output) with one fp32 scale per row, scale [..., 1], or per 128 columns
    (group=128), scale [..., ceil(cols / 128)].  `out` in the storage type is then
    left out unless keep_out=True or a buffer is given.  save_rstd=True also
    returns the statistic that the backward reads.  The buffers default to new
    tensors; residual_out and out may each be x or residual."""
    _cuda_tensor("x", x)
    dt, dev = x.dtype, x.get_device()
    if dt not in _DTYPE_CODE:
        raise TypeError(f"unsupported dtype {dt}")
    if quant not in _QUANT:
        raise ValueError(f"quant must be None, 'e4m3' or 'int8', not {quant!r}")
    code, dt8 = _QUANT[quant]
    rows, cols = _rows(x)
    shape = x.shape
    if residual is not None:
        _like("residual", residual, shape, dt, dev)
        residual_out = torch.empty_like(x) if residual_out is None else \
            _like("residual_out", residual_out, shape, dt, dev)
    elif residual_out is not None:
        raise ValueError("residual_out without a residual")
    if weight is not None:
        _like("weight", weight, (cols,), dt, dev)
    if code == 0:
        if keep_out is False:
            raise ValueError("keep_out=False without an 8-bit output")
        if out8 is not None or scale is not None or group:
            raise ValueError("out8, scale and group belong to an 8-bit output")
    else:
        if group not in (0, 128):
            raise ValueError("group must be 0 or 128")
        out8 = torch.empty_like(x, dtype=dt8) if out8 is None else _like("out8", out8, shape, dt8, dev)
        ss = shape[:-1] + ((cols + 127) // 128 if group else 1,)
        scale = x.new_empty(ss, dtype=torch.float32) if scale is None else _like("scale", scale, ss, torch.float32, dev)
    if code == 0 or keep_out or out is not None:
        out = torch.empty_like(x) if out is None else _like("out", out, shape, dt, dev)
        if residual_out is not None and rows and out.data_ptr() == residual_out.data_ptr():
            raise ValueError("out and residual_out are the same buffer")
    if rstd is not None:
        _like("rstd", rstd, shape[:-1], torch.float32, dev)
    elif save_rstd:
        rstd = x.new_empty(shape[:-1], dtype=torch.float32)
    p = DnormParams(rows, cols, eps, _DTYPE_CODE[dt], code, group)
    _launch(dev, lib().dcn_add_rms_norm_forward, ctypes.byref(p), x.data_ptr(),
            None if residual is None else residual.data_ptr(), None if weight is None else weight.data_ptr(),
            None if residual_out is None else residual_out.data_ptr(), None if out is None else out.data_ptr(),
            None if out8 is None else out8.data_ptr(), None if scale is None else scale.data_ptr(),
            None if rstd is None else rstd.data_ptr())
    return AddRmsNorm(out, residual_out, out8, scale, rstd)


@functools.lru_cache(maxsize=1024)
def _norm_backward_workspace_bytes(rows: int, cols: int, eps: float, code: int) -> int:
    """Workspace of a problem of these sizes (a function of them alone); 16 where they are refused."""
    return max(16, lib().dcn_add_rms_norm_backward_workspace_bytes(ctypes.byref(DnormParams(rows, cols, eps, code, 0, 0))))


def dcn_add_rms_norm_backward(grad_out: torch.Tensor, h: torch.Tensor, rstd: torch.Tensor,
                              weight: Optional[torch.Tensor] = None, *,
                              grad_residual_out: Optional[torch.Tensor] = None, eps: float = 1e-6, grad_x=None,
                              grad_weight=None, workspace: Optional[torch.Tensor] = None,
                              need_grad_weight: bool = True):
    """(grad_x, grad_weight) of dcn_add_rms_norm_forward; see dcn_b200.h.

    h is the forward's residual_out (x without a residual), rstd what it saved;
    grad_x is the gradient of x and of the residual alike.  grad_weight is None
    without a weight, and with need_grad_weight=False (a weight that is not
    trained), which costs no workspace and no second kernel.  eps is part of rstd
    and only checked here."""
    _cuda_tensor("h", h)
    dt, dev, shape = h.dtype, h.get_device(), h.shape
    if dt not in _DTYPE_CODE:
        raise TypeError(f"unsupported dtype {dt}")
    rows, cols = _rows(h)
    _like("grad_out", grad_out, shape, dt, dev)
    _like("rstd", rstd, shape[:-1], torch.float32, dev)
    if grad_residual_out is not None:
        _like("grad_residual_out", grad_residual_out, shape, dt, dev)
    grad_x = torch.empty_like(h) if grad_x is None else _like("grad_x", grad_x, shape, dt, dev)
    p = DnormParams(rows, cols, eps, _DTYPE_CODE[dt], 0, 0)
    ws_ptr, ws_bytes = None, 0
    if weight is not None:
        _like("weight", weight, (cols,), dt, dev)
    if not need_grad_weight:
        if grad_weight is not None or workspace is not None:
            raise ValueError("grad_weight and workspace belong to need_grad_weight")
        _launch(dev, lib().dcn_add_rms_norm_backward_input, ctypes.byref(p), grad_out.data_ptr(), h.data_ptr(),
                rstd.data_ptr(), None if weight is None else weight.data_ptr(),
                None if grad_residual_out is None else grad_residual_out.data_ptr(), grad_x.data_ptr())
        return grad_x, None
    if weight is not None:
        grad_weight = torch.empty_like(weight) if grad_weight is None else \
            _like("grad_weight", grad_weight, (cols,), dt, dev)
        if workspace is None:
            ws_bytes = _norm_backward_workspace_bytes(rows, cols, eps, _DTYPE_CODE[dt])
            workspace = h.new_empty(ws_bytes, dtype=torch.uint8)
            ws_ptr = workspace.data_ptr()
        else:
            ws_ptr, ws_bytes = _workspace(workspace, dev)
    elif grad_weight is not None:
        raise ValueError("grad_weight without a weight")
    _launch(dev, lib().dcn_add_rms_norm_backward, ctypes.byref(p), grad_out.data_ptr(), h.data_ptr(),
            rstd.data_ptr(), None if weight is None else weight.data_ptr(),
            None if grad_residual_out is None else grad_residual_out.data_ptr(), grad_x.data_ptr(),
            None if grad_weight is None else grad_weight.data_ptr(), ws_ptr, ws_bytes)
    return grad_x, grad_weight


_DENSE = {4: (torch.contiguous_format, torch.channels_last), 5: (torch.contiguous_format, torch.channels_last_3d)}


def _dense_formats(t: torch.Tensor):
    """The memory formats in which t is dense: a convolution's weight may lie channels-last, and so its gradient."""
    if t.dim() not in _DENSE:
        return (torch.contiguous_format,) if t.is_contiguous() else ()
    return tuple(f for f in _DENSE[t.dim()] if t.is_contiguous(memory_format=f))


class GradList:
    """The table of gradient buffers that dcn_grad_norm and dcn_clip_grads work on.

    Made once where the buffers stay in place over a training run (both calls
    also take a plain list and make the table each time).  `out` gives a buffer
    of the same shape for each gradient, of any storage type, that receives the
    clipped values; without it clipping is in place.  Buffers are contiguous or
    channels-last, an `out` buffer in its gradient's way, and must not overlap.
    The list keeps its tensors alive; a tensor that is given other memory
    (resize_, set_) needs a new list."""

    def __init__(self, grads: Sequence[torch.Tensor], out: Optional[Sequence[torch.Tensor]] = None):
        self.grads = list(grads)
        self.out = None if out is None else list(out)
        n = len(self.grads)
        if self.out is not None and len(self.out) != n:
            raise ValueError(f"{len(self.out)} out buffers for {n} gradients")
        self.device = None  # index
        for t in self.grads + (self.out or []):
            if not isinstance(t, torch.Tensor):
                raise TypeError("gradients and out buffers must be torch.Tensors")
            if t.dtype not in _DTYPE_CODE:
                raise TypeError(f"unsupported dtype {t.dtype}")
            if not t.is_cuda:
                raise ValueError("gradients must be CUDA tensors (the library has no CPU path)")
            if not t.is_contiguous() and not _dense_formats(t):
                raise ValueError("gradients and out buffers must be contiguous or channels-last")
            if self.device is None:
                self.device = t.get_device()
            elif t.get_device() != self.device:
                raise ValueError("gradients are on different devices")
        spans = []
        for i, g in enumerate(self.grads):
            o = None if self.out is None else self.out[i]
            if o is not None and o.shape != g.shape:
                raise ValueError(f"out[{i}] shape {tuple(o.shape)} != {tuple(g.shape)}")
            if o is not None and not (o.is_contiguous() and g.is_contiguous()) and \
                    not set(_dense_formats(o)) & set(_dense_formats(g)):
                raise ValueError(f"out[{i}] and its gradient lie in different memory formats")
            spans.append((g.data_ptr(), g.numel() * g.element_size()))
            if o is not None and not (o.data_ptr() == g.data_ptr() and o.dtype == g.dtype):
                spans.append((o.data_ptr(), o.numel() * o.element_size()))
        end = 0
        for at, size in sorted(s for s in spans if s[1]):
            if at < end:
                raise ValueError("gradient or out buffers overlap")
            end = at + size
        self.count = n
        self._g = (ctypes.c_void_p * max(n, 1))(*[t.data_ptr() for t in self.grads])
        self._n = (ctypes.c_int64 * max(n, 1))(*[t.numel() for t in self.grads])
        self._d = (ctypes.c_int32 * max(n, 1))(*[_DTYPE_CODE[t.dtype] for t in self.grads])
        self._o = self._od = None
        if self.out is not None:
            self._o = (ctypes.c_void_p * max(n, 1))(*[t.data_ptr() for t in self.out])
            self._od = (ctypes.c_int32 * max(n, 1))(*[_DTYPE_CODE[t.dtype] for t in self.out])
        self._ws = int(lib().dcn_grad_norm_workspace_bytes(n))
        if self._ws < 0:
            raise ValueError(f"{n} gradients are too many")
        self._protos = None

    def _new(self, index: int):
        """A norm and a workspace of a call's own (two calls may overlap on the GPU)."""
        if self._protos is None:  # empty_like of these takes half the time of torch.empty
            dev = torch.device("cuda", index)
            self._protos = (torch.empty((), dtype=torch.float32, device=dev),
                            torch.empty(self._ws, dtype=torch.uint8, device=dev))
        return torch.empty_like(self._protos[0]), torch.empty_like(self._protos[1])


_NORM_KIND = {2: 0, 2.0: 0, float("inf"): 1}


def _grad_call(grads, out, norm_type, norm, workspace):
    if not isinstance(grads, GradList):
        grads = GradList(grads, out)
    elif out is not None:
        raise ValueError("out belongs to the GradList")
    if norm_type not in _NORM_KIND:
        raise ValueError(f"norm_type must be 2 or inf, not {norm_type}")
    dev = grads.device
    if dev is None:
        if norm is None:
            raise ValueError("no gradients: pass norm, which gives the device")
        _cuda_tensor("norm", norm)
        dev = norm.get_device()
    if norm is not None:
        _like("norm", norm, (), torch.float32, dev)
    if workspace is not None:
        ws_ptr, ws_bytes = _workspace(workspace, dev)
    if norm is None or workspace is None:
        n, w = grads._new(dev)
        if norm is None:
            norm = n
        if workspace is None:
            workspace, ws_ptr, ws_bytes = w, w.data_ptr(), grads._ws
    return grads, dev, norm, workspace, ws_ptr, ws_bytes


def dcn_grad_norm(grads, *, norm_type: float = 2.0, norm=None, workspace=None) -> torch.Tensor:
    """The 2-norm (or largest magnitude, norm_type inf) of all gradients together, an fp32 scalar on the
    device; grads is a GradList or a sequence of tensors.  See dcn_b200.h."""
    grads, dev, norm, workspace, ws_ptr, ws_bytes = _grad_call(grads, None, norm_type, norm, workspace)
    p = DclipParams(grads.count, _NORM_KIND[norm_type], 0.0, 1.0)
    _launch(dev, lib().dcn_grad_norm, ctypes.byref(p), grads._g, grads._n, grads._d, norm.data_ptr(),
            ws_ptr, ws_bytes)
    return norm


def dcn_clip_grads(grads, max_norm: float, *, norm_type: float = 2.0, eps: float = 1e-6, out=None, norm=None,
                   workspace=None) -> torch.Tensor:
    """Scales all gradients by min(1, max_norm / (norm + eps)), in place or into `out`, and returns the norm
    before that (fp32 scalar on the device; nothing synchronises).  See dcn_b200.h."""
    grads, dev, norm, workspace, ws_ptr, ws_bytes = _grad_call(grads, out, norm_type, norm, workspace)
    p = DclipParams(grads.count, _NORM_KIND[norm_type], max_norm, eps)
    _launch(dev, lib().dcn_clip_grads, ctypes.byref(p), grads._g, grads._n, grads._d, grads._o, grads._od,
            norm.data_ptr(), ws_ptr, ws_bytes)
    return norm


@functools.lru_cache(maxsize=1024)
def _adapters_workspace_bytes(*sizes) -> int:
    """Workspace of a problem of these sizes (a function of them alone) in one pass; 16 where they are refused."""
    return max(16, lib().dcn_proj_adapters_workspace_full_bytes(ctypes.byref(DadaptParams(*sizes))))


def dcn_proj_adapters_forward(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor],
                              a: torch.Tensor, b: torch.Tensor, request_start: torch.Tensor,
                              request_adapter: torch.Tensor, *, scale: Optional[torch.Tensor] = None,
                              out: Optional[torch.Tensor] = None,
                              workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out[..., cout] = bias + x . weight^T + scale[i] * (x . a[i]^T) . b[i]^T, i the adapter of the row's
    request; see dcn_b200.h.

    x is [..., cin], its leading dimensions flattened to rows; weight [cout, cin], a [adapters, rank, cin],
    b [adapters, cout, rank], scale [adapters] fp32.  Request s owns rows request_start[s] up to
    request_start[s + 1] (int32 [requests + 1], on the device) and uses adapter request_adapter[s] (int32
    [requests], -1 for none).  Rows of no request are not written: in a new `out` they hold no value."""
    _cuda_tensor("x", x)
    dt, dev = x.dtype, x.get_device()
    if dt not in _DTYPE_CODE:
        raise TypeError(f"unsupported dtype {dt}")
    rows, cin = _rows(x)
    ws, sa, sr = weight.shape, a.shape, request_adapter.shape
    if len(ws) != 2 or len(sa) != 3 or len(sr) != 1:
        raise ValueError("weight must be [cout, cin], a [adapters, rank, cin], request_adapter [requests]")
    cout, na, rank, nr = ws[0], sa[0], sa[1], sr[0]
    if cout > _INT32_MAX or na > _INT32_MAX or rank > _INT32_MAX or nr > _INT32_MAX:
        raise ValueError("a size exceeds 32 bits")
    _like("weight", weight, (cout, cin), dt, dev)
    if bias is not None:
        _like("bias", bias, (cout,), dt, dev)
    _like("a", a, (na, rank, cin), dt, dev)
    _like("b", b, (na, cout, rank), dt, dev)
    _like("request_start", request_start, (nr + 1,), torch.int32, dev)
    _like("request_adapter", request_adapter, (nr,), torch.int32, dev)
    if scale is not None:
        _like("scale", scale, (na,), torch.float32, dev)
    if out is not None:
        _like("out", out, x.shape[:-1] + (cout,), dt, dev)
    else:
        out = torch.empty_like(x) if cout == cin else x.new_empty(x.shape[:-1] + (cout,))
    sizes = (rows, cin, cout, rank, na, nr, _DTYPE_CODE[dt])
    p = DadaptParams(*sizes)
    L = lib()
    if workspace is None:
        ws_bytes = _adapters_workspace_bytes(*sizes)
        workspace = x.new_empty(ws_bytes, dtype=torch.uint8)
        ws_ptr = workspace.data_ptr()
    else:
        ws_ptr, ws_bytes = _workspace(workspace, dev)
    _launch(dev, L.dcn_proj_adapters_forward, ctypes.byref(p), x.data_ptr(), weight.data_ptr(),
            None if bias is None else bias.data_ptr(), a.data_ptr(), b.data_ptr(),
            None if scale is None else scale.data_ptr(), request_start.data_ptr(), request_adapter.data_ptr(),
            out.data_ptr(), ws_ptr, ws_bytes)
    return out
