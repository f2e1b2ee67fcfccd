"""ctypes binding of libmge.so (include/mge.h), with the same call names.

Argument marshalling only: tensors are allocated with torch (device memory and the
current stream are torch's), every step of the computation runs in the library's HIP
kernels.  If the library is not built the first call raises — there is no fallback.
"""
from __future__ import annotations

import ctypes as C
import os
from dataclasses import dataclass, field
from typing import Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmge.so")

MGE_OK, MGE_ERR_INVALID_ARG, MGE_ERR_UNSUPPORTED, MGE_ERR_WORKSPACE, MGE_ERR_HIP, MGE_ERR_DEVICE_CHECK = range(6)
PREC = {"bf16": 0, "mxfp8": 1}
DTYPE = {"bf16": 0, "f32": 1}
SCORE = {"softmax": 0, "sigmoid": 1}
FORMAT = {"mxfp8": 0, "mxfp4": 1}
ORIENT_ROW, ORIENT_COL = 1, 2
BLOCK = {"1x128": 0, "128x128": 1}
ROUTE_WANT_COL, ROUTE_PROB_GIVEN = 1, 2

vp = C.c_void_p
i32 = C.c_int32
u32 = C.c_uint32
i64 = C.c_int64


class RouteArgs(C.Structure):
    _fields_ = [("struct_size", u32), ("T", i32), ("E", i32), ("k", i32), ("H", i32), ("align", i32),
                ("prec", i32), ("flags", u32),
                ("logits", vp), ("x", vp), ("topk_idx", vp), ("topk_prob", vp), ("split_sizes", vp),
                ("group_offsets", vp), ("perm_src", vp), ("perm_pos", vp), ("prob_perm", vp),
                ("x_perm", vp), ("x_perm_scale", vp), ("x_col", vp), ("x_col_scale", vp),
                ("workspace", vp), ("workspace_bytes", C.c_size_t), ("x_tensor_scale", vp)]


class QuantArgs(C.Structure):
    _fields_ = [("struct_size", u32), ("batch", i32), ("R", i32), ("C", i32),
                ("in_batch_stride", i64), ("in_row_stride", i64), ("in_", vp), ("orient", u32),
                ("row_codes", vp), ("row_scales", vp), ("col_codes", vp), ("col_scales", vp), ("tensor_scale", vp),
                ("seg_offsets", vp), ("num_segments", i32), ("workspace", vp), ("workspace_bytes", C.c_size_t)]


class TensorScaleArgs(C.Structure):
    _fields_ = [("struct_size", u32), ("batch", i32), ("n", i64), ("batch_stride", i64), ("in_", vp),
                ("scale", vp), ("workspace", vp), ("workspace_bytes", C.c_size_t)]


class FwdArgs(C.Structure):
    _fields_ = [("struct_size", u32), ("prec", i32), ("E", i32), ("H", i32), ("F", i32), ("T", i32),
                ("k", i32), ("align", i32),
                ("split_sizes", vp), ("group_offsets", vp), ("prob_perm", vp), ("x_perm", vp),
                ("x_perm_scale", vp), ("w_gate_up", vp), ("w_gate_up_scale", vp), ("w_down", vp),
                ("w_down_scale", vp), ("y_dtype", i32), ("y_perm", vp), ("h", vp), ("h_scale", vp),
                ("saved_gu", vp), ("h_col", vp), ("h_col_scale", vp), ("workspace", vp),
                ("workspace_bytes", C.c_size_t)]


class FwdUnfusedArgs(C.Structure):
    _fields_ = [("struct_size", u32), ("fwd", FwdArgs), ("gu", vp), ("h_bf16", vp), ("h_tensor_scale", vp)]


class BwdArgs(C.Structure):
    _fields_ = [("struct_size", u32), ("prec", i32), ("E", i32), ("H", i32), ("F", i32), ("T", i32),
                ("k", i32), ("align", i32),
                ("dy", vp), ("split_sizes", vp), ("group_offsets", vp), ("perm_src", vp), ("perm_pos", vp),
                ("prob_perm", vp), ("saved_gu", vp), ("h_col", vp), ("h_col_scale", vp), ("x_col", vp),
                ("x_col_scale", vp), ("w_gate_up", vp), ("w_gate_up_scale", vp), ("w_down", vp),
                ("w_down_scale", vp), ("dx_perm", vp), ("dw_gate_up", vp), ("dw_down", vp), ("d_prob", vp),
                ("accumulate", i32),
                ("dy_row", vp), ("dy_row_scale", vp), ("dy_col", vp), ("dy_col_scale", vp),
                ("dgu_row", vp), ("dgu_row_scale", vp), ("dgu_col", vp), ("dgu_col_scale", vp),
                ("workspace", vp), ("workspace_bytes", C.c_size_t), ("dw_bf16", i32),
                ("dy_tensor_scale", vp), ("dgu_tensor_scale", vp), ("dgu_bf16", vp)]


class FwdSavedSizes(C.Structure):
    _fields_ = [("struct_size", u32), ("rows", i64), ("saved_gu", C.c_size_t), ("h_col", C.c_size_t),
                ("h_col_scale", C.c_size_t), ("total", C.c_size_t)]


class CombineArgs(C.Structure):
    _fields_ = [("struct_size", u32), ("T", i32), ("k", i32), ("H", i32), ("in_dtype", i32), ("out_dtype", i32),
                ("in_", vp), ("perm_pos", vp), ("weights", vp), ("out", vp), ("in_rows", i64)]


class RouterBwdArgs(C.Structure):
    _fields_ = [("struct_size", u32), ("T", i32), ("E", i32), ("k", i32), ("topk_idx", vp), ("topk_prob", vp),
                ("d_prob", vp), ("d_logits", vp)]


class RouteTopkArgs(C.Structure):
    _fields_ = [("struct_size", u32), ("T", i32), ("E", i32), ("k", i32), ("score", i32), ("num_groups", i32),
                ("topk_groups", i32), ("group_topn", i32), ("renormalize", i32), ("scale", C.c_float),
                ("logits_dtype", i32), ("logits_row_stride", i64), ("logits", vp), ("bias", vp), ("topk_idx", vp),
                ("topk_prob", vp)]


class RouteTopkBwdArgs(C.Structure):
    _fields_ = [("struct_size", u32), ("T", i32), ("E", i32), ("k", i32), ("score", i32), ("renormalize", i32),
                ("scale", C.c_float), ("logits_dtype", i32), ("logits_row_stride", i64), ("logits", vp),
                ("topk_idx", vp), ("d_prob", vp), ("d_logits", vp)]


class Quant4Args(C.Structure):
    _fields_ = [("struct_size", u32), ("batch", i32), ("R", i32), ("C", i32), ("in_batch_stride", i64),
                ("in_row_stride", i64), ("in_", vp), ("orient", u32), ("row_codes", vp), ("row_scales", vp),
                ("col_codes", vp), ("col_scales", vp)]


class Dequant4Args(C.Structure):
    _fields_ = [("struct_size", u32), ("rows", i64), ("C", i32), ("out_dtype", i32), ("codes", vp), ("scales", vp),
                ("out", vp)]


class Gemm4Args(C.Structure):
    _fields_ = [("struct_size", u32), ("a_format", i32), ("E", i32), ("N", i32), ("K", i32), ("rows", i64),
                ("total_rows", i64), ("split_sizes", vp), ("group_offsets", vp), ("a", vp), ("a_scale", vp), ("w", vp),
                ("w_scale", vp), ("out_dtype", i32), ("out", vp), ("workspace", vp), ("workspace_bytes", C.c_size_t)]


class RmsnormArgs(C.Structure):
    _fields_ = [("struct_size", u32), ("T", i32), ("H", i32), ("x_dtype", i32), ("weight_dtype", i32), ("y_dtype", i32),
                ("eps", C.c_float), ("x_row_stride", i64), ("x", vp), ("residual", vp), ("weight", vp),
                ("residual_out", vp), ("y", vp), ("codes", vp), ("scales", vp), ("rstd", vp)]


class RmsnormBwdArgs(C.Structure):
    _fields_ = [("struct_size", u32), ("T", i32), ("H", i32), ("x_dtype", i32), ("weight_dtype", i32), ("dy_dtype", i32),
                ("x_row_stride", i64), ("dy_row_stride", i64), ("dy", vp), ("x", vp), ("weight", vp), ("rstd", vp),
                ("d_residual", vp), ("dx", vp), ("d_weight", vp), ("workspace", vp), ("workspace_bytes", C.c_size_t)]


class QuantFbArgs(C.Structure):
    _fields_ = [("struct_size", u32), ("block", i32), ("batch", i32), ("R", i32), ("C", i32), ("in_batch_stride", i64),
                ("in_row_stride", i64), ("in_", vp), ("rows", vp), ("src_rows", i64), ("orient", u32), ("row_codes", vp),
                ("row_scales", vp), ("col_codes", vp), ("col_scales", vp)]


class DequantFbArgs(C.Structure):
    _fields_ = [("struct_size", u32), ("block", i32), ("batch", i32), ("R", i32), ("C", i32), ("out_dtype", i32),
                ("codes", vp), ("scales", vp), ("out", vp)]


class GemmFbArgs(C.Structure):
    _fields_ = [("struct_size", u32), ("E", i32), ("N", i32), ("K", i32), ("rows", i64), ("total_rows", i64),
                ("split_sizes", vp), ("group_offsets", vp), ("a_rows", vp), ("src_rows", i64), ("a", vp), ("a_scale", vp),
                ("w", vp), ("w_scale", vp), ("out_dtype", i32), ("out", vp), ("workspace", vp),
                ("workspace_bytes", C.c_size_t)]


class WgradFbArgs(C.Structure):
    _fields_ = [("struct_size", u32), ("E", i32), ("N", i32), ("K", i32), ("rows", i64), ("split_sizes", vp),
                ("group_offsets", vp), ("dy", vp), ("dy_scale", vp), ("x", vp), ("x_scale", vp), ("out_dtype", i32),
                ("accumulate", i32), ("dw", vp), ("workspace", vp), ("workspace_bytes", C.c_size_t)]


class FwdFbArgs(C.Structure):
    _fields_ = [("struct_size", u32), ("E", i32), ("H", i32), ("F", i32), ("rows", i64), ("total_rows", i64),
                ("split_sizes", vp), ("group_offsets", vp), ("perm_src", vp), ("prob_perm", vp), ("x_rows", i64), ("x", vp),
                ("x_scale", vp), ("w_gate_up", vp), ("w_gate_up_scale", vp), ("w_down", vp), ("w_down_scale", vp),
                ("y_dtype", i32), ("y_perm", vp), ("workspace", vp), ("workspace_bytes", C.c_size_t)]


_LIB = None
EXPORTS = ["rmsnorm_fwd", "mge_rmsnorm_bwd_workspace_bytes", "rmsnorm_bwd", "fp8_block_quantize", "fp8_block_dequantize",
           "mge_gemm_fb_workspace_bytes", "fp8_block_grouped_gemm", "mge_wgrad_fb_workspace_bytes",
           "fp8_block_grouped_wgrad", "mge_fwd_fb_workspace_bytes", "grouped_mlp_fwd_fp8_block",
           "moe_route_topk", "moe_route_topk_bwd", "mxfp4_quantize", "mxfp4_dequantize", "mge_gemm4_workspace_bytes",
           "mxfp4_grouped_gemm", "mge_fwd_mxfp4_workspace_bytes", "grouped_mlp_fwd_mxfp4",
           "mge_perm_rows", "mge_route_workspace_bytes", "moe_route_permute", "moe_route_permute_noalloc",
           "mxfp8_quantize",
           "mge_fwd_workspace_bytes", "grouped_mlp_fwd", "mge_fwd_saved_bytes", "mge_fwd_unfused_workspace_bytes", "grouped_mlp_fwd_unfused",
           "mge_tensor_scale_workspace_bytes", "mge_tensor_scale", "mge_quant_workspace_bytes",
           "mge_bwd_workspace_bytes", "grouped_mlp_bwd",
           "unpermute_combine", "moe_router_bwd", "mge_status_string", "mge_last_error", "mge_check_device_errors", "mge_version",
           "mge_profile_start", "mge_profile_stop"]


class KernelTime(C.Structure):
    _fields_ = [("name", C.c_char * 56), ("ms", C.c_float)]


def lib():
    """Loads libmge.so (raises if it is not built)."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built; run `python -m moe_grouped_expert_amd.build`")
        L = C.CDLL(LIB_PATH)
        L.mge_perm_rows.restype = i64
        L.mge_perm_rows.argtypes = [i32, i32, i32, i32]
        L.mge_route_workspace_bytes.restype = C.c_size_t
        L.mge_route_workspace_bytes.argtypes = [i32, i32]
        L.mge_fwd_workspace_bytes.restype = C.c_size_t
        L.mge_fwd_workspace_bytes.argtypes = [C.POINTER(FwdArgs)]
        L.mge_fwd_saved_bytes.restype = C.c_int
        L.mge_fwd_saved_bytes.argtypes = [i32, i32, i32, i32, i32, i32, C.POINTER(FwdSavedSizes)]
        L.mge_fwd_unfused_workspace_bytes.restype = C.c_size_t
        L.mge_fwd_unfused_workspace_bytes.argtypes = [C.POINTER(FwdUnfusedArgs)]
        L.mge_quant_workspace_bytes.restype = C.c_size_t
        L.mge_quant_workspace_bytes.argtypes = [C.POINTER(QuantArgs)]
        L.mge_tensor_scale_workspace_bytes.restype = C.c_size_t
        L.mge_tensor_scale_workspace_bytes.argtypes = [i32, i64]
        L.mge_bwd_workspace_bytes.restype = C.c_size_t
        L.mge_bwd_workspace_bytes.argtypes = [C.POINTER(BwdArgs)]
        L.mge_gemm4_workspace_bytes.restype = C.c_size_t
        L.mge_gemm4_workspace_bytes.argtypes = [C.POINTER(Gemm4Args)]
        L.mge_fwd_mxfp4_workspace_bytes.restype = C.c_size_t
        L.mge_fwd_mxfp4_workspace_bytes.argtypes = [C.POINTER(FwdArgs)]
        L.mge_rmsnorm_bwd_workspace_bytes.restype = C.c_size_t
        L.mge_rmsnorm_bwd_workspace_bytes.argtypes = [i32, i32]
        for name, st in (("mge_gemm_fb_workspace_bytes", GemmFbArgs), ("mge_wgrad_fb_workspace_bytes", WgradFbArgs),
                         ("mge_fwd_fb_workspace_bytes", FwdFbArgs)):
            getattr(L, name).restype = C.c_size_t
            getattr(L, name).argtypes = [C.POINTER(st)]
        for name, st in (("rmsnorm_fwd", RmsnormArgs), ("rmsnorm_bwd", RmsnormBwdArgs),
                         ("fp8_block_quantize", QuantFbArgs), ("fp8_block_dequantize", DequantFbArgs),
                         ("fp8_block_grouped_gemm", GemmFbArgs), ("fp8_block_grouped_wgrad", WgradFbArgs),
                         ("grouped_mlp_fwd_fp8_block", FwdFbArgs),
                         ("moe_route_topk", RouteTopkArgs), ("moe_route_topk_bwd", RouteTopkBwdArgs),
                         ("mxfp4_quantize", Quant4Args), ("mxfp4_dequantize", Dequant4Args),
                         ("mxfp4_grouped_gemm", Gemm4Args), ("grouped_mlp_fwd_mxfp4", FwdArgs),
                         ("moe_route_permute", RouteArgs), ("moe_route_permute_noalloc", RouteArgs),
                         ("mxfp8_quantize", QuantArgs),
                         ("mge_tensor_scale", TensorScaleArgs),
                         ("grouped_mlp_fwd", FwdArgs), ("grouped_mlp_fwd_unfused", FwdUnfusedArgs),
                         ("grouped_mlp_bwd", BwdArgs),
                         ("unpermute_combine", CombineArgs), ("moe_router_bwd", RouterBwdArgs)):
            f = getattr(L, name)
            f.restype = C.c_int
            f.argtypes = [C.POINTER(st), vp]
        L.mge_status_string.restype = C.c_char_p
        L.mge_status_string.argtypes = [C.c_int]
        L.mge_last_error.restype = C.c_char_p
        L.mge_last_error.argtypes = []
        L.mge_check_device_errors.restype = C.c_int
        L.mge_check_device_errors.argtypes = [vp, vp]
        L.mge_version.restype = C.c_char_p
        L.mge_profile_start.restype = C.c_int
        L.mge_profile_start.argtypes = []
        L.mge_profile_stop.restype = i32
        L.mge_profile_stop.argtypes = [C.c_void_p, i32]
        _LIB = L
    return _LIB


class MgeError(RuntimeError):
    def __init__(self, code: int, where: str):
        L = lib()
        super().__init__(f"{where}: {L.mge_status_string(code).decode()}: {L.mge_last_error().decode()}")
        self.code = code


def _check(code: int, where: str):
    if code != MGE_OK:
        raise MgeError(code, where)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _stream(dev) -> int:
    return torch.cuda.current_stream(dev).cuda_stream


def _ptr_array(ts: Sequence[torch.Tensor]):
    arr = (vp * len(ts))(*[t.data_ptr() for t in ts])
    return arr


def perm_rows(T: int, k: int, E: int, align: int) -> int:
    """Rows of the permuted buffers for T tokens, top-k over E experts, groups starting at
    multiples of `align`: T*k plus the worst-case padding, E*(align-1)."""
    return int(lib().mge_perm_rows(T, k, E, align))


# ------------------------------------------------------------------------------ routing

@dataclass
class RouteOut:
    T: int
    E: int
    k: int
    H: int
    align: int
    prec: str
    R: int
    topk_idx: torch.Tensor
    topk_prob: torch.Tensor
    split_sizes: torch.Tensor
    group_offsets: torch.Tensor
    perm_src: torch.Tensor
    perm_pos: torch.Tensor
    prob_perm: torch.Tensor
    x_perm: Optional[torch.Tensor] = None
    x_perm_scale: Optional[torch.Tensor] = None
    x_col: Optional[torch.Tensor] = None
    x_col_scale: Optional[torch.Tensor] = None
    workspace: Optional[torch.Tensor] = None


def moe_route_permute(logits: Optional[torch.Tensor], x: Optional[torch.Tensor], k: int, E: Optional[int] = None,
                      align: int = 32, prec: str = "bf16", want_col: bool = False,
                      topk_idx: Optional[torch.Tensor] = None, topk_prob: Optional[torch.Tensor] = None,
                      out: Optional[RouteOut] = None, x_tensor_scale: Optional[torch.Tensor] = None,
                      noalloc: bool = False) -> RouteOut:
    """Top-k routing + stable permutation by expert (+ gather / quantize of x; with
    x_tensor_scale, a uint8 [1] tensor from tensor_scale(x), every block of x takes that
    one scale).  noalloc: call moe_route_permute_noalloc, whose workspace is the library's
    fixed scratch (no workspace tensor is allocated or passed)."""
    given = topk_idx is not None
    ref = logits if logits is not None else topk_idx
    dev = ref.device
    if logits is not None:
        T, E = logits.shape
        assert logits.dtype == torch.float32 and logits.is_contiguous()
    else:
        T = topk_idx.shape[0]
        assert E is not None
    H = x.shape[1] if x is not None else 32
    if x is not None:
        assert x.dtype == torch.bfloat16 and x.is_contiguous() and x.shape[0] == T
    R = perm_rows(T, k, E, align)
    if out is None:
        i = dict(device=dev, dtype=torch.int32)
        f = dict(device=dev, dtype=torch.float32)
        o = RouteOut(T=T, E=E, k=k, H=H, align=align, prec=prec, R=R,
                     topk_idx=topk_idx if given else torch.empty((T, k), **i),
                     topk_prob=topk_prob if given else torch.empty((T, k), **f),
                     split_sizes=torch.empty(E, **i), group_offsets=torch.empty(E + 1, **i),
                     perm_src=torch.empty(R, **i), perm_pos=torch.empty((T, k), **i), prob_perm=torch.empty(R, **f))
        if x is not None:
            if prec == "mxfp8":
                o.x_perm = torch.empty((R, H), device=dev, dtype=torch.uint8)
                o.x_perm_scale = torch.empty((R, H // 32), device=dev, dtype=torch.uint8)
                if want_col:
                    o.x_col = torch.empty((H, R), device=dev, dtype=torch.uint8)
                    o.x_col_scale = torch.empty((H, R // 32), device=dev, dtype=torch.uint8)
            else:
                o.x_perm = torch.empty((R, H), device=dev, dtype=torch.bfloat16)
                if want_col:
                    o.x_col = torch.empty((H, R), device=dev, dtype=torch.bfloat16)
        if not noalloc:
            nbytes = int(lib().mge_route_workspace_bytes(T, E))
            o.workspace = torch.empty(max(nbytes, 256), device=dev, dtype=torch.uint8)
    else:
        o = out
    a = RouteArgs()
    a.struct_size = C.sizeof(RouteArgs)
    a.T, a.E, a.k, a.H, a.align = T, E, k, H, align
    a.prec = PREC[prec]
    a.flags = (ROUTE_WANT_COL if want_col else 0) | (ROUTE_PROB_GIVEN if given else 0)
    a.logits = _ptr(logits)
    a.x = _ptr(x)
    a.topk_idx, a.topk_prob = _ptr(o.topk_idx), _ptr(o.topk_prob)
    a.split_sizes, a.group_offsets = _ptr(o.split_sizes), _ptr(o.group_offsets)
    a.perm_src, a.perm_pos, a.prob_perm = _ptr(o.perm_src), _ptr(o.perm_pos), _ptr(o.prob_perm)
    a.x_perm, a.x_perm_scale = _ptr(o.x_perm), _ptr(o.x_perm_scale)
    a.x_col, a.x_col_scale = _ptr(o.x_col), _ptr(o.x_col_scale)
    a.x_tensor_scale = _ptr(x_tensor_scale)
    if noalloc:
        a.workspace, a.workspace_bytes = None, 0
        _check(lib().moe_route_permute_noalloc(C.byref(a), _stream(dev)), "moe_route_permute_noalloc")
    else:
        a.workspace, a.workspace_bytes = _ptr(o.workspace), o.workspace.numel()
        _check(lib().moe_route_permute(C.byref(a), _stream(dev)), "moe_route_permute")
    return o


def check_device_errors(route: RouteOut) -> int:
    """Synchronise the stream and read the routing call's device flag (set when a given
    top-k index was out of range and clamped); returns the library status code.  For
    tests and debugging: it blocks the host."""
    return lib().mge_check_device_errors(_ptr(route.workspace), _stream(route.workspace.device))


# ------------------------------------------------------------------------------ quantize

def mxfp8_quantize(w: torch.Tensor, orient: str = "row", out=None, tensor_scale: Optional[torch.Tensor] = None,
                   seg_offsets: Optional[torch.Tensor] = None):
    """BF16 [..., R, C] -> (row_codes, row_scales, col_codes, col_scales) (absent ones None).
    tensor_scale: optional uint8 [batch] (one scale per matrix, from tensor_scale(w,
    per_matrix=True)) that every block of its matrix takes instead of its own.
    seg_offsets: optional int32 [S+1] on the device: segments along R, each placed at a
    multiple of 32 rows (zero-padded), in perm_rows(R, 1, S, 32) output rows, so that the
    column form's 32-row blocks restart at every segment."""
    assert w.dtype == torch.bfloat16 and w.is_contiguous()
    R, Cc = w.shape[-2], w.shape[-1]
    lead = tuple(w.shape[:-2])
    batch = 1
    for d in lead:
        batch *= d
    Rp = (R + 31) // 32 * 32
    nseg = 0
    if seg_offsets is not None:
        assert seg_offsets.dtype == torch.int32 and seg_offsets.is_contiguous() and seg_offsets.numel() >= 2
        nseg = seg_offsets.numel() - 1
        Rp = perm_rows(R, 1, nseg, 32)
    Rr = Rp if seg_offsets is not None else R   # rows of the row form
    want_row = orient in ("row", "both")
    want_col = orient in ("col", "both")
    dev = w.device
    if out is None:
        u8 = dict(device=dev, dtype=torch.uint8)
        rc = torch.empty(lead + (Rr, Cc), **u8) if want_row else None
        rs = torch.empty(lead + (Rr, Cc // 32), **u8) if want_row else None
        cc = torch.empty(lead + (Cc, Rp), **u8) if want_col else None
        cs = torch.empty(lead + (Cc, Rp // 32), **u8) if want_col else None
    else:
        rc, rs, cc, cs = out
    a = QuantArgs()
    a.struct_size = C.sizeof(QuantArgs)
    a.batch, a.R, a.C = batch, R, Cc
    a.in_batch_stride, a.in_row_stride = R * Cc, Cc
    a.in_ = _ptr(w)
    a.orient = (ORIENT_ROW if want_row else 0) | (ORIENT_COL if want_col else 0)
    a.row_codes, a.row_scales, a.col_codes, a.col_scales = _ptr(rc), _ptr(rs), _ptr(cc), _ptr(cs)
    if tensor_scale is not None:
        assert tensor_scale.dtype == torch.uint8 and tensor_scale.numel() == batch
    a.tensor_scale = _ptr(tensor_scale)
    ws = None
    if seg_offsets is not None:
        a.seg_offsets, a.num_segments = _ptr(seg_offsets), nseg
        ws = torch.empty(max(int(lib().mge_quant_workspace_bytes(C.byref(a))), 256), device=dev, dtype=torch.uint8)
        a.workspace, a.workspace_bytes = _ptr(ws), ws.numel()
    _check(lib().mxfp8_quantize(C.byref(a), _stream(dev)), "mxfp8_quantize")
    return rc, rs, cc, cs


@dataclass
class TensorScaleOut:
    scale: torch.Tensor        # uint8 [batch]
    workspace: torch.Tensor


def tensor_scale(t: torch.Tensor, per_matrix: bool = False, out: Optional[TensorScaleOut] = None) -> TensorScaleOut:
    """One E8M0 scale per tensor (FP8 with one scale per tensor): of all of t, or with
    per_matrix of each t[b] along the leading dimension."""
    assert t.dtype == torch.bfloat16 and t.is_contiguous()
    batch = t.shape[0] if per_matrix else 1
    n = t.numel() // max(batch, 1)
    dev = t.device
    if out is None:
        ws = int(lib().mge_tensor_scale_workspace_bytes(batch, n))
        out = TensorScaleOut(scale=torch.empty(batch, device=dev, dtype=torch.uint8),
                             workspace=torch.empty(max(ws, 256), device=dev, dtype=torch.uint8))
    a = TensorScaleArgs()
    a.struct_size = C.sizeof(TensorScaleArgs)
    a.batch, a.n, a.batch_stride = batch, n, n
    a.in_, a.scale = _ptr(t), _ptr(out.scale)
    a.workspace, a.workspace_bytes = _ptr(out.workspace), out.workspace.numel()
    _check(lib().mge_tensor_scale(C.byref(a), _stream(dev)), "mge_tensor_scale")
    return out


# ------------------------------------------------------------------------------ forward

def fwd_saved_bytes(prec: str, T: int, k: int, E: int, F: int, align: int = 32) -> FwdSavedSizes:
    """Byte sizes of the activations a training forward saves (mge_fwd_saved_bytes)."""
    o = FwdSavedSizes()
    o.struct_size = C.sizeof(FwdSavedSizes)
    _check(lib().mge_fwd_saved_bytes(PREC[prec], T, k, E, F, align, C.byref(o)), "mge_fwd_saved_bytes")
    return o


@dataclass
class FwdOut:
    y_perm: torch.Tensor
    h: torch.Tensor
    h_scale: Optional[torch.Tensor] = None
    saved_gu: Optional[torch.Tensor] = None
    h_col: Optional[torch.Tensor] = None
    h_col_scale: Optional[torch.Tensor] = None
    workspace: Optional[torch.Tensor] = None
    gu: Optional[torch.Tensor] = None          # unfused forward: [G U] bf16 (kept on request)
    h_bf16: Optional[torch.Tensor] = None      # unfused MXFP8 forward: h before its quantize
    h_tensor_scale: Optional[torch.Tensor] = None  # unfused, one scale for all of h: uint8 [1]


def _split(w, E):
    if isinstance(w, torch.Tensor):
        return [w[e] for e in range(E)]
    return list(w)


def _fwd_args(rt: RouteOut, w_gate_up, w_down, w_gate_up_scale, w_down_scale, y_dtype: str, train: bool,
              out: Optional[FwdOut]):
    """Outputs (allocated unless given) and the filled mge_fwd_args; `keep` holds the
    host pointer arrays alive while the call runs."""
    E, H, R = rt.E, rt.H, rt.R
    wg = _split(w_gate_up, E)
    wd = _split(w_down, E)
    F = wg[0].shape[0] // 2
    mx = rt.prec == "mxfp8"
    dev = rt.x_perm.device
    if out is None:
        o = FwdOut(y_perm=torch.empty((R, H), device=dev, dtype=torch.bfloat16 if y_dtype == "bf16" else torch.float32),
                   h=torch.empty((R, F), device=dev, dtype=torch.uint8 if mx else torch.bfloat16))
        if mx:
            o.h_scale = torch.empty((R, F // 32), device=dev, dtype=torch.uint8)
        if train:
            sz = fwd_saved_bytes(rt.prec, rt.T, rt.k, E, F, rt.align)
            assert sz.rows == R
            o.saved_gu = torch.empty(sz.saved_gu, device=dev, dtype=torch.uint8).view(torch.bfloat16).view(R, 2 * F)
            hdt = torch.uint8 if mx else torch.bfloat16
            o.h_col = torch.empty(sz.h_col, device=dev, dtype=torch.uint8).view(hdt).view(F, R)
            if mx:
                o.h_col_scale = torch.empty(sz.h_col_scale, device=dev, dtype=torch.uint8).view(F, R // 32)
    else:
        o = out
    a = FwdArgs()
    a.struct_size = C.sizeof(FwdArgs)
    a.prec, a.E, a.H, a.F, a.T, a.k, a.align = PREC[rt.prec], E, H, F, rt.T, rt.k, rt.align
    a.split_sizes, a.group_offsets, a.prob_perm = _ptr(rt.split_sizes), _ptr(rt.group_offsets), _ptr(rt.prob_perm)
    a.x_perm, a.x_perm_scale = _ptr(rt.x_perm), _ptr(rt.x_perm_scale)
    keep = [_ptr_array(wg), _ptr_array(wd)]
    a.w_gate_up, a.w_down = C.cast(keep[0], vp), C.cast(keep[1], vp)
    if mx:
        keep += [_ptr_array(_split(w_gate_up_scale, E)), _ptr_array(_split(w_down_scale, E))]
        a.w_gate_up_scale, a.w_down_scale = C.cast(keep[2], vp), C.cast(keep[3], vp)
    a.y_dtype = DTYPE[y_dtype]
    a.y_perm, a.h, a.h_scale = _ptr(o.y_perm), _ptr(o.h), _ptr(o.h_scale)
    a.saved_gu, a.h_col, a.h_col_scale = _ptr(o.saved_gu), _ptr(o.h_col), _ptr(o.h_col_scale)
    return o, a, keep, F, dev


def grouped_mlp_fwd(rt: RouteOut, w_gate_up, w_down, w_gate_up_scale=None, w_down_scale=None,
                    y_dtype: str = "bf16", train: bool = False, out: Optional[FwdOut] = None) -> FwdOut:
    """Grouped gate-up GEMM -> SwiGLU x prob (+ quantize) -> grouped down GEMM over every
    expert of `rt`, one launch per projection.
    w_gate_up: [E, 2F, H] (gate rows first), w_down: [E, H, F]; bf16 masters for a BF16
    route, MXFP8 row codes (with w_*_scale) for an MXFP8 one.  y_dtype "bf16" or "f32".
    train=True also keeps what the backward needs (G and U in bf16, h's column form)."""
    o, a, keep, F, dev = _fwd_args(rt, w_gate_up, w_down, w_gate_up_scale, w_down_scale, y_dtype, train, out)
    if o.workspace is None:
        o.workspace = torch.empty(max(int(lib().mge_fwd_workspace_bytes(C.byref(a))), 256), device=dev,
                                  dtype=torch.uint8)
    a.workspace, a.workspace_bytes = _ptr(o.workspace), o.workspace.numel()
    _check(lib().grouped_mlp_fwd(C.byref(a), _stream(dev)), "grouped_mlp_fwd")
    return o


def grouped_mlp_fwd_unfused(rt: RouteOut, w_gate_up, w_down, w_gate_up_scale=None, w_down_scale=None,
                            y_dtype: str = "bf16", keep_intermediates: bool = False, h_per_tensor: bool = False,
                            train: bool = False, out: Optional[FwdOut] = None) -> FwdOut:
    """The forward without the fusion: [G U] to HBM in bf16, a standalone SwiGLU x prob,
    (MXFP8) a standalone quantize of h, the grouped down GEMM.  With keep_intermediates,
    out.gu ([R][2F] bf16) and (MXFP8) out.h_bf16 ([R][F]) are kept; with h_per_tensor, h
    takes one scale for the whole tensor (out.h_tensor_scale).  train: [G U] is written to
    out.saved_gu (out.gu is the same tensor) and the column form of h to out.h_col."""
    o, a, keep, F, dev = _fwd_args(rt, w_gate_up, w_down, w_gate_up_scale, w_down_scale, y_dtype, train, out)
    u = FwdUnfusedArgs()
    u.struct_size = C.sizeof(FwdUnfusedArgs)
    if h_per_tensor and o.h_tensor_scale is None:
        o.h_tensor_scale = torch.empty(1, device=dev, dtype=torch.uint8)
    u.h_tensor_scale = _ptr(o.h_tensor_scale)
    if train:
        o.gu = o.saved_gu
    if keep_intermediates:
        if o.gu is None:
            o.gu = torch.empty((rt.R, 2 * F), device=dev, dtype=torch.bfloat16)
        if rt.prec == "mxfp8" and o.h_bf16 is None:
            o.h_bf16 = torch.empty((rt.R, F), device=dev, dtype=torch.bfloat16)
    u.gu, u.h_bf16 = _ptr(o.gu), _ptr(o.h_bf16)
    u.fwd = a
    if o.workspace is None:
        o.workspace = torch.empty(max(int(lib().mge_fwd_unfused_workspace_bytes(C.byref(u))), 256), device=dev,
                                  dtype=torch.uint8)
    u.fwd.workspace, u.fwd.workspace_bytes = _ptr(o.workspace), o.workspace.numel()
    _check(lib().grouped_mlp_fwd_unfused(C.byref(u), _stream(dev)), "grouped_mlp_fwd_unfused")
    return o


# ------------------------------------------------------------------------------ backward

@dataclass
class BwdOut:
    dx_perm: torch.Tensor
    dw_gate_up: list
    dw_down: list
    d_prob: torch.Tensor
    dy_row: Optional[torch.Tensor] = None
    dy_row_scale: Optional[torch.Tensor] = None
    dy_col: Optional[torch.Tensor] = None
    dy_col_scale: Optional[torch.Tensor] = None
    dgu_row: Optional[torch.Tensor] = None
    dgu_row_scale: Optional[torch.Tensor] = None
    dgu_col: Optional[torch.Tensor] = None
    dgu_col_scale: Optional[torch.Tensor] = None
    workspace: Optional[torch.Tensor] = None
    dy_tensor_scale: Optional[torch.Tensor] = None    # per-tensor mode: uint8 [1] each
    dgu_tensor_scale: Optional[torch.Tensor] = None
    dgu_bf16: Optional[torch.Tensor] = None           # per-tensor mode, kept on request: [R][2F] bf16


def grouped_mlp_bwd(dy: torch.Tensor, rt: RouteOut, fw: FwdOut, w_gate_up_k, w_down_k, w_gate_up_k_scale=None,
                    w_down_k_scale=None, accumulate: bool = False, keep_intermediates: bool = False,
                    out: Optional[BwdOut] = None, dw_dtype: str = "f32", per_tensor: bool = False) -> BwdOut:
    """Backward of the grouped MLP.  Weights: MXFP8 column forms, or the bf16 masters.
    dw_dtype: "f32" (default) or "bf16" (the fp32 sums rounded to nearest even; no accumulate).
    per_tensor (MXFP8): FP8 with one scale per tensor for dY and [dG dU] (out.dy_tensor_scale,
    out.dgu_tensor_scale; with keep_intermediates also the bf16 [dG dU] in out.dgu_bf16)."""
    if dw_dtype not in ("f32", "bf16"):
        raise ValueError(f"dw_dtype must be 'f32' or 'bf16', not {dw_dtype!r}")
    E, H, R, T, k = rt.E, rt.H, rt.R, rt.T, rt.k
    mx = rt.prec == "mxfp8"
    wg = _split(w_gate_up_k, E)
    wd = _split(w_down_k, E)
    F = fw.h.shape[1]
    dev = dy.device
    if out is None:
        f32 = dict(device=dev, dtype=torch.float32)
        dwt = dict(device=dev, dtype=torch.float32 if dw_dtype == "f32" else torch.bfloat16)
        o = BwdOut(dx_perm=torch.empty((R, H), device=dev, dtype=torch.bfloat16),
                   dw_gate_up=[torch.empty((2 * F, H), **dwt) for _ in range(E)],
                   dw_down=[torch.empty((H, F), **dwt) for _ in range(E)],
                   d_prob=torch.empty((T, k), **f32))
        if keep_intermediates:
            cd = torch.uint8 if mx else torch.bfloat16
            o.dy_row = torch.empty((R, H), device=dev, dtype=cd)
            o.dy_col = torch.empty((H, R), device=dev, dtype=cd)
            o.dgu_row = torch.empty((R, 2 * F), device=dev, dtype=cd)
            o.dgu_col = torch.empty((2 * F, R), device=dev, dtype=cd)
            if mx:
                u8 = dict(device=dev, dtype=torch.uint8)
                o.dy_row_scale = torch.empty((R, H // 32), **u8)
                o.dy_col_scale = torch.empty((H, R // 32), **u8)
                o.dgu_row_scale = torch.empty((R, 2 * F // 32), **u8)
                o.dgu_col_scale = torch.empty((2 * F, R // 32), **u8)
            if per_tensor:
                o.dgu_bf16 = torch.empty((R, 2 * F), device=dev, dtype=torch.bfloat16)
        if per_tensor:
            o.dy_tensor_scale = torch.empty(1, device=dev, dtype=torch.uint8)
            o.dgu_tensor_scale = torch.empty(1, device=dev, dtype=torch.uint8)
    else:
        o = out
    a = BwdArgs()
    a.struct_size = C.sizeof(BwdArgs)
    a.prec, a.E, a.H, a.F, a.T, a.k, a.align = PREC[rt.prec], E, H, F, T, k, rt.align
    a.dy = _ptr(dy)
    a.split_sizes, a.group_offsets = _ptr(rt.split_sizes), _ptr(rt.group_offsets)
    a.perm_src, a.perm_pos, a.prob_perm = _ptr(rt.perm_src), _ptr(rt.perm_pos), _ptr(rt.prob_perm)
    a.saved_gu = _ptr(fw.saved_gu)
    a.h_col, a.h_col_scale = _ptr(fw.h_col), _ptr(fw.h_col_scale)
    a.x_col, a.x_col_scale = _ptr(rt.x_col), _ptr(rt.x_col_scale)
    keep = [_ptr_array(wg), _ptr_array(wd), _ptr_array(o.dw_gate_up), _ptr_array(o.dw_down)]
    a.w_gate_up, a.w_down = C.cast(keep[0], vp), C.cast(keep[1], vp)
    a.dw_gate_up, a.dw_down = C.cast(keep[2], vp), C.cast(keep[3], vp)
    if mx:
        keep += [_ptr_array(_split(w_gate_up_k_scale, E)), _ptr_array(_split(w_down_k_scale, E))]
        a.w_gate_up_scale, a.w_down_scale = C.cast(keep[4], vp), C.cast(keep[5], vp)
    a.dx_perm, a.d_prob = _ptr(o.dx_perm), _ptr(o.d_prob)
    a.accumulate = 1 if accumulate else 0
    a.dw_bf16 = 1 if dw_dtype == "bf16" else 0
    a.dy_row, a.dy_row_scale, a.dy_col, a.dy_col_scale = _ptr(o.dy_row), _ptr(o.dy_row_scale), _ptr(o.dy_col), _ptr(o.dy_col_scale)
    a.dgu_row, a.dgu_row_scale = _ptr(o.dgu_row), _ptr(o.dgu_row_scale)
    a.dgu_col, a.dgu_col_scale = _ptr(o.dgu_col), _ptr(o.dgu_col_scale)
    a.dy_tensor_scale, a.dgu_tensor_scale, a.dgu_bf16 = _ptr(o.dy_tensor_scale), _ptr(o.dgu_tensor_scale), _ptr(o.dgu_bf16)
    if o.workspace is None:
        o.workspace = torch.empty(max(int(lib().mge_bwd_workspace_bytes(C.byref(a))), 256), device=dev,
                                  dtype=torch.uint8)
    a.workspace, a.workspace_bytes = _ptr(o.workspace), o.workspace.numel()
    _check(lib().grouped_mlp_bwd(C.byref(a), _stream(dev)), "grouped_mlp_bwd")
    return o


# ------------------------------------------------------------------------------ timing

def profile_start() -> None:
    """Start recording a HIP event pair around every kernel the library launches."""
    _check(lib().mge_profile_start(), "mge_profile_start")


def profile_stop() -> list:
    """Stop recording; returns [(kernel name, milliseconds)] in launch order."""
    L = lib()
    n = int(L.mge_profile_stop(None, 0))
    buf = (KernelTime * max(n, 1))()
    # records are kept until the next start, so a second read returns the same list
    L.mge_profile_stop(C.cast(buf, C.c_void_p), n)
    return [(buf[i].name.decode(), float(buf[i].ms)) for i in range(n)]


# ------------------------------------------------------------------------------ combine

def unpermute_combine(inp: torch.Tensor, perm_pos: torch.Tensor, weights: Optional[torch.Tensor] = None,
                      out_dtype: str = "bf16", out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out[t] = sum over i of weights[t, i] * inp[perm_pos[t, i]] (unweighted when weights
    is None), in slot order and fp32, without atomics; a slot whose entry is outside
    [0, rows of inp), such as -1, adds nothing.  inp: [rows, H] bf16 or f32 (y_perm or
    dx_perm); out_dtype "bf16" or "f32"."""
    T, k = perm_pos.shape
    H = inp.shape[1]
    dev = inp.device
    if out is None:
        out = torch.empty((T, H), device=dev, dtype=torch.bfloat16 if out_dtype == "bf16" else torch.float32)
    a = CombineArgs(C.sizeof(CombineArgs), T, k, H, DTYPE["bf16"] if inp.dtype == torch.bfloat16 else DTYPE["f32"],
                    DTYPE["bf16"] if out.dtype == torch.bfloat16 else DTYPE["f32"], inp.data_ptr(), perm_pos.data_ptr(),
                    _ptr(weights), out.data_ptr(), inp.shape[0])
    _call("unpermute_combine", a, dev)
    return out


# ------------------------------------------------------------------------------ router backward

def moe_router_bwd(topk_idx: torch.Tensor, topk_prob: torch.Tensor, d_prob: torch.Tensor, E: int,
                   out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """d_logits fp32 [T][E] from the slots' indices, probabilities and d_prob ([T][k] each)."""
    T, k = topk_idx.shape
    dev = topk_idx.device
    if out is None:
        out = torch.empty((T, E), device=dev, dtype=torch.float32)
    a = RouterBwdArgs()
    a.struct_size = C.sizeof(RouterBwdArgs)
    a.T, a.E, a.k = T, E, k
    a.topk_idx, a.topk_prob, a.d_prob, a.d_logits = _ptr(topk_idx), _ptr(topk_prob), _ptr(d_prob), _ptr(out)
    _check(lib().moe_router_bwd(C.byref(a), _stream(dev)), "moe_router_bwd")
    return out


# ------------------------------------------------------------------------------ router choice

_TORCH_DTYPE = {torch.bfloat16: 0, torch.float32: 1}


def _need(ok: bool, what: str):
    if not ok:
        raise ValueError(what)


# The current device and a device's current stream: torch's shortcuts, which make no objects,
# or its public calls where it has none.
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or _stream


def _call(fn: str, a, dev) -> None:
    """One library call on the current stream of `dev`, with `dev` current while it launches."""
    f = getattr(_LIB or lib(), fn)
    if dev.index == _current_device():
        code = f(C.byref(a), _raw_stream(dev.index))
    else:
        with torch.cuda.device(dev):
            code = f(C.byref(a), _stream(dev))
    if code:
        raise MgeError(code, fn)


def _on(dev, *ts) -> None:
    if dev.type != "cuda":
        raise ValueError(f"tensors must be on a GPU (got {dev})")
    for t in ts:
        if t is not None and t.device != dev:
            raise ValueError("tensors on different devices")


def _check_logits(logits, score: str) -> int:
    """Checks the router's logits; returns their row stride."""
    if score not in SCORE:
        raise ValueError(f"score must be 'softmax' or 'sigmoid', not {score!r}")
    if logits.dim() != 2 or logits.dtype not in _TORCH_DTYPE:
        raise ValueError("logits must be [T, E], float32 or bfloat16")
    T, E = logits.shape
    ld, one = logits.stride()
    if one != 1 and E > 1:
        raise ValueError("the experts of a row of logits must be contiguous")
    return ld if T > 1 else E


def moe_route_topk(logits: torch.Tensor, k: int, score: str = "softmax", bias: Optional[torch.Tensor] = None,
                   num_groups: int = 1, topk_groups: int = 1, group_topn: int = 2, renormalize: bool = True,
                   scale: float = 1.0, out=None):
    """The k experts of each token and their weights -> (topk_idx int32 [T, k], topk_prob fp32 [T, k]), the pair that
    moe_route_permute takes.  logits: [T, E] fp32 or bf16 (rows may be strided); -inf or NaN masks an expert.
    score "softmax" or "sigmoid"; bias: fp32 [E], added to the scores for the choice only; num_groups / topk_groups:
    choose among the topk_groups best of num_groups equal groups, ranked by the sum of their group_topn (1 or 2)
    best; renormalize: weights divided by their sum; all weights times scale.  out: the pair to write into."""
    ld = _check_logits(logits, score)
    T, E = logits.shape
    dev = logits.device
    _on(dev, bias)
    if bias is not None and (bias.dtype != torch.float32 or not bias.is_contiguous() or bias.numel() != E):
        raise ValueError("bias must be contiguous float32 [E]")
    if out is None:
        _need(k >= 1, "k must be >= 1")
        idx, prob = logits.new_empty((T, k), dtype=torch.int32), logits.new_empty((T, k), dtype=torch.float32)
    else:
        idx, prob = out
        _on(dev, idx, prob)
        _need(idx.dtype == torch.int32 and prob.dtype == torch.float32 and idx.shape == (T, k) and prob.shape == (T, k)
              and idx.is_contiguous() and prob.is_contiguous(), "out must be contiguous (int32 [T, k], float32 [T, k])")
    a = RouteTopkArgs(C.sizeof(RouteTopkArgs), T, E, k, SCORE[score], num_groups, topk_groups, group_topn,
                      1 if renormalize else 0, scale, _TORCH_DTYPE[logits.dtype], ld, logits.data_ptr(),
                      None if bias is None else bias.data_ptr(), idx.data_ptr(), prob.data_ptr())
    _call("moe_route_topk", a, dev)
    return idx, prob


def moe_route_topk_bwd(logits: torch.Tensor, topk_idx: torch.Tensor, d_prob: torch.Tensor, score: str = "softmax",
                       renormalize: bool = True, scale: float = 1.0, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """d_logits [T, E] (the logits' dtype, contiguous) from the forward's logits and choice and d_prob fp32 [T, k];
    score, renormalize and scale as the forward had them (the choice and its bias have no gradient)."""
    ld = _check_logits(logits, score)
    T, E = logits.shape
    dev = logits.device
    _on(dev, topk_idx, d_prob, out)
    if out is None:
        out = logits.new_empty((T, E))
    _need(topk_idx.dim() == 2 and topk_idx.shape[0] == T and topk_idx.dtype == torch.int32 and topk_idx.is_contiguous(),
          "topk_idx must be contiguous int32 [T, k]")
    _need(d_prob.shape == topk_idx.shape and d_prob.dtype == torch.float32 and d_prob.is_contiguous(),
          "d_prob must be contiguous float32 [T, k]")
    _need(out.shape == (T, E) and out.dtype == logits.dtype and out.is_contiguous(),
          "out must be contiguous [T, E] of the logits' dtype")
    a = RouteTopkBwdArgs(C.sizeof(RouteTopkBwdArgs), T, E, topk_idx.shape[1], SCORE[score], 1 if renormalize else 0,
                         scale, _TORCH_DTYPE[logits.dtype], ld, logits.data_ptr(), topk_idx.data_ptr(),
                         d_prob.data_ptr(), out.data_ptr())
    _call("moe_route_topk_bwd", a, dev)
    return out


# ------------------------------------------------------------------------------ MXFP4

def _is_u8(t) -> bool:
    return t.dtype == torch.uint8 and t.is_contiguous()


def mxfp4_quantize(w: torch.Tensor, orient: str = "row", out=None):
    """BF16 [..., R, C] -> (row_codes, row_scales, col_codes, col_scales) in MXFP4 (absent ones None): codes uint8
    [..., R, C/2] (two elements a byte, the even one in the low half) and scales uint8 [..., R, C/32]; the column
    form is that of the transpose, R padded to 32: [..., C, Rp/2] and [..., C, Rp/32].  orient "row", "col" or
    "both".  w: contiguous, or a 2-D matrix with a row stride that is a multiple of 8."""
    shape = w.shape
    if w.dtype != torch.bfloat16 or len(shape) < 2:
        raise ValueError("w must be bfloat16 [..., R, C]")
    if orient not in ("row", "col", "both"):
        raise ValueError(f"orient must be 'row', 'col' or 'both', not {orient!r}")
    R, Cc = shape[-2], shape[-1]
    row_stride = Cc
    if not w.is_contiguous():
        row_stride = w.stride(0)
        if len(shape) != 2 or (Cc > 1 and w.stride(1) != 1) or row_stride < Cc:
            raise ValueError("w must be contiguous, or a matrix of contiguous rows")
    lead = tuple(shape[:-2])
    batch = 1
    for d in lead:
        batch *= d
    Rp = (R + 31) // 32 * 32
    want_row, want_col = orient != "col", orient != "row"
    dev = w.device
    _on(dev)
    rc = rs = cc = cs = None
    if out is None:
        u8 = torch.uint8
        if want_row:
            rc, rs = w.new_empty(lead + (R, Cc // 2), dtype=u8), w.new_empty(lead + (R, Cc // 32), dtype=u8)
        if want_col:
            cc, cs = w.new_empty(lead + (Cc, Rp // 2), dtype=u8), w.new_empty(lead + (Cc, Rp // 32), dtype=u8)
    else:
        rc, rs, cc, cs = out
        _on(dev, rc, rs, cc, cs)
        for t, n, used in ((rc, R * Cc // 2, want_row), (rs, R * (Cc // 32), want_row), (cc, Cc * Rp // 2, want_col),
                           (cs, Cc * (Rp // 32), want_col)):
            _need(not used or (t is not None and _is_u8(t) and t.numel() == batch * n),
                  "out must be contiguous uint8 tensors of the outputs' sizes")
    a = Quant4Args(C.sizeof(Quant4Args), batch, R, Cc, R * row_stride, row_stride, w.data_ptr(),
                   (ORIENT_ROW if want_row else 0) | (ORIENT_COL if want_col else 0), _ptr(rc) if want_row else None,
                   _ptr(rs) if want_row else None, _ptr(cc) if want_col else None, _ptr(cs) if want_col else None)
    _call("mxfp4_quantize", a, dev)
    return rc, rs, cc, cs


def mxfp4_dequantize(codes: torch.Tensor, scales: torch.Tensor, out_dtype: str = "bf16",
                     out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Values [..., C] (bf16 or f32) of MXFP4 codes [..., C/2] and scales [..., C/32]."""
    if out_dtype not in DTYPE:
        raise ValueError(f"out_dtype must be 'bf16' or 'f32', not {out_dtype!r}")
    if codes.dim() < 1 or not _is_u8(codes) or not _is_u8(scales):
        raise ValueError("codes and scales must be contiguous uint8")
    lead, Cc = tuple(codes.shape[:-1]), codes.shape[-1] * 2
    if Cc % 32 or scales.shape != lead + (Cc // 32,):
        raise ValueError("codes must be [..., C/2] and scales [..., C/32], C a multiple of 32")
    dev = codes.device
    dt = torch.bfloat16 if out_dtype == "bf16" else torch.float32
    _on(dev, scales, out)
    if out is None:
        out = codes.new_empty(lead + (Cc,), dtype=dt)
    elif out.shape != lead + (Cc,) or out.dtype != dt or not out.is_contiguous():
        raise ValueError("out has another shape or dtype")
    rows = codes.numel() // max(Cc // 2, 1)
    a = Dequant4Args(C.sizeof(Dequant4Args), rows, Cc, DTYPE[out_dtype], codes.data_ptr(), scales.data_ptr(), out.data_ptr())
    _call("mxfp4_dequantize", a, dev)
    return out


def _expert_ptrs(w, E: int, rows: int, cols: int, dev, what: str):
    """Host array of the E device pointers of [rows][cols] uint8 matrices: one stacked tensor or a sequence."""
    if isinstance(w, torch.Tensor):
        if w.shape != (E, rows, cols) or not _is_u8(w) or w.device != dev:
            raise ValueError(f"{what} must be contiguous uint8 [{E}, {rows}, {cols}] on {dev}")
        p, n = w.data_ptr(), rows * cols
        return (vp * E)(*range(p, p + E * n, n)) if E > 1 and n else (vp * E)(*[p] * E)
    ts = list(w)
    if len(ts) != E or not all(t.shape == (rows, cols) and _is_u8(t) and t.device == dev for t in ts):
        raise ValueError(f"{what} must be {E} contiguous uint8 matrices [{rows}, {cols}] on {dev}")
    return _ptr_array(ts)


def mxfp4_grouped_gemm(a: torch.Tensor, a_scale: torch.Tensor, w, w_scale, split_sizes: Optional[torch.Tensor] = None,
                       group_offsets: Optional[torch.Tensor] = None, out_dtype: str = "bf16",
                       total_rows: Optional[int] = None, out: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out[r] = a[r] w_e^T for the rows r of every expert e, on MXFP4 weights.
    a: MXFP8 codes [rows, K] or MXFP4 codes [rows, K/2], told apart by a_scale [rows, K/32]; w: MXFP4 codes
    [E, N, K/2] with w_scale [E, N, K/32] (stacked, or a sequence of E matrices).  split_sizes int32 [E] and
    group_offsets int32 [E] or [E+1]: the groups' row counts and first rows (absent with one expert: all rows).
    total_rows: rows in all groups at most, where the caller knows fewer than `rows` (T * k).  Rows outside the
    groups are left as they were.  For the input gradient pass the column form of the weight."""
    if out_dtype not in DTYPE:
        raise ValueError(f"out_dtype must be 'bf16' or 'f32', not {out_dtype!r}")
    if a.dim() != 2 or a_scale.dim() != 2 or not _is_u8(a) or not _is_u8(a_scale):
        raise ValueError("a and a_scale must be contiguous uint8 [rows, ...]")
    rows, ka = a.shape
    K = a_scale.shape[1] * 32
    if a_scale.shape[0] != rows or K == 0 or (ka != K and ka != K // 2):
        raise ValueError("a must be [rows, K] (MXFP8) or [rows, K/2] (MXFP4) with a_scale [rows, K/32]")
    E = len(w)
    stacked = isinstance(w, torch.Tensor)
    if E < 1 or len(w_scale) != E or (w.dim() != 3 if stacked else w[0].dim() != 2):
        raise ValueError("w must be [E, N, K/2] with w_scale [E, N, K/32]")
    N = w.shape[1] if stacked else w[0].shape[0]
    _need(workspace is None or workspace.is_contiguous(), "workspace must be contiguous")
    dev = a.device
    dt = torch.bfloat16 if out_dtype == "bf16" else torch.float32
    _on(dev, a_scale, out, split_sizes, group_offsets, workspace)
    if out is None:
        out = a.new_empty((rows, N), dtype=dt)
    elif out.shape != (rows, N) or out.dtype != dt or not out.is_contiguous():
        raise ValueError("out has another shape or dtype")
    for t in (split_sizes, group_offsets):
        if t is not None and (t.dtype != torch.int32 or not t.is_contiguous() or t.numel() < E):
            raise ValueError("split_sizes and group_offsets must be contiguous int32 with an entry for each expert")
    wp = _expert_ptrs(w, E, N, K // 2, dev, "w")
    wsp = _expert_ptrs(w_scale, E, N, K // 32, dev, "w_scale")
    g = Gemm4Args(C.sizeof(Gemm4Args), FORMAT["mxfp8"] if ka == K else FORMAT["mxfp4"], E, N, K, rows, total_rows or 0,
                  _ptr(split_sizes), _ptr(group_offsets), a.data_ptr(), a_scale.data_ptr(), C.addressof(wp),
                  C.addressof(wsp), DTYPE[out_dtype], out.data_ptr())
    if workspace is None:
        need = lib().mge_gemm4_workspace_bytes(C.byref(g))
        if need:
            workspace = a.new_empty(need)
    if workspace is not None:
        g.workspace, g.workspace_bytes = workspace.data_ptr(), workspace.numel()
    _call("mxfp4_grouped_gemm", g, dev)
    return out


def grouped_mlp_fwd_mxfp4(rt: RouteOut, w_gate_up, w_down, w_gate_up_scale, w_down_scale, y_dtype: str = "bf16",
                          out: Optional[FwdOut] = None) -> FwdOut:
    """grouped_mlp_fwd for serving on MXFP4 weights: w_gate_up [E, 2F, H/2] and w_down [E, H, F/2] are mxfp4_quantize
    row codes with their scales; `rt` is an MXFP8 route (activations and h stay in MXFP8)."""
    _need(rt.prec == "mxfp8" and rt.x_perm is not None and rt.x_perm_scale is not None,
          "the route must be prec='mxfp8' and carry the permuted activations and their scales")
    _need(y_dtype in DTYPE, f"y_dtype must be 'bf16' or 'f32', not {y_dtype!r}")
    E, H, R = rt.E, rt.H, rt.R
    F = (w_gate_up.shape[1] if isinstance(w_gate_up, torch.Tensor) else w_gate_up[0].shape[0]) // 2
    x = rt.x_perm
    dev = x.device
    dt = torch.bfloat16 if y_dtype == "bf16" else torch.float32
    _need(out is None or out.workspace is None or out.workspace.is_contiguous(), "out.workspace must be contiguous")
    _on(dev, rt.x_perm_scale, rt.split_sizes, rt.group_offsets, rt.prob_perm)
    if out is None:
        out = FwdOut(y_perm=x.new_empty((R, H), dtype=dt), h=x.new_empty((R, F)), h_scale=x.new_empty((R, F // 32)))
    else:
        _on(dev, out.y_perm, out.h, out.h_scale, out.workspace)
        _need(tuple(out.y_perm.shape) == (R, H) and out.y_perm.dtype == dt and out.y_perm.is_contiguous(),
              "out.y_perm has another shape or dtype")
        _need(out.h is None or (tuple(out.h.shape) == (R, F) and _is_u8(out.h) and out.h_scale is not None
                                and tuple(out.h_scale.shape) == (R, F // 32) and _is_u8(out.h_scale)),
              "out.h / out.h_scale have another shape or dtype")
    keep = [_expert_ptrs(w_gate_up, E, 2 * F, H // 2, dev, "w_gate_up"),
            _expert_ptrs(w_down, E, H, F // 2, dev, "w_down"),
            _expert_ptrs(w_gate_up_scale, E, 2 * F, H // 32, dev, "w_gate_up_scale"),
            _expert_ptrs(w_down_scale, E, H, F // 32, dev, "w_down_scale")]
    a = FwdArgs(C.sizeof(FwdArgs), PREC["mxfp8"], E, H, F, rt.T, rt.k, rt.align, _ptr(rt.split_sizes),
                _ptr(rt.group_offsets), _ptr(rt.prob_perm), _ptr(x), _ptr(rt.x_perm_scale), C.addressof(keep[0]),
                C.addressof(keep[2]), C.addressof(keep[1]), C.addressof(keep[3]), DTYPE[y_dtype], _ptr(out.y_perm),
                _ptr(out.h), _ptr(out.h_scale))
    if out.workspace is None:
        need = lib().mge_fwd_mxfp4_workspace_bytes(C.byref(a))
        if need:
            out.workspace = x.new_empty(need)
    if out.workspace is not None:
        a.workspace, a.workspace_bytes = out.workspace.data_ptr(), out.workspace.numel()
    _call("grouped_mlp_fwd_mxfp4", a, dev)
    return out


# ------------------------------------------------------------------------------ norm

@dataclass
class RmsnormOut:
    y: Optional[torch.Tensor] = None
    codes: Optional[torch.Tensor] = None
    scales: Optional[torch.Tensor] = None
    residual: Optional[torch.Tensor] = None
    rstd: Optional[torch.Tensor] = None


def _int32(sizes: int, what: str):
    """Refuses sizes (or-ed together) that the argument blocks' 32-bit fields would cut off."""
    if sizes >> 31:
        raise ValueError(f"{what} must be below 2^31")


def _rows_of(t: torch.Tensor, what: str):
    """[..., H] as rows: (T, H, row stride) of a contiguous tensor, or of a matrix of contiguous rows."""
    if t.dim() < 1 or t.dtype not in _TORCH_DTYPE:
        raise ValueError(f"{what} must be [..., H], float32 or bfloat16")
    H = t.shape[-1]
    if t.is_contiguous():
        T, ld = (t.numel() // H if H else 0), H
    elif t.dim() != 2 or t.stride(1) != 1:
        raise ValueError(f"{what} must be contiguous, or a matrix of contiguous rows")
    else:
        T = t.shape[0]
        ld = t.stride(0) if T > 1 else H
    _int32(T | H, f"the rows and columns of {what}")
    return T, H, ld


def _like(t, shape, dtype, what: str):
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous {dtype} {list(shape)}")


def _new_like(x, dtype):
    """A new contiguous tensor of x's shape (empty_like is the quickest way there is, where it gives that)."""
    return torch.empty_like(x, dtype=dtype) if x.is_contiguous() else x.new_empty(x.shape, dtype=dtype)


def _fblocks(n: int) -> int:
    return (n + 127) // 128


def rmsnorm_fwd(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, residual: Optional[torch.Tensor] = None,
                form: Optional[str] = None, want_y: bool = True, y_dtype: str = "bf16",
                out: Optional[RmsnormOut] = None) -> RmsnormOut:
    """y = r * rstd * weight with r = x + residual and rstd = 1 / sqrt(mean(r^2) + eps) over the last axis.
    x: [..., H] bf16 or fp32, contiguous or a matrix of strided rows; residual: the same type, contiguous; weight: [H]
    bf16 or fp32.  -> RmsnormOut: y (bf16 or f32 by y_dtype; None without want_y), residual (r, rounded to x's type;
    None without a residual), rstd fp32 [...] and with form="fp8_block" codes uint8 [..., H] and scales fp32
    [..., ceil(H / 128)], the 1x128 row form of the unrounded y.  out: the tensors to write into (out.residual may be
    `residual` itself); those absent there are not written."""
    T, H, ld = _rows_of(x, "x")
    if form not in (None, "fp8_block"):
        raise ValueError(f"form must be None or 'fp8_block', not {form!r}")
    if y_dtype not in DTYPE:
        raise ValueError(f"y_dtype must be 'bf16' or 'f32', not {y_dtype!r}")
    dev, lead = x.device, tuple(x.shape[:-1])
    ydt = torch.bfloat16 if y_dtype == "bf16" else torch.float32
    _on(dev, weight, residual)
    if weight.dim() != 1 or weight.shape[0] != H or weight.dtype not in _TORCH_DTYPE or not weight.is_contiguous():
        raise ValueError("weight must be contiguous [H], float32 or bfloat16")
    if residual is not None:
        _like(residual, x.shape, x.dtype, "residual")
    if out is None:
        _need(want_y or form is not None, "no output asked for (want_y or form)")
        f32 = torch.float32
        out = RmsnormOut(y=_new_like(x, ydt) if want_y else None,
                         residual=None if residual is None else _new_like(x, x.dtype), rstd=x.new_empty(lead, dtype=f32))
        if form is not None:
            out.codes, out.scales = _new_like(x, torch.uint8), x.new_empty(lead + (_fblocks(H),), dtype=f32)
    else:
        _on(dev, out.y, out.codes, out.scales, out.residual, out.rstd)
        _need((residual is None) == (out.residual is None), "out.residual goes with residual")
        for t, shape, dt, what in ((out.y, x.shape, ydt, "out.y"), (out.codes, x.shape, torch.uint8, "out.codes"),
                                   (out.scales, lead + (_fblocks(H),), torch.float32, "out.scales"),
                                   (out.residual, x.shape, x.dtype, "out.residual"), (out.rstd, lead, torch.float32, "out.rstd")):
            if t is not None:
                _like(t, shape, dt, what)
    a = RmsnormArgs(C.sizeof(RmsnormArgs), T, H, _TORCH_DTYPE[x.dtype], _TORCH_DTYPE[weight.dtype], DTYPE[y_dtype], eps, ld,
                    x.data_ptr(), _ptr(residual), weight.data_ptr(), _ptr(out.residual), _ptr(out.y), _ptr(out.codes),
                    _ptr(out.scales), _ptr(out.rstd))
    _call("rmsnorm_fwd", a, dev)
    return out


def rmsnorm_bwd(dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                d_residual: Optional[torch.Tensor] = None, want_dw: bool = True, out=None):
    """(dx, d_weight) of rmsnorm_fwd: x is what the norm was taken of (the forward's residual, or x without one), rstd
    the forward's.  dx has x's type, d_residual (x's type) added: the gradient of x and of the residual alike.
    d_weight: fp32 [H], None without want_dw.  out: the pair to write into."""
    T, H, ld = _rows_of(x, "x")
    Ty, Hy, dld = _rows_of(dy, "dy")
    _need(tuple(dy.shape) == tuple(x.shape), "dy must have x's shape")
    dev, lead = x.device, tuple(x.shape[:-1])
    _on(dev, dy, weight, rstd, d_residual)
    if weight.dim() != 1 or weight.shape[0] != H or weight.dtype not in _TORCH_DTYPE or not weight.is_contiguous():
        raise ValueError("weight must be contiguous [H], float32 or bfloat16")
    _like(rstd, lead, torch.float32, "rstd")
    if d_residual is not None:
        _like(d_residual, x.shape, x.dtype, "d_residual")
    if out is None:
        dx, dw = _new_like(x, x.dtype), x.new_empty(H, dtype=torch.float32) if want_dw else None
    else:
        dx, dw = out
        _on(dev, dx, dw)
        _like(dx, x.shape, x.dtype, "dx")
        if dw is not None:
            _like(dw, (H,), torch.float32, "d_weight")
    need = lib().mge_rmsnorm_bwd_workspace_bytes(T, H) if dw is not None else 0
    ws = x.new_empty(need, dtype=torch.uint8) if need else None
    a = RmsnormBwdArgs(C.sizeof(RmsnormBwdArgs), T, H, _TORCH_DTYPE[x.dtype], _TORCH_DTYPE[weight.dtype],
                       _TORCH_DTYPE[dy.dtype], ld, dld, dy.data_ptr(), x.data_ptr(), weight.data_ptr(), rstd.data_ptr(),
                       _ptr(d_residual), dx.data_ptr(), _ptr(dw), _ptr(ws), need)
    _call("rmsnorm_bwd", a, dev)
    return dx, dw


# ------------------------------------------------------------------------------ FP8, blocks of 128

def _is_f32(t) -> bool:
    return t.dtype == torch.float32 and t.is_contiguous()


def fp8_block_quantize(x: torch.Tensor, orient: str = "row", block: str = "1x128", rows: Optional[torch.Tensor] = None,
                       out=None):
    """BF16 [..., R, C] -> (row_codes, row_scales, col_codes, col_scales) in E4M3 with one fp32 scale per block of 128
    (absent ones None).  block "1x128": scales [..., R, ceil(C/128)], and of the transposed form codes [..., C, Rp] (R
    padded to 32) with scales [..., C, ceil(R/128)]; block "128x128": scales [..., ceil(R/128), ceil(C/128)], the
    transposed form's the transpose.  orient "row", "col" or "both".  rows: int32 map of the output's rows (a 1x128
    matrix): row r is x[rows[r]], zeros where that is outside x.  x: contiguous, or a matrix of strided rows."""
    shape = x.shape
    if x.dtype != torch.bfloat16 or len(shape) < 2:
        raise ValueError("x must be bfloat16 [..., R, C]")
    if orient not in ("row", "col", "both"):
        raise ValueError(f"orient must be 'row', 'col' or 'both', not {orient!r}")
    if block not in BLOCK:
        raise ValueError(f"block must be '1x128' or '128x128', not {block!r}")
    src, Cc = shape[-2], shape[-1]
    ld = Cc
    if not x.is_contiguous():
        if len(shape) != 2 or (Cc > 1 and x.stride(1) != 1) or (src > 1 and x.stride(0) < Cc):
            raise ValueError("x must be contiguous, or a matrix of contiguous rows")
        ld = x.stride(0) if src > 1 else Cc
    lead = tuple(shape[:-2])
    batch = 1
    for d in lead:
        batch *= d
    dev = x.device
    R = src
    if rows is not None:
        _need(rows.dim() == 1 and rows.dtype == torch.int32 and rows.is_contiguous(), "rows must be contiguous int32 [R]")
        _need(len(shape) == 2 and block == "1x128", "rows needs a matrix and block='1x128'")
        R = rows.shape[0]
    _int32(batch | R | Cc, "batch, rows and columns")
    _on(dev, rows)
    Rp, nr, nc = (R + 31) // 32 * 32, _fblocks(R), _fblocks(Cc)
    want_row, want_col = orient != "col", orient != "row"
    tile = block == "128x128"
    shapes = ((R, Cc), (nr, nc) if tile else (R, nc), (Cc, Rp), (nc, nr) if tile else (Cc, nr))
    used = (want_row, want_row, want_col, want_col)
    if out is None:
        dts = (torch.uint8, torch.float32, torch.uint8, torch.float32)
        out = [x.new_empty(lead + s, dtype=dt) if u else None for s, dt, u in zip(shapes, dts, used)]
    else:
        _on(dev, *out)
        for i, (t, s, u) in enumerate(zip(out, shapes, used)):
            _need(not u or (t is not None and tuple(t.shape) == lead + s and (_is_f32(t) if i & 1 else _is_u8(t))),
                  "out must be contiguous uint8 codes and float32 scales of the outputs' sizes")
    rc, rs, cc, cs = (t if u else None for t, u in zip(out, used))
    a = QuantFbArgs(C.sizeof(QuantFbArgs), BLOCK[block], batch, R, Cc, src * ld, ld, x.data_ptr(), _ptr(rows), src,
                    (ORIENT_ROW if want_row else 0) | (ORIENT_COL if want_col else 0), _ptr(rc), _ptr(rs), _ptr(cc), _ptr(cs))
    _call("fp8_block_quantize", a, dev)
    return rc, rs, cc, cs


def fp8_block_dequantize(codes: torch.Tensor, scales: torch.Tensor, out_dtype: str = "bf16",
                         out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Values [..., R, C] (bf16 or f32) of E4M3 codes uint8 [..., R, C] and their fp32 scales, [..., R, ceil(C/128)] or
    [..., ceil(R/128), ceil(C/128)] (told apart by their shape)."""
    if out_dtype not in DTYPE:
        raise ValueError(f"out_dtype must be 'bf16' or 'f32', not {out_dtype!r}")
    if codes.dim() < 2 or not _is_u8(codes) or not _is_f32(scales):
        raise ValueError("codes must be contiguous uint8 [..., R, C], scales contiguous float32")
    lead, R, Cc = tuple(codes.shape[:-2]), codes.shape[-2], codes.shape[-1]
    rowwise = tuple(scales.shape) == lead + (R, _fblocks(Cc))
    if not rowwise and tuple(scales.shape) != lead + (_fblocks(R), _fblocks(Cc)):
        raise ValueError("scales must be [..., R, ceil(C/128)] or [..., ceil(R/128), ceil(C/128)]")
    batch = 1
    for d in lead:
        batch *= d
    _int32(batch | R | Cc, "batch, rows and columns")
    dev = codes.device
    dt = torch.bfloat16 if out_dtype == "bf16" else torch.float32
    _on(dev, scales, out)
    if out is None:
        out = _new_like(codes, dt)
    else:
        _like(out, codes.shape, dt, "out")
    a = DequantFbArgs(C.sizeof(DequantFbArgs), BLOCK["1x128" if rowwise else "128x128"], batch, R, Cc, DTYPE[out_dtype],
                      codes.data_ptr(), scales.data_ptr(), out.data_ptr())
    _call("fp8_block_dequantize", a, dev)
    return out


def _expert_ptrs_of(w, E: int, rows: int, cols: int, dev, dtype, what: str):
    """_expert_ptrs for matrices of any type."""
    if isinstance(w, torch.Tensor):
        if w.shape != (E, rows, cols) or w.dtype != dtype or not w.is_contiguous() or w.device != dev:
            raise ValueError(f"{what} must be contiguous {dtype} [{E}, {rows}, {cols}] on {dev}")
        p, n = w.data_ptr(), rows * cols * w.element_size()
        return (vp * E)(*range(p, p + E * n, n)) if E > 1 and n else (vp * E)(*[p] * E)
    ts = list(w)
    if len(ts) != E or not all(t.shape == (rows, cols) and t.dtype == dtype and t.is_contiguous() and t.device == dev for t in ts):
        raise ValueError(f"{what} must be {E} contiguous {dtype} matrices [{rows}, {cols}] on {dev}")
    return _ptr_array(ts)


def _check_groups(split_sizes, group_offsets, E: int):
    for t in (split_sizes, group_offsets):
        if t is not None and (t.dtype != torch.int32 or not t.is_contiguous() or t.numel() < E):
            raise ValueError("split_sizes and group_offsets must be contiguous int32 with an entry for each expert")


def _codes_rows(a, a_scale, what: str):
    if a.dim() != 2 or not _is_u8(a) or not _is_f32(a_scale) or tuple(a_scale.shape) != (a.shape[0], _fblocks(a.shape[1])):
        raise ValueError(f"{what} must be contiguous uint8 [rows, K] with float32 scales [rows, ceil(K/128)]")
    _int32(a.shape[0] | a.shape[1], f"the rows and columns of {what}")
    return a.shape


def _work(need: int, ws, like):
    """The workspace of a call: the caller's, or a new one of the bytes it needs."""
    if ws is not None:
        _need(ws.is_contiguous(), "workspace must be contiguous")
        return ws
    return like.new_empty(need, dtype=torch.uint8) if need else None


def fp8_block_grouped_gemm(a: torch.Tensor, a_scale: torch.Tensor, w, w_scale, split_sizes: Optional[torch.Tensor] = None,
                           group_offsets: Optional[torch.Tensor] = None, a_rows: Optional[torch.Tensor] = None,
                           out_dtype: str = "bf16", total_rows: Optional[int] = None, out: Optional[torch.Tensor] = None,
                           workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out[r] = a[r] w_e^T for the rows r of every expert e, in FP8 with one fp32 scale per block of 128.
    a: E4M3 codes [rows, K] with a_scale [rows, ceil(K/128)]; w: codes [E, N, K] with w_scale [E, ceil(N/128),
    ceil(K/128)] (stacked, or sequences of E matrices).  a_rows: int32 [rows of out], row r then reads a[a_rows[r]]
    (zeros where that is outside a): a route's perm_src.  split_sizes, group_offsets, total_rows: as
    mxfp4_grouped_gemm.  Rows outside the groups are left as they were.  For the input gradient pass the transposed
    form of the weight.  A block's two scales are multiplied in fp32: past its range the elements that add the two
    blocks are infinite or NaN."""
    if out_dtype not in DTYPE:
        raise ValueError(f"out_dtype must be 'bf16' or 'f32', not {out_dtype!r}")
    src, K = _codes_rows(a, a_scale, "a")
    dev = a.device
    _on(dev, a_scale, out, split_sizes, group_offsets, a_rows, workspace)
    if isinstance(w, torch.Tensor):
        shape = w.shape
        _need(len(shape) == 3 and shape[0] > 0, "w must be [E, N, K]")
        E, N = shape[0], shape[1]
    else:
        E = len(w)
        _need(E > 0 and w[0].dim() == 2, "w must be E matrices [N, K]")
        N = w[0].shape[0]
    _int32(N, "N")
    rows = src
    if a_rows is not None:
        _need(a_rows.dim() == 1 and a_rows.dtype == torch.int32 and a_rows.is_contiguous(), "a_rows must be contiguous int32 [rows]")
        rows = a_rows.shape[0]
    _check_groups(split_sizes, group_offsets, E)
    dt = torch.bfloat16 if out_dtype == "bf16" else torch.float32
    if out is None:
        out = a.new_empty((rows, N), dtype=dt)
    else:
        _like(out, (rows, N), dt, "out")
    wp = _expert_ptrs_of(w, E, N, K, dev, torch.uint8, "w")
    wsp = _expert_ptrs_of(w_scale, E, _fblocks(N), _fblocks(K), dev, torch.float32, "w_scale")
    g = GemmFbArgs(C.sizeof(GemmFbArgs), E, N, K, rows, total_rows or 0, _ptr(split_sizes), _ptr(group_offsets), _ptr(a_rows),
                   src, a.data_ptr(), a_scale.data_ptr(), C.addressof(wp), C.addressof(wsp), DTYPE[out_dtype], out.data_ptr())
    ws = _work(lib().mge_gemm_fb_workspace_bytes(C.byref(g)), workspace, a)
    if ws is not None:
        g.workspace, g.workspace_bytes = ws.data_ptr(), ws.numel() * ws.element_size()
    _call("fp8_block_grouped_gemm", g, dev)
    return out


def fp8_block_grouped_wgrad(dy: torch.Tensor, dy_scale: torch.Tensor, x: torch.Tensor, x_scale: torch.Tensor,
                            split_sizes: Optional[torch.Tensor] = None, group_offsets: Optional[torch.Tensor] = None,
                            out_dtype: str = "f32", accumulate: bool = False, out=None,
                            workspace: Optional[torch.Tensor] = None):
    """dw [E, N, K] (f32 or bf16): the gradient of every expert's weight [N, K] from the transposed forms of the
    permuted dY, codes [N, rows] with dy_scale [N, ceil(rows/128)], and X, [K, rows] with [K, ceil(rows/128)]
    (fp8_block_quantize "col").  split_sizes, group_offsets: the groups, at multiples of 128 rows (align=128), with
    zero rows after each up to the next multiple of 32; absent: one expert, all rows.  out: [E, N, K], or a sequence of
    E matrices; accumulate adds to it (f32)."""
    if out_dtype not in DTYPE:
        raise ValueError(f"out_dtype must be 'bf16' or 'f32', not {out_dtype!r}")
    N, rows = _codes_rows(dy, dy_scale, "dy")
    K, xrows = _codes_rows(x, x_scale, "x")
    _need(xrows == rows, "dy and x must have the same rows")
    dev = dy.device
    _on(dev, dy_scale, x, x_scale, split_sizes, group_offsets, workspace)
    E = 1 if split_sizes is None else split_sizes.numel()
    _check_groups(split_sizes, group_offsets, E)
    dt = torch.bfloat16 if out_dtype == "bf16" else torch.float32
    if out is None:
        _need(not accumulate, "accumulate needs out")
        out = dy.new_empty((E, N, K), dtype=dt)
    ptrs = _expert_ptrs_of(out, E, N, K, dev, dt, "out")
    g = WgradFbArgs(C.sizeof(WgradFbArgs), E, N, K, rows, _ptr(split_sizes), _ptr(group_offsets), dy.data_ptr(),
                    dy_scale.data_ptr(), x.data_ptr(), x_scale.data_ptr(), DTYPE[out_dtype], 1 if accumulate else 0,
                    C.addressof(ptrs))
    ws = _work(lib().mge_wgrad_fb_workspace_bytes(C.byref(g)), workspace, dy)
    if ws is not None:
        g.workspace, g.workspace_bytes = ws.data_ptr(), ws.numel() * ws.element_size()
    _call("fp8_block_grouped_wgrad", g, dev)
    return out


def grouped_mlp_fwd_fp8_block(rt: Optional[RouteOut], x: torch.Tensor, x_scale: torch.Tensor, w_gate_up, w_down, w_gate_up_scale,
                              w_down_scale, y_dtype: str = "bf16", out: Optional[FwdOut] = None) -> FwdOut:
    """The expert MLP for serving on weights in FP8 with one fp32 scale per block of 128: w_gate_up [E, 2F, H] and w_down
    [E, H, F] E4M3 codes with their scales ([E, ceil(2F/128), ceil(H/128)], [E, ceil(H/128), ceil(F/128)]).
    x: codes [T, H] with x_scale [T, ceil(H/128)], one row a token (rmsnorm_fwd, fp8_block_quantize); the route's maps
    (moe_route_permute with x=None will do) gather them.  rt None: one expert that all rows of x go through, with weight
    1 (a dense gated MLP).  -> FwdOut with y_perm [R, H] ([T, H] without a route)."""
    _need(y_dtype in DTYPE, f"y_dtype must be 'bf16' or 'f32', not {y_dtype!r}")
    T, H = _codes_rows(x, x_scale, "x")
    dev = x.device
    E = len(w_gate_up) if rt is None else rt.E
    _need(rt is not None or E == 1, "without a route there is one expert")
    _need(rt is None or rt.T == T, "x must have a row for each of the route's tokens")
    R = T if rt is None else rt.R
    F = (w_gate_up.shape[1] if isinstance(w_gate_up, torch.Tensor) else w_gate_up[0].shape[0]) // 2
    _int32(F, "F")
    dt = torch.bfloat16 if y_dtype == "bf16" else torch.float32
    _on(dev, x_scale)
    if rt is not None:
        _on(dev, rt.split_sizes, rt.group_offsets, rt.perm_src, rt.prob_perm)
    if out is None:
        out = FwdOut(y_perm=x.new_empty((R, H), dtype=dt), h=None)
    else:
        _on(dev, out.y_perm, out.workspace)
        _like(out.y_perm, (R, H), dt, "out.y_perm")
    u8, f32 = torch.uint8, torch.float32
    keep = [_expert_ptrs_of(w_gate_up, E, 2 * F, H, dev, u8, "w_gate_up"),
            _expert_ptrs_of(w_gate_up_scale, E, _fblocks(2 * F), _fblocks(H), dev, f32, "w_gate_up_scale"),
            _expert_ptrs_of(w_down, E, H, F, dev, u8, "w_down"),
            _expert_ptrs_of(w_down_scale, E, _fblocks(H), _fblocks(F), dev, f32, "w_down_scale")]
    maps = (None,) * 4 if rt is None else (_ptr(rt.split_sizes), _ptr(rt.group_offsets), _ptr(rt.perm_src), _ptr(rt.prob_perm))
    a = FwdFbArgs(C.sizeof(FwdFbArgs), E, H, F, R, T if rt is None else rt.T * rt.k, *maps, T, x.data_ptr(), x_scale.data_ptr(),
                  *(C.addressof(k) for k in keep), DTYPE[y_dtype], out.y_perm.data_ptr())
    out.workspace = _work(lib().mge_fwd_fb_workspace_bytes(C.byref(a)), out.workspace, x)
    if out.workspace is not None:
        a.workspace, a.workspace_bytes = out.workspace.data_ptr(), out.workspace.numel() * out.workspace.element_size()
    _call("grouped_mlp_fwd_fp8_block", a, dev)
    return out
