"""Python binding of libmoe, the MI355X MoE expert layer (argument marshalling only).

Every function here has the name of a C entry point in include/moe.h and does
nothing but check tensor shapes/dtypes on the host, pass `data_ptr()`s, sizes
and the current HIP stream to the library, and raise on a non-OK status. All
arithmetic runs in the library's HIP kernels. The library is loaded from this
package's directory; if it is missing, importing the binding raises (there is
no fallback path).

`MoELayer` strings the calls together in the layer's order (route -> permute
-> grouped GEMM + SwiGLU -> grouped GEMM -> combine; `moe_backward`) and owns
the saved tensors and intermediates as torch allocations.
"""
from __future__ import annotations

import array
import ctypes
import operator
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe.so")

MOE_OK, MOE_ERR_NULL, MOE_ERR_SHAPE, MOE_ERR_DTYPE, MOE_ERR_ALIGN, MOE_ERR_WORKSPACE, \
    MOE_ERR_LAUNCH = range(7)
MOE_F32, MOE_BF16, MOE_MXFP8 = 0, 1, 2
MOE_GG_FWD, MOE_GG_DGRAD, MOE_GG_WGRAD = 0, 1, 2
MOE_EPI_NONE, MOE_EPI_SWIGLU_FWD, MOE_EPI_SWIGLU_BWD = 0, 1, 2

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I32 = ctypes.c_int32
_SZ = ctypes.c_size_t


class MoeError(RuntimeError):
    def __init__(self, fn, status):
        super().__init__(f"{fn}: {_lib.moe_status_str(status).decode()} (status {status})")
        self.status = status


class GemmDesc(ctypes.Structure):
    _fields_ = [("mode", _I32), ("dtype", _I32), ("epilogue", _I32), ("n_groups", _I32),
                ("rows", _I64), ("M", _I32), ("N", _I32), ("K", _I32),
                ("offsets", _P), ("A", _P), ("B", _P), ("C", _P), ("a_scale", _P),
                ("b_scale", _P), ("aux", _P), ("aux_out", _P), ("aux_out_scale", _P),
                ("ws", _P), ("ws_bytes", _SZ), ("accumulate", _I32), ("aux_out_cols", _P),
                ("aux_out_cols_scale", _P)]


class BwdDesc(ctypes.Structure):
    _fields_ = [("dtype", _I32), ("d", _I32), ("h", _I32), ("E", _I32), ("k", _I32), ("T", _I64),
                ("x_perm", _P), ("ab", _P), ("hp", _P), ("y_perm", _P), ("topk_gate", _P),
                ("topk_idx", _P), ("token_pos", _P), ("offsets", _P), ("w1", _P), ("w2", _P),
                ("dout", _P), ("dx", _P), ("dlogits", _P), ("dw1", _P), ("dw2", _P),
                ("dgate", _P), ("dy_perm", _P), ("dab", _P), ("dx_perm", _P), ("x", _P),
                ("sorted_token", _P), ("w1t", _P), ("w1t_scale", _P), ("w2t", _P),
                ("w2t_scale", _P), ("ws", _P), ("ws_bytes", _SZ), ("accumulate_dw", _I32),
                ("stage_events", ctypes.POINTER(_P)), ("hp_cols", _P), ("hp_cols_scale", _P)]

class CopyWalk(ctypes.Structure):
    _fields_ = [("extent", _I64 * 4), ("copies", _I64), ("zero_copies", _I64),
                ("lowest", _I64 * 4), ("end", _I64 * 4), ("first_bad", _I32),
                ("bad_offset", _I64), ("bad_bytes", _I64)]


class Act8Saved(ctypes.Structure):
    _fields_ = [("ab8", _P), ("ab8_scale", _P), ("y8", _P), ("y8_scale", _P)]


class W4Desc(ctypes.Structure):
    _fields_ = [("d", _I32), ("h", _I32), ("E", _I32), ("k", _I32), ("T", _I64), ("x", _P),
                ("topk_gate", _P), ("token_pos", _P), ("sorted_token", _P), ("offsets", _P),
                ("w1q", _P), ("w1_scale", _P), ("w2q", _P), ("w2_scale", _P), ("out", _P),
                ("ws", _P), ("ws_bytes", _SZ)]


class W4GemmDesc(ctypes.Structure):
    _fields_ = [("n_groups", _I32), ("epilogue", _I32), ("rows", _I64), ("N", _I32), ("K", _I32),
                ("offsets", _P), ("a_rows", _P), ("a", _P), ("a_scale", _P), ("b", _P),
                ("b_scale", _P), ("c", _P), ("c_scale", _P)]


class BwdWsLayout(ctypes.Structure):
    _fields_ = [(n, _SZ) for n in ("row_q", "row_s", "col0_q", "col0_s", "col1_q", "col1_s",
                                   "total")]


MOE_BWD_MAX_STAGES = 10
BWD_STAGES = {
    "bf16": ("combine_bwd", "gemm2_dgrad_swiglu", "gemm2_wgrad", "gemm1_dgrad", "unpermute_bwd",
             "gemm1_wgrad"),
    "mxfp8": ("combine_bwd", "quant_dy_both", "gemm2_dgrad_swiglu", "quant_hp_cols", "gemm2_wgrad",
              "quant_dab_both", "gemm1_dgrad", "unpermute_bwd", "quant_x_cols", "gemm1_wgrad"),
}


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python -m routing_grouped_gemm_router_amd.build` "
            "(the MoE layer has no non-HIP path)")
    lib = ctypes.CDLL(LIB_PATH)
    lib.moe_status_str.argtypes = [_I32]
    lib.moe_status_str.restype = ctypes.c_char_p
    lib.moe_version.restype = _I32
    lib.moe_route_workspace_size.argtypes = [_I64, _I32, _I32]
    lib.moe_route_workspace_size.restype = _SZ
    lib.moe_route.argtypes = [_P, _I64, _I32, _I32, _I32] + [_P] * 9 + [_SZ, _P]
    lib.moe_route.restype = _I32
    lib.moe_route_noalloc.argtypes = [_P, _I64, _I32, _I32, _I32] + [_P] * 9
    lib.moe_route_noalloc.restype = _I32
    lib.moe_permute.argtypes = [_P, _P, _I32, _I64, _I32, _I32, _P, _P, _P, _P]
    lib.moe_permute.restype = _I32
    lib.moe_combine.argtypes = [_P, _I32, _P, _P, _I64, _I32, _I32, _P, _P]
    lib.moe_combine.restype = _I32
    lib.moe_grouped_gemm.argtypes = [ctypes.POINTER(GemmDesc), _P]
    lib.moe_grouped_gemm.restype = _I32
    lib.moe_grouped_gemm_workspace_size.argtypes = [ctypes.POINTER(GemmDesc)]
    lib.moe_grouped_gemm_workspace_size.restype = _SZ
    lib.moe_backward.argtypes = [ctypes.POINTER(BwdDesc), _P]
    lib.moe_backward.restype = _I32
    lib.moe_backward_workspace_size.argtypes = [ctypes.POINTER(BwdDesc)]
    lib.moe_backward_workspace_size.restype = _SZ
    lib.moe_backward_workspace_layout.argtypes = [ctypes.POINTER(BwdDesc), ctypes.POINTER(BwdWsLayout)]
    lib.moe_backward_workspace_layout.restype = _I32
    lib.moe_gemm_copy_walk.argtypes = [ctypes.POINTER(GemmDesc), _P, ctypes.POINTER(CopyWalk)]
    lib.moe_gemm_copy_walk.restype = _I32
    lib.moe_gemm_hp_store_walk.argtypes = [ctypes.POINTER(GemmDesc), _P, ctypes.POINTER(CopyWalk)]
    lib.moe_gemm_hp_store_walk.restype = _I32
    lib.mxfp8_quantize.argtypes = [_P, _I32, _I64, _I64, _I32, _P, _I32, _P, _P, _P, _P]
    lib.mxfp8_quantize.restype = _I32
    lib.mxfp8_col_blocks.argtypes = [_I64, _I32]
    lib.mxfp8_col_blocks.restype = _SZ
    lib.mxfp8_quantize_both.argtypes = [_P, _I32, _I64, _I64, _P, _I32, _P, _P, _P, _P, _P]
    lib.mxfp8_quantize_both.restype = _I32
    lib.moe_capacity_pad.argtypes = [_P, _P, _P, _I64, _I32, _I32, _I32, _P, _P, _P]
    lib.moe_capacity_pad.restype = _I32
    lib.moe_capacity_zero_rows.argtypes = [_P, _I32, _P, _I32, _I32, _I32, _P]
    lib.moe_capacity_zero_rows.restype = _I32
    lib.moe_load_balance_workspace_size.argtypes = [_I64, _I32]
    lib.moe_load_balance_workspace_size.restype = _SZ
    lib.moe_load_balance.argtypes = [_P, _P, _I64, _I32, _I32, ctypes.c_float, _P, _P, _P, _SZ, _P]
    lib.moe_load_balance.restype = _I32
    lib.moe_act8_store.argtypes = [_P, _I32, _I64, _I64, _P, _P, _P]
    lib.moe_act8_store.restype = _I32
    lib.moe_act8_load.argtypes = [_P, _P, _I32, _I64, _I64, _P, _P]
    lib.moe_act8_load.restype = _I32
    lib.moe_act8_swiglu.argtypes = [_P, _P, _I32, _I64, _I32, _P, _P, _P]
    lib.moe_act8_swiglu.restype = _I32
    lib.moe_combine_act8.argtypes = [_P, _I32, _P, _P, _I64, _I32, _I32, _P, _P, _P, _P]
    lib.moe_combine_act8.restype = _I32
    lib.moe_combine_backward_act8.argtypes = [_P, _I32, _P, _P, _P, _P, _P, _I64, _I32, _I32,
                                              _I32, _P, _P, _P, _P]
    lib.moe_combine_backward_act8.restype = _I32
    lib.moe_backward_act8.argtypes = [ctypes.POINTER(BwdDesc), ctypes.POINTER(Act8Saved), _P]
    lib.moe_backward_act8.restype = _I32
    lib.moe_layer_norm.argtypes = [_P, _I32, _P, _P, _P, ctypes.c_float, _I64, _I32, _P, _P, _P,
                                   _P, _P, _P, _P]
    lib.moe_layer_norm.restype = _I32
    lib.moe_layer_norm_backward_workspace_size.argtypes = [_I32, _I64, _I32]
    lib.moe_layer_norm_backward_workspace_size.restype = _SZ
    lib.moe_layer_norm_backward.argtypes = [_P, _I32, _P, _P, _P, _P, _P, _P, _P, _I64, _I32, _P,
                                            _P, _P, _I32, _P, _SZ, _P]
    lib.moe_layer_norm_backward.restype = _I32
    lib.moe_rms_norm.argtypes = [_P, _I32, _P, _P, ctypes.c_float, _I64, _I32, _P, _P, _P, _P, _P,
                                 _P, _P, _P]
    lib.moe_rms_norm.restype = _I32
    lib.moe_rms_norm_backward_workspace_size.argtypes = [_I32, _I64, _I32]
    lib.moe_rms_norm_backward_workspace_size.restype = _SZ
    lib.moe_rms_norm_backward.argtypes = [_P, _I32, _P, _P, _P, _P, _P, _P, _I64, _I32, _P, _P,
                                          _I32, _P, _SZ, _P]
    lib.moe_rms_norm_backward.restype = _I32
    lib.mxfp8_dequantize.argtypes = [_P, _P, _I32, _I64, _I64, _P, _P]
    lib.mxfp8_dequantize.restype = _I32
    lib.moe_grad_norm_workspace_size.argtypes = [_I32]
    lib.moe_grad_norm_workspace_size.restype = _SZ
    lib.moe_grad_norm.argtypes = [_P, _I32, _P, _P, _SZ, _P]
    lib.moe_grad_norm.restype = _I32
    lib.moe_clip_grad_norm.argtypes = [_P, _I32, ctypes.c_float, _P, _P, _SZ, _P]
    lib.moe_clip_grad_norm.restype = _I32
    lib.moe_grad_clip.argtypes = [_P, _I32, _P, ctypes.c_float, _P]
    lib.moe_grad_clip.restype = _I32
    lib.moe_w4_quantize.argtypes = [_P, _I32, _I64, _I64, _P, _P, _P]
    lib.moe_w4_quantize.restype = _I32
    lib.moe_w4_experts_workspace_size.argtypes = [_I64, _I32, _I32, _I32]
    lib.moe_w4_experts_workspace_size.restype = _SZ
    lib.moe_w4_experts.argtypes = [ctypes.POINTER(W4Desc), _P]
    lib.moe_w4_experts.restype = _I32
    lib.moe_w4_gemm.argtypes = [ctypes.POINTER(W4GemmDesc), _P]
    lib.moe_w4_gemm.restype = _I32
    lib.moe_w4_experts8_workspace_size.argtypes = [_I64, _I32, _I32, _I32]
    lib.moe_w4_experts8_workspace_size.restype = _SZ
    lib.moe_w4_experts8.argtypes = [ctypes.POINTER(W4Desc), _P, _P]
    lib.moe_w4_experts8.restype = _I32
    return lib


# torch must be imported first so that libmoe binds to the HIP runtime torch
# already loaded (both carry the soname libamdhip64.so.7)
_lib = _load()


def lib():
    return _lib


def _check(fn, st):
    if st != MOE_OK:
        raise MoeError(fn, st)


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return MOE_F32
    if t.dtype == torch.bfloat16:
        return MOE_BF16
    if t.dtype == torch.uint8:
        return MOE_MXFP8
    raise TypeError(f"unsupported dtype {t.dtype}")


def _need(t, shape, dtype, name):
    if t is None:
        raise ValueError(f"{name} is required")
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype or not t.is_contiguous() or not t.is_cuda:
        raise ValueError(f"{name}: expected contiguous {dtype} {tuple(shape)} on GPU, got "
                         f"{t.dtype} {tuple(t.shape)} (contiguous={t.is_contiguous()}, "
                         f"device={t.device})")


def _need_bytes(t, nbytes, name):
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype != torch.uint8 or not t.is_contiguous() or not t.is_cuda or t.numel() < nbytes:
        raise ValueError(f"{name}: expected a contiguous uint8 GPU buffer of at least {nbytes} "
                         f"bytes, got {t.dtype} {tuple(t.shape)}")


# ---------------------------------------------------------------------------
# entry points (same names as the C ABI)


def moe_route_workspace_size(T: int, E: int, k: int) -> int:
    return int(_lib.moe_route_workspace_size(T, E, k))


def moe_route(logits: torch.Tensor, k: int, tile_m: int = 128, out: dict | None = None,
              ws: torch.Tensor | None = None) -> dict:
    """Top-k routing + metadata (see moe.h). Returns a dict of device tensors."""
    T, E = logits.shape
    dev = logits.device
    R = T * k
    if out is None:
        i32 = dict(dtype=torch.int32, device=dev)
        out = dict(topk_idx=torch.empty((T, k), **i32),
                   topk_gate=torch.empty((T, k), dtype=torch.float32, device=dev),
                   counts=torch.empty(E, **i32), offsets=torch.empty(E + 1, **i32),
                   token_pos=torch.empty((T, k), **i32), sorted_token=torch.empty(R, **i32),
                   sorted_slot=torch.empty(R, **i32), tile_offsets=torch.empty(E + 1, **i32))
    _need(logits, (T, E), torch.float32, "logits")
    wsb = moe_route_workspace_size(T, E, k)
    if ws is None:
        ws = torch.empty(max(wsb, 1), dtype=torch.uint8, device=dev)
    _check("moe_route", _lib.moe_route(
        _p(logits), T, E, k, tile_m, _p(out["topk_idx"]), _p(out["topk_gate"]), _p(out["counts"]),
        _p(out["offsets"]), _p(out["token_pos"]), _p(out["sorted_token"]), _p(out["sorted_slot"]),
        _p(out["tile_offsets"]), _p(ws), ws.numel(), _stream()))
    return out


MOE_ROUTE_NOALLOC_SCRATCH_BYTES = 4 << 20


def moe_route_noalloc(logits: torch.Tensor, k: int, tile_m: int = 128,
                      out: dict | None = None) -> dict:
    """moe_route with the library's own per-GPU scratch (see moe.h): the C
    call allocates nothing. Pass `out` (as moe_route returns) to avoid the
    output allocations here as well."""
    T, E = logits.shape
    dev = logits.device
    R = T * k
    if out is None:
        i32 = dict(dtype=torch.int32, device=dev)
        out = dict(topk_idx=torch.empty((T, k), **i32),
                   topk_gate=torch.empty((T, k), dtype=torch.float32, device=dev),
                   counts=torch.empty(E, **i32), offsets=torch.empty(E + 1, **i32),
                   token_pos=torch.empty((T, k), **i32), sorted_token=torch.empty(R, **i32),
                   sorted_slot=torch.empty(R, **i32), tile_offsets=torch.empty(E + 1, **i32))
    _need(logits, (T, E), torch.float32, "logits")
    _check("moe_route_noalloc", _lib.moe_route_noalloc(
        _p(logits), T, E, k, tile_m, _p(out["topk_idx"]), _p(out["topk_gate"]), _p(out["counts"]),
        _p(out["offsets"]), _p(out["token_pos"]), _p(out["sorted_token"]), _p(out["sorted_slot"]),
        _p(out["tile_offsets"]), _stream()))
    return out


def moe_permute(x: torch.Tensor, token_pos: torch.Tensor, x_perm: torch.Tensor | None = None,
                x_scale: torch.Tensor | None = None, x_perm_scale: torch.Tensor | None = None):
    """x_perm[token_pos[t, j]] = x[t]. For MXFP8 pass uint8 x plus x_scale."""
    T, d = x.shape
    k = token_pos.shape[1]
    if x_perm is None:
        x_perm = torch.empty((T * k, d), dtype=x.dtype, device=x.device)
    dt = _dt(x)
    if dt == MOE_MXFP8 and x_perm_scale is None:
        x_perm_scale = torch.empty((T * k, d // 32), dtype=torch.uint8, device=x.device)
    _check("moe_permute", _lib.moe_permute(_p(x), _p(x_scale), dt, T, d, k, _p(token_pos),
                                           _p(x_perm), _p(x_perm_scale), _stream()))
    return (x_perm, x_perm_scale) if dt == MOE_MXFP8 else x_perm


def moe_combine(y_perm: torch.Tensor, topk_gate: torch.Tensor, token_pos: torch.Tensor,
                out: torch.Tensor | None = None) -> torch.Tensor:
    T, k = token_pos.shape
    d = y_perm.shape[1]
    if out is None:
        out = torch.empty((T, d), dtype=y_perm.dtype, device=y_perm.device)
    _check("moe_combine", _lib.moe_combine(_p(y_perm), _dt(y_perm), _p(topk_gate), _p(token_pos),
                                           T, d, k, _p(out), _stream()))
    return out


def _need_elems(t, n, dtype, name):
    """t is a contiguous GPU tensor of `dtype` with at least n elements."""
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype != dtype or not t.is_contiguous() or not t.is_cuda:
        raise ValueError(f"{name}: expected a contiguous {dtype} GPU tensor, got {t.dtype} "
                         f"(contiguous={t.is_contiguous()}, device={t.device})")
    if t.numel() < n:
        raise ValueError(f"{name}: needs at least {n} elements, has {t.numel()}")


_TORCH_DT = {MOE_F32: torch.float32, MOE_BF16: torch.bfloat16, MOE_MXFP8: torch.uint8}


def _check_gemm_operands(mode, dt, epilogue, A, B, C, offsets, rows, M, N, K, aux, aux_out,
                         a_scale, b_scale, aux_out_scale=None, aux_out_cols=None,
                         aux_out_cols_scale=None):
    """Host-side sizes of every operand against what the mode reads and
    writes (the C ABI sees only pointers, so an undersized tensor would be
    read or written past its end on the device)."""
    E = offsets.numel() - 1
    _need_elems(offsets, E + 1, torch.int32, "offsets")
    hp_quantised = aux_out_scale is not None
    if hp_quantised and (dt != MOE_MXFP8 or epilogue != MOE_EPI_SWIGLU_FWD):
        raise ValueError("aux_out_scale: only the MXFP8 SwiGLU forward stores H' quantised")
    if offsets.device != A.device:
        raise ValueError("offsets must be on A's device")
    et = _TORCH_DT[dt]
    act = torch.bfloat16 if dt == MOE_MXFP8 else et      # stored activations
    if mode == MOE_GG_WGRAD:
        if dt == MOE_MXFP8:
            nb = mxfp8_col_blocks(rows, E)
            _need_elems(A, nb * 32 * M, et, "A")
            _need_elems(B, nb * 32 * N, et, "B")
            _need_elems(a_scale, nb * M, torch.uint8, "a_scale")
            _need_elems(b_scale, nb * N, torch.uint8, "b_scale")
        else:
            _need_elems(A, rows * M, et, "A")
            _need_elems(B, rows * N, et, "B")
        _need_elems(C, E * M * N, torch.float32, "C")
        return
    _need_elems(A, rows * K, et, "A")
    _need_elems(B, E * N * K, et, "B")
    if dt == MOE_MXFP8:
        _need_elems(a_scale, rows * (K // 32), torch.uint8, "a_scale")
        _need_elems(b_scale, E * N * (K // 32), torch.uint8, "b_scale")
    if epilogue == MOE_EPI_SWIGLU_BWD:
        _need_elems(C, rows * 2 * N, act, "C")
        _need_elems(aux, rows * 2 * N, act, "aux")
    else:
        _need_elems(C, rows * N, act, "C")
    if epilogue == MOE_EPI_SWIGLU_FWD:
        if hp_quantised:
            # H' stored as MXFP8 in both layouts instead of bf16
            h, nb = N // 2, mxfp8_col_blocks(rows, E)
            _need_elems(aux_out, rows * h, torch.uint8, "aux_out")
            _need_elems(aux_out_scale, rows * (h // 32), torch.uint8, "aux_out_scale")
            _need_elems(aux_out_cols, nb * 32 * h, torch.uint8, "aux_out_cols")
            _need_elems(aux_out_cols_scale, nb * h, torch.uint8, "aux_out_cols_scale")
        else:
            _need_elems(aux_out, rows * (N // 2), act, "aux_out")


def moe_grouped_gemm(mode: int, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                     offsets: torch.Tensor, epilogue: int = MOE_EPI_NONE, M: int = 0, N: int = 0,
                     K: int = 0, aux: torch.Tensor | None = None,
                     aux_out: torch.Tensor | None = None, a_scale=None, b_scale=None,
                     aux_out_scale=None, dtype: int | None = None, accumulate: bool = False,
                     rows: int | None = None, aux_out_cols=None, aux_out_cols_scale=None):
    """One grouped GEMM (see moe.h for the modes and epilogues). Every
    operand's dtype and size is checked against the mode before the call.
    rows = total routed rows (offsets[-1]); it defaults to A.shape[0] and must
    be given for MXFP8 WGRAD, whose operands are flat column-block arrays.
    MXFP8 SwiGLU forward with aux_out_scale: H' is stored quantised, along h
    into aux_out (uint8 [rows, h]) and aux_out_scale, and along the rows of
    each group into aux_out_cols / aux_out_cols_scale (the layouts
    mxfp8_quantize_both writes)."""
    dt = _dt(A) if dtype is None else dtype
    if dt not in _TORCH_DT:
        raise ValueError(f"unsupported GEMM dtype {dt}")
    if rows is None:
        if mode == MOE_GG_WGRAD and dt == MOE_MXFP8:
            raise ValueError("MXFP8 WGRAD: pass rows (the column-block operands are flat)")
        rows = A.shape[0]
    _check_gemm_operands(mode, dt, epilogue, A, B, C, offsets, rows, M, N, K, aux, aux_out,
                         a_scale, b_scale, aux_out_scale, aux_out_cols, aux_out_cols_scale)
    desc = GemmDesc()
    desc.accumulate = 1 if accumulate else 0
    desc.mode = mode
    desc.dtype = dt
    desc.epilogue = epilogue
    desc.n_groups = offsets.numel() - 1
    desc.rows = rows
    desc.M, desc.N, desc.K = M, N, K
    desc.offsets = offsets.data_ptr()
    desc.A, desc.B, desc.C = A.data_ptr(), B.data_ptr(), C.data_ptr()
    desc.a_scale = a_scale.data_ptr() if a_scale is not None else None
    desc.b_scale = b_scale.data_ptr() if b_scale is not None else None
    desc.aux = aux.data_ptr() if aux is not None else None
    desc.aux_out = aux_out.data_ptr() if aux_out is not None else None
    desc.aux_out_scale = aux_out_scale.data_ptr() if aux_out_scale is not None else None
    desc.aux_out_cols = aux_out_cols.data_ptr() if aux_out_cols is not None else None
    desc.aux_out_cols_scale = (aux_out_cols_scale.data_ptr() if aux_out_cols_scale is not None
                               else None)
    wsb = int(_lib.moe_grouped_gemm_workspace_size(ctypes.byref(desc)))
    ws = torch.empty(wsb, dtype=torch.uint8, device=A.device) if wsb else None
    desc.ws = ws.data_ptr() if ws is not None else None
    desc.ws_bytes = wsb
    _check("moe_grouped_gemm", _lib.moe_grouped_gemm(ctypes.byref(desc), _stream()))
    return C


def moe_backward(saved: dict, dout: torch.Tensor, E: int, k: int, d: int, h: int,
                 out: dict | None = None, want_dgate: bool = True, mxfp8: bool = False,
                 accumulate_dw: bool = False, stage_events=None,
                 act8: dict | None = None) -> dict:
    """Backward of the whole layer. `saved` holds the forward tensors
    (x_perm, ab, hp, y_perm, topk_gate, topk_idx, token_pos, offsets, w1, w2;
    with mxfp8: x, sorted_token, w1t, w1t_scale, w2t, w2t_scale instead of
    x_perm, w1, w2). act8: the checkpoints ab8, ab8_scale, y8, y8_scale of a
    layer that held these instead of ab and y_perm (moe_backward_act8): saved's
    ab and hp are then scratch that the call writes, its y_perm is not used."""
    T = dout.shape[0]
    R = T * k
    dev, dt = dout.device, dout.dtype
    if out is None:
        out = dict(dx=torch.empty((T, d), dtype=dt, device=dev),
                   dlogits=torch.empty((T, E), dtype=torch.float32, device=dev),
                   dw1=torch.empty((E, 2 * h, d), dtype=torch.float32, device=dev),
                   dw2=torch.empty((E, d, h), dtype=torch.float32, device=dev),
                   dgate=torch.empty((T, k), dtype=torch.float32, device=dev) if want_dgate else None,
                   dy_perm=torch.empty((R, d), dtype=dt, device=dev),
                   dab=torch.empty((R, 2 * h), dtype=dt, device=dev),
                   dx_perm=torch.empty((R, d), dtype=dt, device=dev))
    b = BwdDesc()
    b.accumulate_dw = 1 if accumulate_dw else 0
    b.dtype = MOE_MXFP8 if mxfp8 else _dt(dout)
    b.d, b.h, b.E, b.k, b.T = d, h, E, k, T
    names = ("ab", "hp", "topk_gate", "topk_idx", "token_pos", "offsets")
    if act8 is None:
        names += ("y_perm",)
    else:
        act = torch.bfloat16 if mxfp8 else dt
        _act8_need(act8["ab8"], act8["ab8_scale"], R, 2 * h, dout.get_device(), "ab8")
        _act8_need(act8["y8"], act8["y8_scale"], R, d, dout.get_device(), "y8")
        _need(saved["ab"], (R, 2 * h), act, "ab")
        if saved.get("hp") is not None or not mxfp8:
            _need(saved["hp"], (R, h), act, "hp")
    names += (("x", "sorted_token", "w1t", "w1t_scale", "w2t", "w2t_scale") if mxfp8
              else ("x_perm", "w1", "w2"))
    for name in names:
        if name == "hp" and saved.get(name) is None and mxfp8:
            continue                               # H' brought in its column layout instead
        setattr(b, name, saved[name].data_ptr())
    if mxfp8 and saved.get("hp_cols") is not None:
        b.hp_cols = saved["hp_cols"].data_ptr()
        b.hp_cols_scale = saved["hp_cols_scale"].data_ptr()
    b.dout = dout.data_ptr()
    for name in ("dx", "dlogits", "dw1", "dw2", "dy_perm", "dab", "dx_perm"):
        setattr(b, name, out[name].data_ptr())
    b.dgate = out["dgate"].data_ptr() if out.get("dgate") is not None else None
    wsb = int(_lib.moe_backward_workspace_size(ctypes.byref(b)))
    ws = out.get("_ws")
    if wsb and (ws is None or ws.numel() < wsb):
        ws = torch.empty(wsb, dtype=torch.uint8, device=dev)
        out["_ws"] = ws
    b.ws = ws.data_ptr() if wsb else None
    b.ws_bytes = wsb
    if stage_events is not None:
        # hipEvent_t handles of recorded torch.cuda.Event objects, one per stage
        arr = (_P * MOE_BWD_MAX_STAGES)(*[ctypes.c_void_p(e.cuda_event) if e is not None else None
                                          for e in list(stage_events) +
                                          [None] * (MOE_BWD_MAX_STAGES - len(stage_events))])
        b.stage_events = ctypes.cast(arr, ctypes.POINTER(_P))
    if act8 is None:
        _check("moe_backward", _lib.moe_backward(ctypes.byref(b), _stream()))
    else:
        c = Act8Saved(*(act8[n].data_ptr() for n, _ in Act8Saved._fields_))
        _check("moe_backward_act8", _lib.moe_backward_act8(ctypes.byref(b), ctypes.byref(c),
                                                           _stream()))
    return out


def moe_gemm_copy_walk(mode: int, dtype: int, epilogue: int, offsets, M: int = 0, N: int = 0,
                       K: int = 0, extents=(0, 0, 0, 0)) -> dict:
    """Host-side walk of every copy moe_grouped_gemm would issue (no GPU).
    offsets: host sequence of n_groups + 1 ints; extents: readable bytes of
    A, B, a_scale, b_scale."""
    off = (ctypes.c_int32 * len(offsets))(*[int(v) for v in offsets])
    g = GemmDesc()
    g.mode, g.dtype, g.epilogue = mode, dtype, epilogue
    g.n_groups = len(offsets) - 1
    g.rows = int(offsets[-1])
    g.M, g.N, g.K = M, N, K
    w = CopyWalk()
    for i, x in enumerate(extents):
        w.extent[i] = int(x)
    _check("moe_gemm_copy_walk", _lib.moe_gemm_copy_walk(ctypes.byref(g), off, ctypes.byref(w)))
    return {"copies": w.copies, "zero_copies": w.zero_copies, "lowest": list(w.lowest),
            "end": list(w.end), "first_bad": w.first_bad, "bad_offset": w.bad_offset,
            "bad_bytes": w.bad_bytes}


def moe_gemm_hp_store_walk(offsets, h: int, K: int, extents=(0, 0, 0, 0)) -> dict:
    """Host-side walk of every store of the MXFP8 SwiGLU forward that writes
    H' quantised (no GPU). offsets: host sequence of n_groups + 1 ints;
    extents: writable bytes of aux_out, aux_out_scale, aux_out_cols,
    aux_out_cols_scale."""
    off = (ctypes.c_int32 * len(offsets))(*[int(v) for v in offsets])
    g = GemmDesc()
    g.mode, g.dtype, g.epilogue = MOE_GG_FWD, MOE_MXFP8, MOE_EPI_SWIGLU_FWD
    g.n_groups = len(offsets) - 1
    g.rows = int(offsets[-1])
    g.N, g.K = 2 * h, K
    w = CopyWalk()
    for i, x in enumerate(extents):
        w.extent[i] = int(x)
    _check("moe_gemm_hp_store_walk", _lib.moe_gemm_hp_store_walk(ctypes.byref(g), off,
                                                                 ctypes.byref(w)))
    return {"stores": w.copies, "lowest": list(w.lowest), "end": list(w.end),
            "first_bad": w.first_bad, "bad_offset": w.bad_offset, "bad_bytes": w.bad_bytes}


def moe_backward_workspace_layout(T: int, E: int, k: int, d: int, h: int) -> dict:
    """Byte offsets of the MXFP8 backward's regions inside its workspace."""
    b = BwdDesc()
    b.dtype, b.T, b.E, b.k, b.d, b.h = MOE_MXFP8, T, E, k, d, h
    L = BwdWsLayout()
    _check("moe_backward_workspace_layout",
           _lib.moe_backward_workspace_layout(ctypes.byref(b), ctypes.byref(L)))
    return {n: getattr(L, n) for n, _ in BwdWsLayout._fields_}


def moe_backward_workspace_size(T: int, E: int, k: int, d: int, h: int, dtype: int) -> int:
    b = BwdDesc()
    b.dtype, b.T, b.E, b.k, b.d, b.h = dtype, T, E, k, d, h
    return _lib.moe_backward_workspace_size(ctypes.byref(b))


def mxfp8_col_blocks(rows: int, n_groups: int) -> int:
    return int(_lib.mxfp8_col_blocks(rows, n_groups))


def mxfp8_quantize(x: torch.Tensor, axis: int = 1, group_offsets: torch.Tensor | None = None,
                   q: torch.Tensor | None = None, scale: torch.Tensor | None = None,
                   row_map: torch.Tensor | None = None):
    """OCP MXFP8 quantisation (see moe.h). axis=1 returns q [rows, cols] and
    scale [rows, cols/32]; axis=0 returns the flat column-block layout (groups
    padded to 128 rows) sized for the worst case. With row_map, output row r
    quantises x[row_map[r]] (rows = row_map.numel())."""
    rows = x.shape[0] if row_map is None else row_map.numel()
    cols = x.shape[1]
    dev = x.device
    ng = 0 if group_offsets is None else group_offsets.numel() - 1
    if axis == 1:
        q = q if q is not None else torch.empty((rows, cols), dtype=torch.uint8, device=dev)
        scale = scale if scale is not None else torch.empty((rows, cols // 32), dtype=torch.uint8,
                                                            device=dev)
    else:
        nb = mxfp8_col_blocks(rows, max(ng, 1))
        q = q if q is not None else torch.empty(nb * 32 * cols, dtype=torch.uint8, device=dev)
        scale = scale if scale is not None else torch.empty(nb * cols, dtype=torch.uint8, device=dev)
    _check("mxfp8_quantize", _lib.mxfp8_quantize(_p(x), _dt(x), rows, cols, axis,
                                                 _p(group_offsets), ng, _p(row_map), _p(q),
                                                 _p(scale), _stream()))
    return q, scale


def mxfp8_quantize_both(x: torch.Tensor, group_offsets: torch.Tensor | None = None,
                        out: tuple | None = None):
    """Both orientations from one read (see moe.h): returns (q_rows, s_rows)
    as mxfp8_quantize axis=1 and (q_cols, s_cols) as axis=0 with these groups,
    into `out` = (q_rows, s_rows, q_cols, s_cols) when given."""
    rows, cols = x.shape
    dev = x.device
    ng = 0 if group_offsets is None else group_offsets.numel() - 1
    nb = mxfp8_col_blocks(rows, max(ng, 1))
    if out is not None:
        q1, s1, q0, s0 = out
        _need(q1, (rows, cols), torch.uint8, "q_rows")
        _need(s1, (rows, cols // 32), torch.uint8, "s_rows")
        _need_bytes(q0, nb * 32 * cols, "q_cols")
        _need_bytes(s0, nb * cols, "s_cols")
    else:
        q1 = torch.empty((rows, cols), dtype=torch.uint8, device=dev)
        s1 = torch.empty((rows, cols // 32), dtype=torch.uint8, device=dev)
        q0 = torch.empty(nb * 32 * cols, dtype=torch.uint8, device=dev)
        s0 = torch.empty(nb * cols, dtype=torch.uint8, device=dev)
    _check("mxfp8_quantize_both", _lib.mxfp8_quantize_both(
        _p(x), _dt(x), rows, cols, _p(group_offsets), ng, _p(q1), _p(s1), _p(q0), _p(s0),
        _stream()))
    return (q1, s1), (q0, s0)


def moe_capacity_pad(route: dict, capacity: int, out: dict | None = None) -> dict:
    """Padded-capacity layout of moe_route's dropless metadata (see moe.h):
    token_pos [T, k] with dropped slots at -1, offsets [E+1] = e * capacity."""
    T, k = route["topk_idx"].shape
    E = route["offsets"].numel() - 1
    dev = route["offsets"].device
    if out is None:
        out = dict(token_pos=torch.empty((T, k), dtype=torch.int32, device=dev),
                   offsets=torch.empty(E + 1, dtype=torch.int32, device=dev))
    _check("moe_capacity_pad", _lib.moe_capacity_pad(
        _p(route["topk_idx"]), _p(route["token_pos"]), _p(route["offsets"]), T, E, k, capacity,
        _p(out["token_pos"]), _p(out["offsets"]), _stream()))
    return out


def moe_capacity_zero_rows(buf: torch.Tensor, offsets: torch.Tensor, capacity: int) -> torch.Tensor:
    """Zero the unused capacity rows of a [E*capacity, cols] buffer; offsets
    are the dropless ones (see moe.h)."""
    E = offsets.numel() - 1
    _check("moe_capacity_zero_rows", _lib.moe_capacity_zero_rows(
        _p(buf), _dt(buf), _p(offsets), E, capacity, buf.shape[-1], _stream()))
    return buf


# ---------------------------------------------------------------------------
# 8-bit activation checkpoints and the layer norm


# The stream handle and the current device without the objects around them:
# torch.cuda.current_stream() costs as much host time as a kernel launch.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_cur_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _enqueue(name, fn, index, *args):
    """fn(*args, stream) on GPU `index`'s current stream, with that GPU
    current while the call is made (tensors need not be on the current one)."""
    if _cur_device() == index:
        st = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            st = fn(*args, _raw_stream(index))
    if st != MOE_OK:
        raise MoeError(name, st)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _need_on(t, shape, dtype, index, name):
    """t is a contiguous tensor of this shape and dtype on GPU `index`."""
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype is not dtype or t.get_device() != index or index < 0 or t.shape != shape or \
            not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous {dtype} {tuple(shape)} on "
                         f"{'a GPU' if index < 0 else f'cuda:{index}'}, got "
                         f"{t.dtype} {tuple(t.shape)} (contiguous={t.is_contiguous()}, "
                         f"device={t.device})")


def _act_matrix(x, name):
    """rows, cols of a contiguous 2-d f32 / bf16 GPU tensor whose rows are
    whole blocks of 32, its C dtype and its GPU."""
    if x is None:
        raise ValueError(f"{name} is required")
    if x.dtype is torch.bfloat16:
        dt = MOE_BF16
    elif x.dtype is torch.float32:
        dt = MOE_F32
    else:
        raise ValueError(f"{name}: expected bf16 or f32, got {x.dtype}")
    shape, index = x.shape, x.get_device()
    if len(shape) != 2 or shape[1] < 32 or shape[1] % 32:
        raise ValueError(f"{name}: expected [rows, a multiple of 32], got {tuple(shape)}")
    if index < 0 or not x.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor on a GPU, got device={x.device}, "
                         f"contiguous={x.is_contiguous()}")
    return shape[0], shape[1], dt, index


def _act8_need(q, scale, rows, cols, index, name):
    _need_on(q, (rows, cols), torch.uint8, index, name)
    _need_on(scale, (rows, cols // 32), torch.uint8, index, name + "_scale")


def _act8_new(rows, cols, dev):
    u8 = dict(dtype=torch.uint8, device=dev)
    return torch.empty(rows, cols, **u8), torch.empty(rows, cols // 32, **u8)


def _act8_out(rows, cols, like, index, q, scale, name):
    """The tensors of a checkpoint to be written: the caller's, or new ones."""
    if q is None and scale is None:
        return _act8_new(rows, cols, like.device)
    _act8_need(q, scale, rows, cols, index, name)
    return q, scale


def _act8_in(q, scale, dtype, name):
    if dtype is not torch.bfloat16 and dtype is not torch.float32:
        raise ValueError(f"dtype: expected bf16 or f32, got {dtype}")
    shape = () if q is None else q.shape
    if len(shape) != 2 or shape[1] < 32 or shape[1] % 32:
        raise ValueError(f"{name}: expected [rows, a multiple of 32], got "
                         f"{None if q is None else tuple(shape)}")
    rows, cols = shape
    index = q.get_device()
    _act8_need(q, scale, rows, cols, index, name)
    return rows, cols, MOE_BF16 if dtype is torch.bfloat16 else MOE_F32, index


def moe_act8_store(x: torch.Tensor, q: torch.Tensor | None = None,
                   scale: torch.Tensor | None = None):
    """The 8-bit checkpoint (MXINT8, see moe.h) of x [rows, cols]: uint8 q
    [rows, cols] and scale [rows, cols/32]."""
    rows, cols, dt, gpu = _act_matrix(x, "x")
    q, scale = _act8_out(rows, cols, x, gpu, q, scale, "q")
    _enqueue("moe_act8_store", _lib.moe_act8_store, gpu, x.data_ptr(), dt, rows, cols,
             q.data_ptr(), scale.data_ptr())
    return q, scale


def moe_act8_load(q: torch.Tensor, scale: torch.Tensor, dtype: torch.dtype = torch.bfloat16,
                  out: torch.Tensor | None = None) -> torch.Tensor:
    """The values that a checkpoint stands for, as `dtype` (exact in both)."""
    rows, cols, dt, gpu = _act8_in(q, scale, dtype, "q")
    if out is None:
        out = torch.empty_like(q, dtype=dtype)
    else:
        _need_on(out, (rows, cols), dtype, gpu, "out")
    _enqueue("moe_act8_load", _lib.moe_act8_load, gpu, q.data_ptr(), scale.data_ptr(), dt, rows,
             cols, out.data_ptr())
    return out


def moe_act8_swiglu(ab8: torch.Tensor, ab8_scale: torch.Tensor,
                    dtype: torch.dtype = torch.bfloat16, ab: torch.Tensor | None = None,
                    hp: torch.Tensor | None = None):
    """From the checkpoint of A||B [rows, 2h]: (ab, hp), its values and
    H' = silu(a) b of them."""
    rows, cols, dt, gpu = _act8_in(ab8, ab8_scale, dtype, "ab8")
    h = cols // 2
    if h % 32:
        raise ValueError(f"ab8: the hidden width must be a multiple of 32, got {h}")
    if ab is None:
        ab = torch.empty_like(ab8, dtype=dtype)
    else:
        _need_on(ab, (rows, cols), dtype, gpu, "ab")
    if hp is None:
        hp = torch.empty(rows, h, dtype=dtype, device=ab8.device)
    else:
        _need_on(hp, (rows, h), dtype, gpu, "hp")
    _enqueue("moe_act8_swiglu", _lib.moe_act8_swiglu, gpu, ab8.data_ptr(), ab8_scale.data_ptr(),
             dt, rows, h, ab.data_ptr(), hp.data_ptr())
    return ab, hp


def _slots(token_pos, T=None):
    """(T, k) of a [T, k] tensor."""
    if token_pos is None or token_pos.dim() != 2 or T not in (None, token_pos.shape[0]):
        raise ValueError(f"token_pos: expected [{'T' if T is None else T}, k], got "
                         f"{None if token_pos is None else tuple(token_pos.shape)}")
    return token_pos.shape[0], token_pos.shape[1]


def moe_combine_act8(y_perm: torch.Tensor, topk_gate: torch.Tensor, token_pos: torch.Tensor,
                     out: torch.Tensor | None = None, y8: torch.Tensor | None = None,
                     y8_scale: torch.Tensor | None = None):
    """moe_combine that also stores the checkpoint of the rows it reads:
    (out [T, d], y8 [R, d], y8_scale [R, d/32]). token_pos must stay below R,
    the rows of y_perm."""
    rows, d, dt, gpu = _act_matrix(y_perm, "y_perm")
    T, k = _slots(token_pos)
    _need_on(token_pos, (T, k), torch.int32, gpu, "token_pos")
    _need_on(topk_gate, (T, k), torch.float32, gpu, "topk_gate")
    if out is None:
        out = torch.empty(T, d, dtype=y_perm.dtype, device=y_perm.device)
    else:
        _need_on(out, (T, d), y_perm.dtype, gpu, "out")
    y8, y8_scale = _act8_out(rows, d, y_perm, gpu, y8, y8_scale, "y8")
    _enqueue("moe_combine_act8", _lib.moe_combine_act8, gpu, y_perm.data_ptr(), dt,
             topk_gate.data_ptr(), token_pos.data_ptr(), T, d, k, out.data_ptr(), y8.data_ptr(),
             y8_scale.data_ptr())
    return out, y8, y8_scale


def moe_combine_backward_act8(dout: torch.Tensor, y8: torch.Tensor, y8_scale: torch.Tensor,
                              topk_gate: torch.Tensor, topk_idx: torch.Tensor,
                              token_pos: torch.Tensor, E: int, out: dict | None = None,
                              want_dgate: bool = True) -> dict:
    """The combine's backward with the router's, y_perm read from its
    checkpoint (see moe.h): dict of dy_perm [R, d], dlogits [T, E], dgate
    [T, k]. With `out`, into its tensors (dgate only if it has one)."""
    T, d, dt, gpu = _act_matrix(dout, "dout")
    if y8 is None or y8.dim() != 2:
        raise ValueError("y8: expected [rows, d]")
    R = y8.shape[0]
    _, k = _slots(token_pos, T)
    _act8_need(y8, y8_scale, R, d, gpu, "y8")
    _need_on(topk_gate, (T, k), torch.float32, gpu, "topk_gate")
    _need_on(topk_idx, (T, k), torch.int32, gpu, "topk_idx")
    _need_on(token_pos, (T, k), torch.int32, gpu, "token_pos")
    if out is None:
        dev = dout.device
        out = dict(dy_perm=torch.empty(R, d, dtype=dout.dtype, device=dev),
                   dlogits=torch.empty(T, E, dtype=torch.float32, device=dev))
        if want_dgate:
            out["dgate"] = torch.empty(T, k, dtype=torch.float32, device=dev)
    else:
        _need_on(out.get("dy_perm"), (R, d), dout.dtype, gpu, "dy_perm")
        _need_on(out.get("dlogits"), (T, E), torch.float32, gpu, "dlogits")
        if out.get("dgate") is not None:
            _need_on(out["dgate"], (T, k), torch.float32, gpu, "dgate")
    _enqueue("moe_combine_backward_act8", _lib.moe_combine_backward_act8, gpu, dout.data_ptr(), dt,
             y8.data_ptr(), y8_scale.data_ptr(), topk_gate.data_ptr(), topk_idx.data_ptr(),
             token_pos.data_ptr(), T, d, k, E, out["dy_perm"].data_ptr(),
             out["dlogits"].data_ptr(), _ptr(out.get("dgate")))
    return out


def moe_layer_norm(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None,
                   eps: float = 1e-5, residual: torch.Tensor | None = None, act8: bool = False,
                   stats: bool = True, out: dict | None = None) -> dict:
    """Layer norm over the rows of x [T, d], or of x + residual (see moe.h).
    Returns a dict: y; with a residual sum (x + residual, the stream); with
    stats mean and rstd [T] fp32 for the backward; with act8 x8 and x8_scale,
    the normalised input's 8-bit checkpoint. `out`: a dict of an earlier call
    with the same arguments, whose tensors are written again."""
    T, d, dt, gpu = _act_matrix(x, "x")
    f32 = torch.float32
    _need_on(weight, (d,), f32, gpu, "weight")
    if bias is not None:
        _need_on(bias, (d,), f32, gpu, "bias")
    if residual is not None:
        _need_on(residual, (T, d), x.dtype, gpu, "residual")
    if out is None:
        dev = x.device
        out = dict(y=torch.empty_like(x))
        if residual is not None:
            out["sum"] = torch.empty_like(x)
        if stats:
            out["mean"] = torch.empty(T, dtype=f32, device=dev)
            out["rstd"] = torch.empty(T, dtype=f32, device=dev)
        if act8:
            out["x8"], out["x8_scale"] = _act8_new(T, d, dev)
    else:
        _need_on(out.get("y"), (T, d), x.dtype, gpu, "y")
        if residual is not None:
            _need_on(out.get("sum"), (T, d), x.dtype, gpu, "sum")
        if stats:
            _need_on(out.get("mean"), (T,), f32, gpu, "mean")
            _need_on(out.get("rstd"), (T,), f32, gpu, "rstd")
        if act8:
            _act8_need(out.get("x8"), out.get("x8_scale"), T, d, gpu, "x8")
    _enqueue("moe_layer_norm", _lib.moe_layer_norm, gpu, x.data_ptr(), dt, _ptr(residual),
             weight.data_ptr(), _ptr(bias), eps, T, d, out["y"].data_ptr(),
             None if residual is None else out["sum"].data_ptr(),
             out["mean"].data_ptr() if stats else None, out["rstd"].data_ptr() if stats else None,
             out["x8"].data_ptr() if act8 else None,
             out["x8_scale"].data_ptr() if act8 else None)
    return out


def moe_layer_norm_backward_workspace_size(dtype: int, T: int, d: int) -> int:
    return _lib.moe_layer_norm_backward_workspace_size(dtype, T, d)


def _need_ws(ws, nbytes, like, gpu):
    """The caller's workspace, checked, or a new one."""
    if ws is None:
        return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=like.device)
    _need_bytes(ws, nbytes, "ws")
    if ws.get_device() != gpu:
        raise ValueError(f"ws: expected on cuda:{gpu}, got {ws.device}")
    return ws


def moe_layer_norm_backward(saved: dict, dy: torch.Tensor, weight: torch.Tensor,
                            dsum: torch.Tensor | None = None, out: dict | None = None,
                            accumulate_dw: bool = False, want_dweight: bool = True,
                            want_dbias: bool = True, ws: torch.Tensor | None = None) -> dict:
    """Backward of moe_layer_norm (see moe.h). saved: mean and rstd, and the
    normalised input as x or as x8 and x8_scale (x, if both are there).
    Returns a dict: dx [T, d] (with a residual, its gradient too), dweight and
    dbias [d] fp32. dsum: the gradient that reaches x (or sum) by its other
    uses, added to dx. out: tensors of an earlier call; accumulate_dw adds to
    its dweight and dbias."""
    T, d, dt, gpu = _act_matrix(dy, "dy")
    f32 = torch.float32
    x = saved.get("x")
    x8 = x8s = None
    if x is not None:
        _need_on(x, (T, d), dy.dtype, gpu, "x")
    else:
        x8, x8s = saved.get("x8"), saved.get("x8_scale")
        _act8_need(x8, x8s, T, d, gpu, "x8")
    mean, rstd = saved.get("mean"), saved.get("rstd")
    _need_on(mean, (T,), f32, gpu, "mean")
    _need_on(rstd, (T,), f32, gpu, "rstd")
    _need_on(weight, (d,), f32, gpu, "weight")
    if dsum is not None:
        _need_on(dsum, (T, d), dy.dtype, gpu, "dsum")
    if out is None:
        if accumulate_dw:
            raise ValueError("accumulate_dw needs the gradients of an earlier backward (out)")
        dev = dy.device
        out = dict(dx=torch.empty_like(dy))
        if want_dweight:
            out["dweight"] = torch.empty(d, dtype=f32, device=dev)
        if want_dbias:
            out["dbias"] = torch.empty(d, dtype=f32, device=dev)
    else:
        _need_on(out.get("dx"), (T, d), dy.dtype, gpu, "dx")
        if want_dweight:
            _need_on(out.get("dweight"), (d,), f32, gpu, "dweight")
        if want_dbias:
            _need_on(out.get("dbias"), (d,), f32, gpu, "dbias")
    if want_dweight or want_dbias:
        ws = _need_ws(ws, moe_layer_norm_backward_workspace_size(dt, T, d), dy, gpu)
    _enqueue("moe_layer_norm_backward", _lib.moe_layer_norm_backward, gpu, dy.data_ptr(), dt,
             _ptr(x), _ptr(x8), _ptr(x8s), mean.data_ptr(), rstd.data_ptr(), weight.data_ptr(),
             _ptr(dsum), T, d, out["dx"].data_ptr(),
             out["dweight"].data_ptr() if want_dweight else None,
             out["dbias"].data_ptr() if want_dbias else None, 1 if accumulate_dw else 0, _ptr(ws),
             0 if ws is None else ws.numel())
    return out


# ---------------------------------------------------------------------------
# the root-mean-square norm with an output in 8 bits


def moe_rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                 residual: torch.Tensor | None = None, quantize: bool = False, want_y: bool = True,
                 act8: bool = False, stats: bool = True, out: dict | None = None) -> dict:
    """Root-mean-square norm over the rows of x [T, d], or of x + residual
    (see moe.h). Returns a dict: y (unless want_y is False, which needs
    quantize); with a residual sum; with stats rstd [T] fp32 for the backward;
    with quantize yq and yq_scale, y in MXFP8 along its rows; with act8 x8 and
    x8_scale, the normalised input's 8-bit checkpoint. `out`: a dict of an
    earlier call with the same arguments, whose tensors are written again."""
    T, d, dt, gpu = _act_matrix(x, "x")
    f32 = torch.float32
    if not (want_y or quantize):
        raise ValueError("want_y=False needs quantize=True")
    _need_on(weight, (d,), f32, gpu, "weight")
    if residual is not None:
        _need_on(residual, (T, d), x.dtype, gpu, "residual")
    if out is None:
        dev = x.device
        out = {}
        if want_y:
            out["y"] = torch.empty_like(x)
        if residual is not None:
            out["sum"] = torch.empty_like(x)
        if stats:
            out["rstd"] = torch.empty(T, dtype=f32, device=dev)
        if quantize:
            out["yq"], out["yq_scale"] = _act8_new(T, d, dev)
        if act8:
            out["x8"], out["x8_scale"] = _act8_new(T, d, dev)
    else:
        if want_y:
            _need_on(out.get("y"), (T, d), x.dtype, gpu, "y")
        if residual is not None:
            _need_on(out.get("sum"), (T, d), x.dtype, gpu, "sum")
        if stats:
            _need_on(out.get("rstd"), (T,), f32, gpu, "rstd")
        if quantize:
            _act8_need(out.get("yq"), out.get("yq_scale"), T, d, gpu, "yq")
        if act8:
            _act8_need(out.get("x8"), out.get("x8_scale"), T, d, gpu, "x8")
    _enqueue("moe_rms_norm", _lib.moe_rms_norm, gpu, x.data_ptr(), dt, _ptr(residual),
             weight.data_ptr(), eps, T, d, out["y"].data_ptr() if want_y else None,
             None if residual is None else out["sum"].data_ptr(),
             out["rstd"].data_ptr() if stats else None,
             out["yq"].data_ptr() if quantize else None,
             out["yq_scale"].data_ptr() if quantize else None,
             out["x8"].data_ptr() if act8 else None,
             out["x8_scale"].data_ptr() if act8 else None)
    return out


def moe_rms_norm_backward_workspace_size(dtype: int, T: int, d: int) -> int:
    return _lib.moe_rms_norm_backward_workspace_size(dtype, T, d)


def moe_rms_norm_backward(saved: dict, dy: torch.Tensor, weight: torch.Tensor,
                          dsum: torch.Tensor | None = None, out: dict | None = None,
                          accumulate_dw: bool = False, want_dweight: bool = True,
                          ws: torch.Tensor | None = None) -> dict:
    """Backward of moe_rms_norm (see moe.h). saved: rstd, and the normalised
    input as x or as x8 and x8_scale (x, if both are there). Returns a dict:
    dx [T, d] (with a residual, its gradient too) and dweight [d] fp32. dsum:
    the gradient that reaches x (or sum) by its other uses, added to dx. out:
    tensors of an earlier call; accumulate_dw adds to its dweight."""
    T, d, dt, gpu = _act_matrix(dy, "dy")
    f32 = torch.float32
    x = saved.get("x")
    x8 = x8s = None
    if x is not None:
        _need_on(x, (T, d), dy.dtype, gpu, "x")
    else:
        x8, x8s = saved.get("x8"), saved.get("x8_scale")
        _act8_need(x8, x8s, T, d, gpu, "x8")
    rstd = saved.get("rstd")
    _need_on(rstd, (T,), f32, gpu, "rstd")
    _need_on(weight, (d,), f32, gpu, "weight")
    if dsum is not None:
        _need_on(dsum, (T, d), dy.dtype, gpu, "dsum")
    if out is None:
        if accumulate_dw:
            raise ValueError("accumulate_dw needs the gradients of an earlier backward (out)")
        out = dict(dx=torch.empty_like(dy))
        if want_dweight:
            out["dweight"] = torch.empty(d, dtype=f32, device=dy.device)
    else:
        _need_on(out.get("dx"), (T, d), dy.dtype, gpu, "dx")
        if want_dweight:
            _need_on(out.get("dweight"), (d,), f32, gpu, "dweight")
    if want_dweight:
        ws = _need_ws(ws, moe_rms_norm_backward_workspace_size(dt, T, d), dy, gpu)
    _enqueue("moe_rms_norm_backward", _lib.moe_rms_norm_backward, gpu, dy.data_ptr(), dt, _ptr(x),
             _ptr(x8), _ptr(x8s), rstd.data_ptr(), weight.data_ptr(), _ptr(dsum), T, d,
             out["dx"].data_ptr(), out["dweight"].data_ptr() if want_dweight else None,
             1 if accumulate_dw else 0, _ptr(ws), 0 if ws is None else ws.numel())
    return out


def mxfp8_dequantize(q: torch.Tensor, scale: torch.Tensor, dtype: torch.dtype = torch.bfloat16,
                     out: torch.Tensor | None = None) -> torch.Tensor:
    """The values that MXFP8 rows (q [rows, cols], scale [rows, cols/32]) stand
    for, as `dtype` (see moe.h)."""
    rows, cols, dt, gpu = _act8_in(q, scale, dtype, "q")
    if out is None:
        out = torch.empty_like(q, dtype=dtype)
    else:
        _need_on(out, (rows, cols), dtype, gpu, "out")
    _enqueue("mxfp8_dequantize", _lib.mxfp8_dequantize, gpu, q.data_ptr(), scale.data_ptr(), dt,
             rows, cols, out.data_ptr())
    return out


# ---------------------------------------------------------------------------
# the gradients' norm, and clipping

MOE_GRAD_MAX = 4096
_GRAD_DT = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16}


_t_ptr, _t_numel, _t_gpu = torch.Tensor.data_ptr, torch.Tensor.numel, torch.Tensor.get_device
_t_contiguous, _t_dtype = torch.Tensor.is_contiguous, operator.attrgetter("dtype")


def _grad_bad(name, t, i, gpu, want):
    raise ValueError(f"{name}[{i}]: expected a contiguous {want} on "
                     f"{'a GPU' if gpu < 0 else f'cuda:{gpu}'}, got {t.dtype} {tuple(t.shape)} "
                     f"(contiguous={t.is_contiguous()}, device={t.device})")


def _grad_list(grads, out=None):
    """The C descriptors (moe_grad: data, out, n, dtype) of a list of
    tensors, their address and number, the tensors' GPU, and the lists of the
    tensors, which the caller holds until its kernels are enqueued (an iterator's
    tensors are in no other place). Checked by whole lists: a model's list is
    long, and a call's host time is its length's."""
    if not isinstance(grads, (list, tuple)):
        grads = list(grads)
    if out is not None and not isinstance(out, (list, tuple)):
        out = list(out)
    n = len(grads)
    if not n:
        raise ValueError("grads: expected at least one tensor")
    if out is not None and len(out) != n:
        raise ValueError(f"out: expected {n} tensors, got {len(out)}")
    gpu = grads[0].get_device()
    dts = list(map(_t_dtype, grads))
    codes = list(map(_GRAD_DT.get, dts))
    if gpu < 0 or None in codes or not all(map(_t_contiguous, grads)) or \
            list(map(_t_gpu, grads)) != [gpu] * n:
        for i, t in enumerate(grads):
            if gpu < 0 or codes[i] is None or t.get_device() != gpu or not t.is_contiguous():
                _grad_bad("grads", t, i, gpu, "f32 or bf16 tensor")
    sizes = list(map(_t_numel, grads))
    v = array.array("q", bytes(32 * n))
    v[0::4] = array.array("q", list(map(_t_ptr, grads)))
    v[2::4] = array.array("q", sizes)
    v[3::4] = array.array("q", codes)
    if out is not None:
        if list(map(_t_dtype, out)) != dts or list(map(_t_numel, out)) != sizes or \
                not all(map(_t_contiguous, out)) or list(map(_t_gpu, out)) != [gpu] * n:
            for i, (t, g) in enumerate(zip(out, grads)):
                if t.dtype is not g.dtype or t.numel() != g.numel() or t.get_device() != gpu or \
                        not t.is_contiguous():
                    _grad_bad("out", t, i, gpu, f"{g.dtype} tensor of {g.numel()} elements")
        v[1::4] = array.array("q", list(map(_t_ptr, out)))
    return v, v.buffer_info()[0], n, gpu, (grads, out)


def _grad_norm_args(n, like, gpu, norm, ws):
    if norm is None:
        norm = torch.empty((), dtype=torch.float32, device=like.device)
    elif norm.dtype is not torch.float32 or norm.numel() != 1 or norm.get_device() != gpu:
        raise ValueError(f"norm: expected one f32 element on cuda:{gpu}, got {norm.dtype} "
                         f"{tuple(norm.shape)} on {norm.device}")
    return norm, _need_ws(ws, _lib.moe_grad_norm_workspace_size(n), like, gpu)


def moe_grad_norm_workspace_size(n_grads: int) -> int:
    return _lib.moe_grad_norm_workspace_size(n_grads)


def moe_grad_norm(grads, norm: torch.Tensor | None = None,
                  ws: torch.Tensor | None = None) -> torch.Tensor:
    """The norm of all elements of a list of f32 and bf16 tensors (see moe.h):
    one f32 element on their GPU."""
    v, at, n, gpu, held = _grad_list(grads)
    norm, ws = _grad_norm_args(n, held[0][0], gpu, norm, ws)
    _enqueue("moe_grad_norm", _lib.moe_grad_norm, gpu, at, n, norm.data_ptr(), ws.data_ptr(),
             ws.numel())
    return norm


def moe_clip_grad_norm(grads, max_norm: float, out=None, norm: torch.Tensor | None = None,
                       ws: torch.Tensor | None = None) -> torch.Tensor:
    """moe_grad_norm, and every tensor times min(1, max_norm / (norm + 1e-6)),
    in place or into the tensors of `out` (of the same types and numbers of
    elements). Returns the norm in front of it."""
    v, at, n, gpu, held = _grad_list(grads, out)
    norm, ws = _grad_norm_args(n, held[0][0], gpu, norm, ws)
    _enqueue("moe_clip_grad_norm", _lib.moe_clip_grad_norm, gpu, at, n, max_norm, norm.data_ptr(),
             ws.data_ptr(), ws.numel())
    return norm


def moe_grad_clip(grads, norm: torch.Tensor, max_norm: float, out=None):
    """The clipping alone, with a norm that is given (one f32 element on the
    tensors' GPU)."""
    v, at, n, gpu, held = _grad_list(grads, out)
    if norm is None or norm.dtype is not torch.float32 or norm.numel() != 1 or \
            norm.get_device() != gpu:
        raise ValueError(f"norm: expected one f32 element on cuda:{gpu}")
    _enqueue("moe_grad_clip", _lib.moe_grad_clip, gpu, at, n, norm.data_ptr(), max_norm)


# ---------------------------------------------------------------------------
# the experts for few tokens, weights in 4 bits


def moe_w4_quantize(w: torch.Tensor, q: torch.Tensor | None = None,
                    scale: torch.Tensor | None = None):
    """OCP MXFP4 quantisation (see moe.h) of w [..., rows, cols] (f32 or
    bf16) along its rows: q [..., rows, cols/2] and scale [..., rows, cols/32]."""
    if w is None or w.dim() < 2:
        raise ValueError("w: expected [..., rows, cols]")
    if not w.is_contiguous():
        raise ValueError("w: expected a contiguous tensor")
    rows, cols, dt, gpu = _act_matrix(w.reshape(-1, w.shape[-1]), "w")
    lead = tuple(w.shape[:-1])
    if q is None:
        q = torch.empty(lead + (cols // 2,), dtype=torch.uint8, device=w.device)
    if scale is None:
        scale = torch.empty(lead + (cols // 32,), dtype=torch.uint8, device=w.device)
    _need_on(q, lead + (cols // 2,), torch.uint8, gpu, "q")
    _need_on(scale, lead + (cols // 32,), torch.uint8, gpu, "scale")
    _enqueue("moe_w4_quantize", _lib.moe_w4_quantize, gpu, w.data_ptr(), dt, rows, cols,
             q.data_ptr(), scale.data_ptr())
    return q, scale


def moe_w4_experts_workspace_size(T: int, k: int, d: int, h: int) -> int:
    return _lib.moe_w4_experts_workspace_size(T, k, d, h)


def _w4_operands(T, d, route, w1q, w1_scale, w2q, w2_scale, gpu):
    """E, k, h of the experts' calls, their operands checked, and the
    routing's tensors that they read."""
    u8, i32 = torch.uint8, torch.int32
    if w1q is None or w1q.dim() != 3 or w1q.shape[1] % 64:
        raise ValueError("w1q: expected [E, 2h, d/2] with h a multiple of 32")
    E, h2 = w1q.shape[0], w1q.shape[1]
    h = h2 // 2
    gate, pos, tok, off = (route.get(n) for n in ("topk_gate", "token_pos", "sorted_token",
                                                  "offsets"))
    _, k = _slots(pos, T)
    _need_on(w1q, (E, h2, d // 2), u8, gpu, "w1q")
    _need_on(w1_scale, (E, h2, d // 32), u8, gpu, "w1_scale")
    _need_on(w2q, (E, d, h // 2), u8, gpu, "w2q")
    _need_on(w2_scale, (E, d, h // 32), u8, gpu, "w2_scale")
    _need_on(gate, (T, k), torch.float32, gpu, "topk_gate")
    _need_on(pos, (T, k), i32, gpu, "token_pos")
    _need_on(tok, (T * k,), i32, gpu, "sorted_token")
    _need_on(off, (E + 1,), i32, gpu, "offsets")
    return E, k, h, gate, pos, tok, off


def moe_w4_experts(x: torch.Tensor, route: dict, w1q: torch.Tensor, w1_scale: torch.Tensor,
                   w2q: torch.Tensor, w2_scale: torch.Tensor, out: torch.Tensor | None = None,
                   ws: torch.Tensor | None = None) -> torch.Tensor:
    """The expert layer's forward for few tokens after the routing, weights
    as moe_w4_quantize writes them (see moe.h). route: moe_route's dict for
    these tokens (topk_gate, token_pos, sorted_token, offsets are read)."""
    T, d, dt, gpu = _act_matrix(x, "x")
    if dt != MOE_BF16:
        raise ValueError(f"x: expected bf16, got {x.dtype}")
    E, k, h, gate, pos, tok, off = _w4_operands(T, d, route, w1q, w1_scale, w2q, w2_scale, gpu)
    if out is None:
        out = torch.empty_like(x)
    else:
        _need_on(out, (T, d), x.dtype, gpu, "out")
    ws = _need_ws(ws, moe_w4_experts_workspace_size(T, k, d, h), x, gpu)
    w = W4Desc(d, h, E, k, T, x.data_ptr(), gate.data_ptr(), pos.data_ptr(), tok.data_ptr(),
               off.data_ptr(), w1q.data_ptr(), w1_scale.data_ptr(), w2q.data_ptr(),
               w2_scale.data_ptr(), out.data_ptr(), ws.data_ptr(), ws.numel())
    _enqueue("moe_w4_experts", _lib.moe_w4_experts, gpu, ctypes.byref(w))
    return out


def moe_w4_gemm(a: torch.Tensor, a_scale: torch.Tensor, bq: torch.Tensor, b_scale: torch.Tensor,
                offsets: torch.Tensor, epilogue: int = MOE_EPI_NONE,
                a_rows: torch.Tensor | None = None, out: torch.Tensor | None = None,
                out_scale: torch.Tensor | None = None):
    """Grouped product of MXFP8 rows with MXFP4 weights (see moe.h): a [*, K]
    and a_scale, bq [E, N, K/2] and b_scale, offsets [E+1]. a_rows (int32): row
    r of the product reads a[a_rows[r]]; else a's rows are the product's.
    Returns out, bf16 [rows, N]; with MOE_EPI_SWIGLU_FWD (out, out_scale), H' in
    MXFP8 [rows, N/2]. offsets[E] and a_rows stay within the tensors: the
    caller's to keep, they are read on the device."""
    total, K, _, gpu = _act8_in(a, a_scale, torch.bfloat16, "a")
    if bq is None or bq.dim() != 3:
        raise ValueError("bq: expected [E, N, K/2]")
    E, N = bq.shape[0], bq.shape[1]
    _need_on(bq, (E, N, K // 2), torch.uint8, gpu, "bq")
    _need_on(b_scale, (E, N, K // 32), torch.uint8, gpu, "b_scale")
    _need_on(offsets, (E + 1,), torch.int32, gpu, "offsets")
    rows = total
    if a_rows is not None:
        rows = a_rows.numel()
        _need_on(a_rows, (rows,), torch.int32, gpu, "a_rows")
    swiglu = epilogue == MOE_EPI_SWIGLU_FWD
    if swiglu:
        if N % 64:
            raise ValueError(f"bq: N = 2h with h a multiple of 32, got {N}")
        out, out_scale = _act8_out(rows, N // 2, a, gpu, out, out_scale, "out")
    elif out is None:
        out = torch.empty(rows, N, dtype=torch.bfloat16, device=a.device)
    else:
        _need_on(out, (rows, N), torch.bfloat16, gpu, "out")
    if not swiglu and out_scale is not None:
        raise ValueError("out_scale: only the SwiGLU epilogue writes 8 bits")
    g = W4GemmDesc(E, epilogue, rows, N, K, offsets.data_ptr(), _ptr(a_rows), a.data_ptr(),
                   a_scale.data_ptr(), bq.data_ptr(), b_scale.data_ptr(), out.data_ptr(),
                   _ptr(out_scale))
    _enqueue("moe_w4_gemm", _lib.moe_w4_gemm, gpu, ctypes.byref(g))
    return (out, out_scale) if swiglu else out


def moe_w4_experts8_workspace_size(T: int, k: int, d: int, h: int) -> int:
    return _lib.moe_w4_experts8_workspace_size(T, k, d, h)


def moe_w4_experts8(xq: torch.Tensor, x_scale: torch.Tensor, route: dict, w1q: torch.Tensor,
                    w1_scale: torch.Tensor, w2q: torch.Tensor, w2_scale: torch.Tensor,
                    out: torch.Tensor | None = None,
                    ws: torch.Tensor | None = None) -> torch.Tensor:
    """moe_w4_experts for the many tokens of a prompt, their rows in MXFP8
    (xq [T, d], x_scale [T, d/32]; see moe.h): out [T, d] bf16."""
    T, d, _, gpu = _act8_in(xq, x_scale, torch.bfloat16, "xq")
    E, k, h, gate, pos, tok, off = _w4_operands(T, d, route, w1q, w1_scale, w2q, w2_scale, gpu)
    if out is None:
        out = torch.empty(T, d, dtype=torch.bfloat16, device=xq.device)
    else:
        _need_on(out, (T, d), torch.bfloat16, gpu, "out")
    ws = _need_ws(ws, moe_w4_experts8_workspace_size(T, k, d, h), xq, gpu)
    w = W4Desc(d, h, E, k, T, xq.data_ptr(), gate.data_ptr(), pos.data_ptr(), tok.data_ptr(),
               off.data_ptr(), w1q.data_ptr(), w1_scale.data_ptr(), w2q.data_ptr(),
               w2_scale.data_ptr(), out.data_ptr(), ws.data_ptr(), ws.numel())
    _enqueue("moe_w4_experts8", _lib.moe_w4_experts8, gpu, ctypes.byref(w), x_scale.data_ptr())
    return out


# ---------------------------------------------------------------------------
# the layer


# Scratch tensors shared by every recomputing (or 8-bit checkpointing) layer
# of one shape: what a layer rebuilds in its backward lives here instead of
# being held from its forward to its backward. Layers may be given a dict of
# their own instead (their `scratch` argument).
_SCRATCH: dict = {}


def _scratch(name: str, shape, dtype, device, store: dict | None = None) -> torch.Tensor:
    store = _SCRATCH if store is None else store
    key = (name, tuple(shape), dtype, str(device))
    t = store.get(key)
    if t is None:
        t = store[key] = torch.empty(shape, dtype=dtype, device=device)
    return t


def _nbytes(ts) -> int:
    return sum(t.numel() * t.element_size() for t in ts if t is not None)


def _tensors(v):
    """The tensors in a (nested) dict of buffers."""
    if isinstance(v, dict):
        return [t for w in v.values() for t in _tensors(w)]
    return [v] if isinstance(v, torch.Tensor) else []


_cur_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing", None) or (
    torch.cuda.is_current_stream_capturing)


def _capturing(index: int) -> bool:
    """Whether GPU `index`'s current stream is being captured into a graph."""
    if _cur_device() == index:
        return _cur_capturing()
    with torch.cuda.device(index):
        return _cur_capturing()


# Bytes of buffers that a layer object keeps for sizes it was called with
# before its last one: enough for the batch sizes of text generation, next to
# nothing beside a training step's activations.
_KEPT_BYTES = 64 << 20


class _Sizes:
    """The buffers of a layer object: a dict for each size it is called with.

    A replay reads and writes the buffers of the call that was captured, so a
    dict that was in use during a capture stays as long as the object does.
    Of the others the last used stays, and earlier ones while they take
    _KEPT_BYTES at most together."""

    def __init__(self):
        self._all, self._bytes, self._last = {}, {}, None

    def at(self, key) -> dict:
        """The dict of this size, the caller's to fill."""
        if key != self._last:
            if self._last is not None:
                self._bytes[self._last] = _nbytes(_tensors(self._all[self._last]))
            self._last = key
            self._all[key] = self._all.pop(key, {})         # last used last
            room = _KEPT_BYTES
            for k in list(self._all)[-2::-1]:
                if "captured" not in self._all[k]:
                    if 0 < self._bytes[k] <= room:
                        room -= self._bytes[k]
                    else:
                        del self._all[k]
        return self._all[key]


def _mark(buf, index):
    """To be called when kernels that use a size's dict have been enqueued."""
    if "captured" not in buf and _capturing(index):
        buf["captured"] = True


MOE_LB_NSTATS = 8
LB_STAT_NAMES = ("loss", "soft_hard_balance", "hard_balance", "soft_balance", "max_load_over_mean",
                 "min_load_over_mean", "count_cv", "empty_experts")


def moe_load_balance_workspace_size(T: int, E: int) -> int:
    return int(_lib.moe_load_balance_workspace_size(T, E))


def moe_load_balance(logits: torch.Tensor, counts: torch.Tensor, k: int, alpha: float,
                     stats: torch.Tensor | None = None, dlogits: torch.Tensor | None = None,
                     ws: torch.Tensor | None = None) -> torch.Tensor:
    """Switch-style balancing loss and load statistics (see moe.h); with
    dlogits, its gradient is added into dlogits. Returns the device stats."""
    T, E = logits.shape
    _need(logits, (T, E), torch.float32, "logits")
    _need(counts, (E,), torch.int32, "counts")
    if stats is None:
        stats = torch.empty(MOE_LB_NSTATS, dtype=torch.float32, device=logits.device)
    if dlogits is not None:
        _need(dlogits, (T, E), torch.float32, "dlogits")
    wsb = moe_load_balance_workspace_size(T, E)
    if ws is None or ws.numel() < wsb:
        ws = torch.empty(max(wsb, 4), dtype=torch.uint8, device=logits.device)
    _check("moe_load_balance", _lib.moe_load_balance(
        _p(logits), _p(counts), T, E, k, float(alpha), _p(stats), _p(dlogits), _p(ws), ws.numel(),
        _stream()))
    return stats


class _Balance:
    """The optional balancing loss of a layer: statistics after routing in
    the forward, its gradient added into dlogits after the backward."""

    def __init__(self, alpha: float):
        self.alpha = alpha
        self.stats = None

    def forward(self, logits, counts, k, buf):
        """buf: the layer's buffers of this size (_Sizes)."""
        T, E = logits.shape
        if self.stats is None:
            self.stats = torch.empty(MOE_LB_NSTATS, dtype=torch.float32, device=logits.device)
        if "lb_ws" not in buf:
            wsb = max(moe_load_balance_workspace_size(T, E), 4)
            buf["lb_ws"] = torch.empty(wsb, dtype=torch.uint8, device=logits.device)
        self.ws = buf["lb_ws"]
        self.logits, self.counts, self.k = logits, counts, k
        return moe_load_balance(logits, counts, k, self.alpha, stats=self.stats, ws=self.ws)

    def backward(self, dlogits):
        moe_load_balance(self.logits, self.counts, self.k, self.alpha, stats=self.stats,
                         dlogits=dlogits, ws=self.ws)


class LayerNorm:
    """A layer norm with its gradient, in front of the layer (y is what the
    router and the layer take) or behind it (the layers' `out_norm`).

    weight, bias (may be None): [d] fp32. forward(x, residual) normalises x +
    residual and leaves that stream in `sum`. act8=True holds the normalised
    input from forward to backward as an 8-bit checkpoint (33/64 of its bf16
    size), written by the forward's kernel; otherwise the backward reads x (or
    sum), which the caller must leave as it was. Buffers are allocated at the
    first call with a size and reused: calls (or replays) of one object must
    not overlap in time. They stay for sizes that a captured graph uses, for
    the last one, and for small earlier ones (64 MiB in all)."""

    def __init__(self, weight: torch.Tensor, bias: torch.Tensor | None = None, eps: float = 1e-5,
                 act8: bool = False):
        self.weight, self.bias, self.eps, self.act8 = weight, bias, eps, act8
        self.sum = None
        self._sizes, self._key = _Sizes(), None

    def forward(self, x: torch.Tensor, residual: torch.Tensor | None = None) -> torch.Tensor:
        key = (x.shape, x.dtype, x.device, residual is None)
        if self._key != key:
            self._out = self.grads = self._key = None
            self._buf = self._sizes.at(key)
        buf = self._buf
        self._out = buf["out"] = moe_layer_norm(x, self.weight, self.bias, self.eps, residual,
                                                self.act8, out=buf.get("out"))
        _mark(buf, x.get_device())
        self._key = key
        self.sum = self._out.get("sum")
        self._x = None if self.act8 else (x if residual is None else self.sum)
        return self._out["y"]

    def backward(self, dy: torch.Tensor, dsum: torch.Tensor | None = None,
                 accumulate_dw: bool = False) -> dict:
        """dict of dx (the gradient of x and of the residual), dweight, dbias.
        dsum: the gradient that reaches sum by its other uses."""
        if self._key is None:
            raise ValueError("backward without a forward")
        if accumulate_dw and self.grads is None:
            raise ValueError("accumulate_dw needs the gradients of an earlier backward")
        buf = self._buf
        if "ws" not in buf:
            y = self._out["y"]
            wsb = moe_layer_norm_backward_workspace_size(_dt(y), *y.shape)
            buf["ws"] = torch.empty(max(wsb, 16), dtype=torch.uint8, device=y.device)
        self.grads = buf["grads"] = moe_layer_norm_backward(
            dict(self._out, x=self._x), dy, self.weight, dsum, out=buf.get("grads"),
            accumulate_dw=accumulate_dw, want_dbias=self.bias is not None, ws=buf["ws"])
        _mark(buf, dy.get_device())
        return self.grads

    def held_bytes(self) -> int:
        """Bytes held from forward to backward (x, or sum, is the caller's)."""
        o = self._out
        return _nbytes([o["mean"], o["rstd"], o.get("x8"), o.get("x8_scale")])


class RMSNorm:
    """A root-mean-square norm with its gradient, in front of the layer or
    behind it (the layers' `out_norm`): LayerNorm without a mean and a bias.

    weight: [d] fp32. forward(x, residual) normalises x + residual and leaves
    that stream in `sum`. quantize=True also writes y in MXFP8, left in `q` (a
    pair of elements and scales): what MoELayerMX.forward and
    MoELayerW4.prompt take as `xq` in place of quantising x themselves.
    act8=True and the buffers as in LayerNorm."""

    def __init__(self, weight: torch.Tensor, eps: float = 1e-6, act8: bool = False,
                 quantize: bool = False):
        self.weight, self.eps, self.act8, self.quantize = weight, eps, act8, quantize
        self.sum = self.q = None
        self._sizes, self._key = _Sizes(), None

    def forward(self, x: torch.Tensor, residual: torch.Tensor | None = None) -> torch.Tensor:
        key = (x.shape, x.dtype, x.device, residual is None, self.quantize, self.act8)
        if self._key != key:
            self._out = self.grads = self._key = None
            self._buf = self._sizes.at(key)
        buf = self._buf
        self._out = buf["out"] = moe_rms_norm(x, self.weight, self.eps, residual, self.quantize,
                                              act8=self.act8, out=buf.get("out"))
        _mark(buf, x.get_device())
        self._key = key
        self.sum = self._out.get("sum")
        self.q = (self._out["yq"], self._out["yq_scale"]) if self.quantize else None
        self._x = None if self.act8 else (x if residual is None else self.sum)
        return self._out["y"]

    def backward(self, dy: torch.Tensor, dsum: torch.Tensor | None = None,
                 accumulate_dw: bool = False) -> dict:
        """dict of dx (the gradient of x and of the residual) and dweight.
        dsum: the gradient that reaches sum by its other uses."""
        if self._key is None:
            raise ValueError("backward without a forward")
        if accumulate_dw and self.grads is None:
            raise ValueError("accumulate_dw needs the gradients of an earlier backward")
        buf = self._buf
        if "ws" not in buf:
            y = self._out["y"]
            wsb = moe_rms_norm_backward_workspace_size(_dt(y), *y.shape)
            buf["ws"] = torch.empty(max(wsb, 16), dtype=torch.uint8, device=y.device)
        self.grads = buf["grads"] = moe_rms_norm_backward(
            dict(self._out, x=self._x), dy, self.weight, dsum, out=buf.get("grads"),
            accumulate_dw=accumulate_dw, ws=buf["ws"])
        _mark(buf, dy.get_device())
        return self.grads

    def held_bytes(self) -> int:
        """Bytes held from forward to backward (x, or sum, is the caller's)."""
        o = self._out
        return _nbytes([o["rstd"], o.get("x8"), o.get("x8_scale")])


def _norm_backward(norm, dout, accumulate_dw):
    """dout taken back through a layer's out_norm."""
    if norm is None:
        return dout
    return norm.backward(dout, accumulate_dw=accumulate_dw)["dx"]


def _norm_grads(norm, grads):
    if norm is not None:
        grads["dnorm_weight"], grads["dnorm_bias"] = norm.grads["dweight"], norm.grads.get("dbias")
    return grads


def _use_buffers(obj, key, new):
    """The buffers of a size made the attributes of a layer object: new()'s,
    or those of an earlier call. Returns the key and the size's dict, which
    also keeps the gradients of the size's backward."""
    if obj._T == key:
        return key, obj._buf
    if obj._T is not None:                        # no old tensor is kept from being freed
        for name in obj._buf["tensors"]:
            obj.__dict__.pop(name, None)
        obj._T = obj._buf = None
    obj.grads = None
    buf = obj._sizes.at(key)
    if "tensors" not in buf:
        buf["tensors"] = new()
    obj.__dict__.update(buf["tensors"])
    return key, buf


def _act8_buffers(R, d, h, dev):
    """The checkpoints that a layer holds: of A||B and of y_perm."""
    ab8, ab8_scale = _act8_new(R, 2 * h, dev)
    y8, y8_scale = _act8_new(R, d, dev)
    return dict(ab8=ab8, ab8_scale=ab8_scale, y8=y8, y8_scale=y8_scale)


class MoELayer:
    """Forward and backward of the MoE expert layer through the C ABI.

    Buffers are allocated at the first call with a (T, dtype, device) and reused, so a step
    issues only kernel launches (no allocation, no device->host traffic) and can be captured
    in a HIP graph. They stay for sizes that a captured graph uses, for the last one, and for
    small earlier ones (64 MiB in all).

    recompute=True trades compute for activation memory (the trade-off the
    Olmo-core 3 report measures, kongchang.com "where the costs are"): the
    layer keeps only y_perm and the routing metadata from its forward to its
    backward. x_perm, A||B and H' are written to scratch shared by all
    recomputing layers of the shape, and the backward rebuilds them (permute,
    then GEMM1 + SwiGLU) before the layer's backward kernels run. The rebuilt
    tensors are bit-identical to the forward's, so are the gradients.

    aux_alpha adds the balancing loss of moe_load_balance: its statistics
    are in `lb_stats` (device) after forward, and backward adds its
    gradient to dlogits.

    act8=True holds 8-bit checkpoints (moe_act8_store) of A||B and y_perm and
    the routing metadata, nothing else: the backward dispatches x again,
    rebuilds A||B and H' from the checkpoint and reads y_perm's in the combine
    backward. The output is the plain layer's; the gradients are those of the
    rounded A||B and y_perm. x must be unchanged until the backward (as with
    recompute).

    What recompute and act8 rebuild lives in scratch shared by all such layers
    of a shape in the process. Layers whose work may overlap in time (on
    different streams, in graphs replayed side by side) need `scratch` dicts
    of their own; layers that run one after the other may share one.

    out_norm: a LayerNorm applied to the layer's output; the backward's dict
    then has dnorm_weight and dnorm_bias."""

    def __init__(self, w1: torch.Tensor, w2: torch.Tensor, k: int, recompute: bool = False,
                 aux_alpha: float | None = None, act8: bool = False,
                 scratch: dict | None = None, out_norm: LayerNorm | None = None):
        if recompute and act8:
            raise ValueError("recompute and act8 exclude each other")
        self.w1, self.w2, self.k = w1, w2, k
        self.E, h2, self.d = w1.shape
        self.h = h2 // 2
        self.recompute, self.act8 = recompute, act8
        self.scratch, self.out_norm = scratch, out_norm
        self.balance = _Balance(aux_alpha) if aux_alpha is not None else None
        self.lb_stats = None
        self._sizes, self._T = _Sizes(), None

    def _check_input(self, x, logits):
        if x.dim() != 2 or x.shape[1] != self.d:
            raise ValueError(f"x: expected [T, {self.d}], got {tuple(x.shape)}")
        if x.dtype != self.w1.dtype or self.w2.dtype != self.w1.dtype:
            raise ValueError(f"x ({x.dtype}) and the weights ({self.w1.dtype}, {self.w2.dtype}) "
                             "must share one dtype")
        if x.device != self.w1.device or x.device != self.w2.device or not x.is_cuda:
            raise ValueError("x and the weights must be on the same GPU")
        _need(x, (x.shape[0], self.d), x.dtype, "x")
        _need(logits, (x.shape[0], self.E), torch.float32, "logits")

    def _alloc(self, T, dev, dt):
        self._T, self._buf = _use_buffers(self, (T, dt, str(dev)), lambda: self._new(T, dev, dt))

    def _new(self, T, dev, dt) -> dict:
        """The tensors of a size, by the names that they have in the object."""
        E, k, d, h = self.E, self.k, self.d, self.h
        R = T * k
        i32 = dict(dtype=torch.int32, device=dev)
        route = dict(topk_idx=torch.empty((T, k), **i32),
                     topk_gate=torch.empty((T, k), dtype=torch.float32, device=dev),
                     counts=torch.empty(E, **i32), offsets=torch.empty(E + 1, **i32),
                     token_pos=torch.empty((T, k), **i32), sorted_token=torch.empty(R, **i32),
                     sorted_slot=torch.empty(R, **i32), tile_offsets=torch.empty(E + 1, **i32))
        own = (lambda name, shape: torch.empty(shape, dtype=dt, device=dev))
        tmp = ((lambda name, shape: _scratch(name, shape, dt, dev, self.scratch))
               if self.recompute or self.act8 else own)
        return dict(route=route,
                    route_ws=torch.empty(max(moe_route_workspace_size(T, E, k), 1),
                                         dtype=torch.uint8, device=dev),
                    x_perm=tmp("x_perm", (R, d)), ab=tmp("ab", (R, 2 * h)), hp=tmp("hp", (R, h)),
                    y_perm=(tmp if self.act8 else own)("y_perm", (R, d)),
                    ckpt=_act8_buffers(R, d, h, dev) if self.act8 else None,
                    out=torch.empty((T, d), dtype=dt, device=dev))

    def _gemm1(self, offsets):
        moe_grouped_gemm(MOE_GG_FWD, self.x_perm, self.w1, self.ab, offsets,
                         MOE_EPI_SWIGLU_FWD, N=2 * self.h, K=self.d, aux_out=self.hp)

    def forward(self, x: torch.Tensor, logits: torch.Tensor) -> torch.Tensor:
        self._check_input(x, logits)
        T, d = x.shape
        self._alloc(T, x.device, x.dtype)
        self.x = x
        r = moe_route(logits, self.k, out=self.route, ws=self.route_ws)
        if self.balance is not None:
            self.lb_stats = self.balance.forward(logits, r["counts"], self.k, self._buf)
        moe_permute(x, r["token_pos"], self.x_perm)
        self._gemm1(r["offsets"])
        if self.act8:
            moe_act8_store(self.ab, self.ckpt["ab8"], self.ckpt["ab8_scale"])
        moe_grouped_gemm(MOE_GG_FWD, self.hp, self.w2, self.y_perm, r["offsets"], N=d, K=self.h)
        if self.act8:
            moe_combine_act8(self.y_perm, r["topk_gate"], r["token_pos"], self.out,
                             self.ckpt["y8"], self.ckpt["y8_scale"])
        else:
            moe_combine(self.y_perm, r["topk_gate"], r["token_pos"], self.out)
        _mark(self._buf, x.get_device())
        return self.out if self.out_norm is None else self.out_norm.forward(self.out)

    def saved(self) -> dict:
        r = self.route
        return dict(x_perm=self.x_perm, ab=self.ab, hp=self.hp, y_perm=self.y_perm,
                    topk_gate=r["topk_gate"], topk_idx=r["topk_idx"], token_pos=r["token_pos"],
                    offsets=r["offsets"], w1=self.w1, w2=self.w2)

    def held_bytes(self) -> int:
        """Bytes of activations this layer holds from its forward to its
        backward (the input x and the weights are the caller's)."""
        r = self.route
        meta = _nbytes(r.values())
        if self.out_norm is not None:
            meta += self.out_norm.held_bytes() + (0 if self.out_norm.act8 else _nbytes([self.out]))
        if self.act8:
            return meta + _nbytes(self.ckpt.values())
        if self.recompute:
            return meta + _nbytes([self.y_perm])
        return meta + _nbytes([self.x_perm, self.ab, self.hp, self.y_perm])

    def backward(self, dout: torch.Tensor, accumulate_dw: bool = False,
                 stage_events=None) -> dict:
        """accumulate_dw: add this micro-batch's dW1, dW2 to the ones already
        in self.grads (gradient accumulation between optimizer steps).
        stage_events: optional recorded torch.cuda.Event per backward stage
        (moe_bwd_desc.stage_events)."""
        _need(dout, tuple(self.x.shape), self.x.dtype, "dout")
        if accumulate_dw and self.grads is None:
            raise ValueError("accumulate_dw needs the gradients of an earlier backward")
        dout = _norm_backward(self.out_norm, dout, accumulate_dw)
        if self.recompute or self.act8:
            moe_permute(self.x, self.route["token_pos"], self.x_perm)
        if self.recompute:
            self._gemm1(self.route["offsets"])
        self.grads = self._buf["grads"] = moe_backward(
            self.saved(), dout, self.E, self.k, self.d, self.h, out=self._buf.get("grads"),
            accumulate_dw=accumulate_dw, stage_events=stage_events, act8=self.ckpt)
        if self.balance is not None:
            self.balance.backward(self.grads["dlogits"])
        _mark(self._buf, dout.get_device())
        return _norm_grads(self.out_norm, self.grads)


class MoELayerPadded(MoELayer):
    """The padded-capacity alternative the report compares the dropless layer
    against: every expert owns `capacity` rows of [E*capacity, .] buffers,
    rows past an expert's capacity are dropped (no output, no gradient, gates
    not renormalised) and its unused rows are zero. Routing, dispatch, the
    grouped GEMMs, combine and the backward are the dropless layer's own
    kernels, run on the padded metadata, so only the padding differs."""

    def __init__(self, w1: torch.Tensor, w2: torch.Tensor, k: int, capacity: int):
        super().__init__(w1, w2, k)
        self.capacity = capacity

    def _new(self, T, dev, dt) -> dict:
        E, k, d, h, C = self.E, self.k, self.d, self.h, self.capacity
        P = max(E * C, 1)   # capacity 0 drops everything; keep the buffers non-null
        e = lambda *shape, dtype=dt: torch.empty(shape, dtype=dtype, device=dev)
        f32 = torch.float32
        return dict(super()._new(T, dev, dt), pad=dict(token_pos=e(T, k, dtype=torch.int32),
                                                       offsets=e(E + 1, dtype=torch.int32)),
                    x_perm=e(P, d), ab=e(P, 2 * h), hp=e(P, h), y_perm=e(P, d),
                    pad_grads=dict(dx=e(T, d), dlogits=e(T, E, dtype=f32),
                                   dw1=e(E, 2 * h, d, dtype=f32), dw2=e(E, d, h, dtype=f32),
                                   dgate=e(T, k, dtype=f32), dy_perm=e(P, d), dab=e(P, 2 * h),
                                   dx_perm=e(P, d)))

    def forward(self, x: torch.Tensor, logits: torch.Tensor) -> torch.Tensor:
        self._check_input(x, logits)
        T, d = x.shape
        C = self.capacity
        self._alloc(T, x.device, x.dtype)
        self.x = x
        r = moe_route(logits, self.k, out=self.route, ws=self.route_ws)
        p = moe_capacity_pad(r, C, out=self.pad)
        moe_permute(x, p["token_pos"], self.x_perm)
        moe_capacity_zero_rows(self.x_perm, r["offsets"], C)
        moe_grouped_gemm(MOE_GG_FWD, self.x_perm, self.w1, self.ab, p["offsets"],
                         MOE_EPI_SWIGLU_FWD, N=2 * self.h, K=d, aux_out=self.hp)
        moe_grouped_gemm(MOE_GG_FWD, self.hp, self.w2, self.y_perm, p["offsets"], N=d, K=self.h)
        moe_combine(self.y_perm, r["topk_gate"], p["token_pos"], self.out)
        _mark(self._buf, x.get_device())
        return self.out

    def saved(self) -> dict:
        sv = super().saved()
        sv["token_pos"] = self.pad["token_pos"]
        sv["offsets"] = self.pad["offsets"]
        return sv

    def backward(self, dout: torch.Tensor, accumulate_dw: bool = False,
                 stage_events=None) -> dict:
        self._buf["grads"] = self.pad_grads
        moe_capacity_zero_rows(self.pad_grads["dy_perm"], self.route["offsets"], self.capacity)
        return super().backward(dout, accumulate_dw, stage_events)


class MoELayerMX:
    """The layer with MXFP8 GEMMs and an MXFP8 dispatch payload.

    fp32 master weights are quantised once per weight update
    (`prepare_weights`), in both orientations: along d / h for the forward
    GEMMs and, per expert, along 2h / d for the backward dgrads. The forward
    quantises x along d before dispatch, so the row-wise dispatch moves E4M3
    bytes plus their scales; GEMM1 writes AB in bf16 and H' already
    quantised, along h for GEMM2 and along rows per expert for GEMM2's weight
    gradient (fuse_hp; with fuse_hp = False GEMM1 writes bf16 H' and a
    separate pass quantises it: the same bytes); y and out stay
    bf16. The backward (moe_backward with MXFP8) quantises its own GEMM
    operands.

    act8, scratch and out_norm as in MoELayer: with act8 the layer holds
    checkpoints of A||B and y_perm in their place (H' is held in MXFP8 along
    rows either way)."""

    def __init__(self, w1_master: torch.Tensor, w2_master: torch.Tensor, k: int,
                 recompute: bool = False, aux_alpha: float | None = None, act8: bool = False,
                 scratch: dict | None = None, out_norm: LayerNorm | None = None):
        if recompute and act8:
            raise ValueError("recompute and act8 exclude each other")
        self.E, h2, self.d = w1_master.shape
        self.h = h2 // 2
        self.k = k
        self.recompute, self.act8 = recompute, act8
        self.scratch, self.out_norm = scratch, out_norm
        self.fuse_hp = True
        self.balance = _Balance(aux_alpha) if aux_alpha is not None else None
        self.lb_stats = None
        self.w1q = self.w2q = None
        self.prepare_weights(w1_master, w2_master)
        self._sizes, self._T = _Sizes(), None

    def prepare_weights(self, w1: torch.Tensor, w2: torch.Tensor):
        """Re-quantise the fp32 masters, once per optimizer step: each master
        is read once and written in both orientations (mxfp8_quantize_both).
        Again into the same tensors, so that the replays of a captured step
        take the new weights (masters on another GPU get tensors there): the
        call must not overlap with the layer's others."""
        E, d, h = self.E, self.d, self.h
        dev = w1.device
        w1, w2 = w1.reshape(E * 2 * h, d), w2.reshape(E * d, h)
        old = self.w1q is not None and self.w1q.device == dev
        g1 = torch.arange(0, E + 1, dtype=torch.int32, device=dev) * (2 * h)
        g2 = torch.arange(0, E + 1, dtype=torch.int32, device=dev) * d
        (self.w1q, self.w1s), (self.w1t, self.w1ts) = mxfp8_quantize_both(
            w1, g1, out=(self.w1q, self.w1s, self.w1t, self.w1ts) if old else None)
        (self.w2q, self.w2s), (self.w2t, self.w2ts) = mxfp8_quantize_both(
            w2, g2, out=(self.w2q, self.w2s, self.w2t, self.w2ts) if old else None)

    def _alloc(self, T, dev):
        self._T, self._buf = _use_buffers(self, (T, str(dev)), lambda: self._new(T, dev))

    def _new(self, T, dev) -> dict:
        """The tensors of a size, by the names that they have in the object."""
        E, k, d, h = self.E, self.k, self.d, self.h
        R = T * k
        i32 = dict(dtype=torch.int32, device=dev)
        bf = dict(dtype=torch.bfloat16, device=dev)
        u8 = dict(dtype=torch.uint8, device=dev)
        route = dict(topk_idx=torch.empty((T, k), **i32),
                     topk_gate=torch.empty((T, k), dtype=torch.float32, device=dev),
                     counts=torch.empty(E, **i32), offsets=torch.empty(E + 1, **i32),
                     token_pos=torch.empty((T, k), **i32), sorted_token=torch.empty(R, **i32),
                     sorted_slot=torch.empty(R, **i32), tile_offsets=torch.empty(E + 1, **i32))
        # dispatch payload, A||B, H' and its MXFP8 copy: scratch when recomputing
        shared = lambda name, shape, dt: _scratch("mx_" + name, shape, dt, dev, self.scratch)
        tmp = (shared if self.recompute
               else (lambda name, shape, dt: torch.empty(shape, dtype=dt, device=dev)))
        # H' along rows per expert (GEMM2 wgrad's operand), written by GEMM1
        # with GEMM2's; held instead of bf16 H' (when recomputing, the backward
        # quantises the H' it recomputes and these are scratch)
        nb = mxfp8_col_blocks(R, E)
        if not self.recompute:
            hpc, hpcs = torch.empty(nb * 32 * h, **u8), torch.empty(nb * h, **u8)
        else:
            hpc = shared("hpc", (nb * 32 * h,), torch.uint8)
            hpcs = shared("hpcs", (nb * h,), torch.uint8)
        return dict(route=route,
                    route_ws=torch.empty(max(moe_route_workspace_size(T, E, k), 1), **u8),
                    xq=tmp("xq", (T, d), torch.uint8), xs=tmp("xs", (T, d // 32), torch.uint8),
                    xpq=tmp("xpq", (R, d), torch.uint8),
                    xps=tmp("xps", (R, d // 32), torch.uint8),
                    ab=(shared if self.act8 else tmp)("ab", (R, 2 * h), torch.bfloat16),
                    # H' and its GEMM2 operand are read in the forward only
                    hp=shared("hp", (R, h), torch.bfloat16),
                    hpq=shared("hpq", (R, h), torch.uint8),
                    hps=shared("hps", (R, h // 32), torch.uint8), hpc=hpc, hpcs=hpcs,
                    y_perm=(shared("y_perm", (R, d), torch.bfloat16) if self.act8
                            else torch.empty((R, d), **bf)),
                    ckpt=_act8_buffers(R, d, h, dev) if self.act8 else None,
                    out=torch.empty((T, d), **bf))

    def hp_quantised_in_gemm1(self) -> bool:
        """The forward's GEMM1 stores H' in both MXFP8 layouts (the backward's
        recomputation of GEMM1 stores bf16 H', which moe_backward quantises)."""
        return self.fuse_hp

    def _gemm1(self, x, offsets, token_pos, quantised_hp: bool = False, xq: tuple | None = None):
        """Quantised dispatch of x and GEMM1 + SwiGLU (forward, and again in
        the backward when recomputing). quantised_hp: H' goes straight to its
        two MXFP8 layouts instead of bf16."""
        if xq is None:
            mxfp8_quantize(x, 1, q=self.xq, scale=self.xs)
            xq = self.xq, self.xs
        moe_permute(xq[0], token_pos, self.xpq, x_scale=xq[1], x_perm_scale=self.xps)
        hp = (dict(aux_out=self.hpq, aux_out_scale=self.hps, aux_out_cols=self.hpc,
                   aux_out_cols_scale=self.hpcs) if quantised_hp else dict(aux_out=self.hp))
        moe_grouped_gemm(MOE_GG_FWD, self.xpq, self.w1q, self.ab, offsets, MOE_EPI_SWIGLU_FWD,
                         N=2 * self.h, K=self.d, a_scale=self.xps, b_scale=self.w1s,
                         dtype=MOE_MXFP8, **hp)

    def forward(self, x: torch.Tensor, logits: torch.Tensor, xq: tuple | None = None) -> torch.Tensor:
        """xq: x in MXFP8 along its rows (elements [T, d], scales [T, d/32]),
        where the norm in front has written it (RMSNorm.q), read during the
        forward only; else the layer quantises x. It must be x's own."""
        if x.dim() != 2 or x.shape[1] != self.d or x.dtype != torch.bfloat16:
            raise ValueError(f"x: expected bf16 [T, {self.d}], got {x.dtype} {tuple(x.shape)}")
        if x.device != self.w1q.device:
            raise ValueError("x and the weights must be on the same GPU")
        _need(x, tuple(x.shape), torch.bfloat16, "x")
        _need(logits, (x.shape[0], self.E), torch.float32, "logits")
        T, d = x.shape
        h = self.h
        if xq is not None:
            _act8_need(xq[0], xq[1], T, d, x.get_device(), "xq")
        self._alloc(T, x.device)
        self.x = x
        r = moe_route(logits, self.k, out=self.route, ws=self.route_ws)
        if self.balance is not None:
            self.lb_stats = self.balance.forward(logits, r["counts"], self.k, self._buf)
        fused = self.hp_quantised_in_gemm1()
        self._gemm1(x, r["offsets"], r["token_pos"], quantised_hp=fused, xq=xq)
        if self.act8:
            moe_act8_store(self.ab, self.ckpt["ab8"], self.ckpt["ab8_scale"])
        if not fused:
            self.quantize_hp(r["offsets"])
        moe_grouped_gemm(MOE_GG_FWD, self.hpq, self.w2q, self.y_perm, r["offsets"], N=d, K=h,
                         a_scale=self.hps, b_scale=self.w2s, dtype=MOE_MXFP8)
        if self.act8:
            moe_combine_act8(self.y_perm, r["topk_gate"], r["token_pos"], self.out,
                             self.ckpt["y8"], self.ckpt["y8_scale"])
        else:
            moe_combine(self.y_perm, r["topk_gate"], r["token_pos"], self.out)
        _mark(self._buf, x.get_device())
        return self.out if self.out_norm is None else self.out_norm.forward(self.out)

    def quantize_hp(self, offsets):
        """H' along h for GEMM2 and, unless recomputing (the backward then
        quantises the H' it recomputes), along rows per expert for GEMM2's
        weight gradient, both from one read."""
        if self.recompute:
            mxfp8_quantize(self.hp, 1, q=self.hpq, scale=self.hps)
        else:
            mxfp8_quantize_both(self.hp, offsets, out=(self.hpq, self.hps, self.hpc, self.hpcs))

    def saved(self) -> dict:
        r = self.route
        sv = dict(x=self.x, sorted_token=r["sorted_token"], ab=self.ab, hp=self.hp,
                  y_perm=self.y_perm, topk_gate=r["topk_gate"], topk_idx=r["topk_idx"],
                  token_pos=r["token_pos"], offsets=r["offsets"], w1t=self.w1t,
                  w1t_scale=self.w1ts, w2t=self.w2t, w2t_scale=self.w2ts)
        if not self.recompute:
            sv.update(hp=None, hp_cols=self.hpc, hp_cols_scale=self.hpcs)
        return sv

    def held_bytes(self) -> int:
        """Bytes of activations held from forward to backward (x and the
        weights are the caller's)."""
        meta = _nbytes(self.route.values())
        if self.out_norm is not None:
            meta += self.out_norm.held_bytes() + (0 if self.out_norm.act8 else _nbytes([self.out]))
        if self.act8:
            return meta + _nbytes([self.hpc, self.hpcs, *self.ckpt.values()])
        if self.recompute:
            return meta + _nbytes([self.y_perm])
        return meta + _nbytes([self.ab, self.hpc, self.hpcs, self.y_perm])

    def backward(self, dout: torch.Tensor, accumulate_dw: bool = False,
                 stage_events=None) -> dict:
        """accumulate_dw: add this micro-batch's dW1, dW2 to the ones already
        in self.grads. stage_events: as MoELayer.backward."""
        _need(dout, tuple(self.x.shape), torch.bfloat16, "dout")
        if accumulate_dw and self.grads is None:
            raise ValueError("accumulate_dw needs the gradients of an earlier backward")
        dout = _norm_backward(self.out_norm, dout, accumulate_dw)
        if self.recompute:
            self._gemm1(self.x, self.route["offsets"], self.route["token_pos"])
        self.grads = self._buf["grads"] = moe_backward(
            self.saved(), dout, self.E, self.k, self.d, self.h, out=self._buf.get("grads"),
            mxfp8=True, accumulate_dw=accumulate_dw, stage_events=stage_events, act8=self.ckpt)
        if self.balance is not None:
            self.balance.backward(self.grads["dlogits"])
        _mark(self._buf, dout.get_device())
        return _norm_grads(self.out_norm, self.grads)


class MoELayerW4:
    """The layer's forward for text generation: routing, then the experts
    with MXFP4 weights (moe_w4_experts), for a step's few tokens. w1 [E, 2h,
    d], w2 [E, d, h] (f32 or bf16) are quantised once and not kept. Buffers
    are allocated at the first call with a T and reused, so a step is kernel
    launches alone and can be captured in a HIP graph, one for each batch
    size; calls (or replays) of one layer object must not overlap in time,
    they share its buffers. Those stay for every T that a captured graph uses,
    for the last T, and for small earlier ones (64 MiB in all).

    prompt() is the same for a prompt's many tokens, with rows and H' in MXFP8
    (moe_w4_experts8; d and h multiples of 128)."""

    def __init__(self, w1: torch.Tensor, w2: torch.Tensor, k: int):
        self.E, h2, self.d = w1.shape
        self.h, self.k = h2 // 2, k
        self.w1q = self.w1s = self.w2q = self.w2s = None
        self.prepare_weights(w1, w2)
        self._sizes, self._T = _Sizes(), None

    def prepare_weights(self, w1: torch.Tensor, w2: torch.Tensor):
        """Quantise the weights, again after they have changed: into the same
        tensors, so that the replays of a captured step take the new ones
        (weights on another GPU get tensors there): the call must not overlap
        with the layer's others."""
        gpu = w1.get_device()
        _need_on(w1, (self.E, 2 * self.h, self.d), w1.dtype, gpu, "w1")
        _need_on(w2, (self.E, self.d, self.h), w2.dtype, gpu, "w2")
        if self.w1q is not None and self.w1q.device != w1.device:
            self.w1q = self.w1s = self.w2q = self.w2s = None
        self.w1q, self.w1s = moe_w4_quantize(w1, self.w1q, self.w1s)
        self.w2q, self.w2s = moe_w4_quantize(w2, self.w2q, self.w2s)

    def forward(self, x: torch.Tensor, logits: torch.Tensor) -> torch.Tensor:
        if x.dim() != 2 or x.shape[1] != self.d or x.dtype != torch.bfloat16:
            raise ValueError(f"x: expected bf16 [T, {self.d}], got {x.dtype} {tuple(x.shape)}")
        T, gpu = x.shape[0], self.w1q.get_device()
        _need_on(x, (T, self.d), torch.bfloat16, gpu, "x")
        buf = self._route(logits, T, gpu, (T, gpu), moe_w4_experts_workspace_size)
        self.out = moe_w4_experts(x, self.route, self.w1q, self.w1s, self.w2q, self.w2s,
                                  buf["out"], buf["ws"])
        _mark(buf, gpu)
        return self.out

    def prompt(self, x: torch.Tensor | None, logits: torch.Tensor,
               xq: tuple | None = None) -> torch.Tensor:
        """The forward of a prompt's T tokens. xq: x in MXFP8 along its rows
        (elements [T, d], scales [T, d/32]), where the norm in front has written
        it (RMSNorm.q); x may then be None. Else the layer quantises x (bf16)."""
        gpu, T = self.w1q.get_device(), logits.shape[0]
        if xq is None:
            _need_on(x, (T, self.d), torch.bfloat16, gpu, "x")
        else:
            _act8_need(xq[0], xq[1], T, self.d, gpu, "xq")
        buf = self._route(logits, T, gpu, (T, gpu, "prompt"), moe_w4_experts8_workspace_size)
        if xq is None:
            if "xq" not in buf:
                buf["xq"], buf["xs"] = _act8_new(T, self.d, self.w1q.device)
            xq = buf["xq"], buf["xs"]
            with torch.cuda.device(gpu):
                mxfp8_quantize(x, 1, q=xq[0], scale=xq[1])
        self.out = moe_w4_experts8(xq[0], xq[1], self.route, self.w1q, self.w1s, self.w2q, self.w2s,
                                   buf["out"], buf["ws"])
        _mark(buf, gpu)
        return self.out

    def _route(self, logits, T, gpu, key, ws_size) -> dict:
        """The buffers of a size, with the routing of its logits in them."""
        _need_on(logits, (T, self.E), torch.float32, gpu, "logits")
        if self._T != key:
            self._buf, self._T = self._sizes.at(key), key
        buf, dev = self._buf, self.w1q.device
        with torch.cuda.device(gpu):
            if "out" not in buf:
                self.route = self.route_ws = self.ws = self.out = None
                u8 = lambda n: torch.empty(n, dtype=torch.uint8, device=dev)
                wsb = ws_size(T, self.k, self.d, self.h)
                buf.update(route=None, out=torch.empty((T, self.d), dtype=torch.bfloat16, device=dev),
                           route_ws=u8(max(moe_route_workspace_size(T, self.E, self.k), 1)),
                           ws=u8(max(wsb, 16)))
            self.route = buf["route"] = moe_route(logits, self.k, out=buf["route"],
                                                  ws=buf["route_ws"])
        self.route_ws, self.ws = buf["route_ws"], buf["ws"]
        return buf
