"""Python binding of the GB300 FP8 linear-layer library (libfp8gb.so).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  PyTorch provides device memory and the current stream.  If the
library is missing, every entry point raises -- there is no fallback.

The C ABI (include/fp8gb.h) is mirrored one to one:

  fp8_quantize             fused amax + scale + saturating cast, rowwise and
                           colwise-transposed layouts from one read
  fp8_update_amax_history  delayed-scaling history roll + scale update
  fp8_scaled_gemm          FP8 x FP8 -> bf16 with scales in the epilogue
  fp8_grouped_gemm         the same over MoE expert groups
  fp8_group_padded_offsets host helper for the grouped colwise layout
  fp8_sync_status          stream sync + device error word
  fp8_norm_forward         layer / RMS norm, optionally with an 8-bit
                           checkpoint of the normalized rows
  fp8_norm_backward        its backward, from x or from the checkpoint
  fp8_swiglu_checkpoint    SwiGLU that stores gate|up in 8 bits
  fp8_swiglu_backward      its backward, from gate|up or from the checkpoint
  fp8_checkpoint[_restore] any activation to 8 bits and back
  fp8[_mx]_norm_quantize   residual add, norm and quantize in one read
  fp8_residual_norm_backward  fp8_norm_backward plus the gradient past the norm
  fp8[_mx]_swiglu_gemm     gate|up product with the SwiGLU in its epilogue
  fp8[_mx]_swiglu_gemm_backward  dh product with its backward in the epilogue

`quantize`, `scaled_gemm`, `grouped_gemm` are convenience wrappers that
allocate the outputs with torch and call the entry points above.
"""
from __future__ import annotations

import ctypes
import os
import threading
from dataclasses import dataclass

import torch

E4M3FN, E5M2, E4M3FNUZ, E5M2FNUZ = 0, 1, 2, 3
DELAYED, TENSORWISE, ROWWISE = 0, 1, 2
MOST_RECENT, MAX = 0, 1
LAYOUT_ROW, LAYOUT_COLT = 1, 2
SCALE_TENSOR, SCALE_PER_ROW = 0, 1
GROUPED_M, GROUPED_K, GROUPED_M_BT = 0, 1, 2
LAYER_NORM, RMS_NORM = 0, 1
DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
STATUS = {0: "FP8_OK", 1: "FP8_ERR_INVALID_ARG", 2: "FP8_ERR_UNSUPPORTED", 3: "FP8_ERR_ALIGNMENT",
          4: "FP8_ERR_CUDA", 5: "FP8_ERR_TIMEOUT"}

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfp8gb.so")
EXPORTED = ("fp8_quantize", "fp8_update_amax_history", "fp8_scaled_gemm", "fp8_grouped_gemm",
            "fp8_group_padded_offsets", "fp8_sync_status", "fp8_selftest_bounded_wait", "fp8_status_string",
            "fp8_last_cuda_error", "fp8_version", "fp8_mx_scale_bytes", "fp8_mx_quantize", "fp8_mx_gemm",
            "fp8_mx_grouped_gemm", "fp8_mx_permute_quantize", "fp8_mx_swiglu_quantize", "fp8_blockwise_quantize",
            "fp8_quantize_rowwise_resident", "fp8_permute_quantize", "fp8_swiglu_quantize", "fp8_checkpoint",
            "fp8_checkpoint_restore", "fp8_swiglu_checkpoint", "fp8_swiglu_backward", "fp8_norm_forward",
            "fp8_norm_workspace_bytes", "fp8_norm_backward", "fp8_norm_quantize", "fp8_mx_norm_quantize",
            "fp8_residual_norm_backward", "fp8_swiglu_gemm", "fp8_mx_swiglu_gemm", "fp8_swiglu_gemm_backward",
            "fp8_mx_swiglu_gemm_backward")
MX_BLOCK = 32
MX_GROUP_ALIGN = 128

_lock = threading.Lock()
_lib = None


class Fp8Error(RuntimeError):
    def __init__(self, status: int, where: str, detail: str = ""):
        self.status = status
        msg = f"{where}: {STATUS.get(status, status)}"
        if detail:
            msg += f" ({detail})"
        super().__init__(msg)


class fp8_recipe_t(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int), ("margin", ctypes.c_int), ("history_len", ctypes.c_int),
                ("algo", ctypes.c_int)]


@dataclass
class Recipe:
    """The recipe knobs: kind (DELAYED / TENSORWISE / ROWWISE), margin,
    history_len, algo (MOST_RECENT / MAX)."""
    kind: int = DELAYED
    margin: int = 0
    history_len: int = 1024
    algo: int = MOST_RECENT

    def c(self) -> fp8_recipe_t:
        return fp8_recipe_t(self.kind, self.margin, self.history_len, self.algo)


def format_for(fp8: str, role: str) -> int:
    """FP8 format of a tensor role under the "e4m3" or "hybrid" setting:
    hybrid keeps activations and weights in E4M3 and gradients in E5M2."""
    if fp8 == "e4m3":
        return E4M3FN
    if fp8 == "hybrid":
        return E5M2 if role in ("grad", "grad_output", "dy") else E4M3FN
    raise ValueError(f"unknown fp8 setting {fp8!r}")


def load_library():
    """Load libfp8gb.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is missing: build it with fp8_mixed_precision_scale_gb300.build")
            lib = ctypes.CDLL(LIB_PATH)
            P, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
            lib.fp8_quantize.restype = i32
            lib.fp8_quantize.argtypes = [P, i64, i64, i64, i32, ctypes.POINTER(fp8_recipe_t), i32, P, P, P, P, P,
                                         i64, P, P, i32, P]
            lib.fp8_quantize_rowwise_resident.restype = i32
            lib.fp8_quantize_rowwise_resident.argtypes = [P, i64, i64, i64, i32, i32, i32, P, P, P, P, i64, P, P]
            lib.fp8_permute_quantize.restype = i32
            lib.fp8_permute_quantize.argtypes = [P, i64, i64, i64, P, i64, i32, i32, i32, P, P, P, P, i64, P, P, i32,
                                                 P]
            lib.fp8_swiglu_quantize.restype = i32
            lib.fp8_swiglu_quantize.argtypes = [P, i64, i64, i64, i32, i32, i32, P, i64, P, P, P, P, i64, P, P, i32, P]
            lib.fp8_update_amax_history.restype = i32
            lib.fp8_update_amax_history.argtypes = [P, P, P, P, i32, i32, i32, i32, P, P]
            lib.fp8_scaled_gemm.restype = i32
            lib.fp8_scaled_gemm.argtypes = [P, i32, i64, P, i32, i64, i64, i64, i64, P, i32, P, i32, P, i64, P]
            lib.fp8_grouped_gemm.restype = i32
            lib.fp8_grouped_gemm.argtypes = [i32, P, i32, P, i32, P, i32, i64, i64, i64, P, i32, P, i32, P, i64, P]
            lib.fp8_group_padded_offsets.restype = i64
            lib.fp8_group_padded_offsets.argtypes = [P, i32, i32, P]
            lib.fp8_sync_status.restype = i32
            lib.fp8_sync_status.argtypes = [P]
            lib.fp8_selftest_bounded_wait.restype = i32
            lib.fp8_selftest_bounded_wait.argtypes = [i64, P]
            lib.fp8_status_string.restype = ctypes.c_char_p
            lib.fp8_status_string.argtypes = [i32]
            lib.fp8_last_cuda_error.restype = ctypes.c_char_p
            lib.fp8_last_cuda_error.argtypes = []
            lib.fp8_version.restype = ctypes.c_char_p
            lib.fp8_version.argtypes = []
            lib.fp8_mx_scale_bytes.restype = i64
            lib.fp8_mx_scale_bytes.argtypes = [i64, i64]
            lib.fp8_mx_quantize.restype = i32
            lib.fp8_mx_quantize.argtypes = [P, i64, i64, i64, i32, i32, P, P, P, i64, P, P, i32, P]
            lib.fp8_mx_permute_quantize.restype = i32
            lib.fp8_mx_permute_quantize.argtypes = [P, i64, i64, i64, P, i64, i32, i32, P, P, P, i64, P, P, i32, P]
            lib.fp8_mx_swiglu_quantize.restype = i32
            lib.fp8_mx_swiglu_quantize.argtypes = [P, i64, i64, i64, i32, i32, P, i64, P, P, P, i64, P, P, i32, P]
            lib.fp8_blockwise_quantize.restype = i32
            lib.fp8_blockwise_quantize.argtypes = [P, i64, i64, i64, i32, i32, i32, P, P, P, i64, P, P]
            f32 = ctypes.c_float
            lib.fp8_checkpoint.restype = i32
            lib.fp8_checkpoint.argtypes = [P, i32, i64, i64, i64, i32, i32, P, i64, P, i64, P]
            lib.fp8_checkpoint_restore.restype = i32
            lib.fp8_checkpoint_restore.argtypes = [P, i64, P, i64, i32, i64, i64, i32, P, i32, i64, P]
            lib.fp8_swiglu_checkpoint.restype = i32
            lib.fp8_swiglu_checkpoint.argtypes = [P, i64, i64, i64, i32, P, i64, P, i64, P, i64, P]
            lib.fp8_swiglu_backward.restype = i32
            lib.fp8_swiglu_backward.argtypes = [P, i64, P, i64, P, i64, P, i64, i32, i64, i64, P, i64, P, i64, P]
            lib.fp8_norm_forward.restype = i32
            lib.fp8_norm_forward.argtypes = [P, i32, i64, i64, i64, i32, f32, P, P, i32, P, i32, i64, P, P, i32, P,
                                             i64, P, i64, P]
            lib.fp8_norm_workspace_bytes.restype = i64
            lib.fp8_norm_workspace_bytes.argtypes = [i64, i64]
            lib.fp8_norm_backward.restype = i32
            lib.fp8_norm_backward.argtypes = [P, i32, i64, P, i64, P, i64, P, i64, i32, i64, i64, i32, P, P, P, i32, P,
                                              i32, i64, P, P, P, i64, P]
            lib.fp8_norm_quantize.restype = i32
            lib.fp8_norm_quantize.argtypes = [P, i32, i64, P, i32, i64, i64, i64, i32, f32, P, P, i32, P, i64, P, P,
                                              i32, ctypes.POINTER(fp8_recipe_t), i32, P, P, P, P, P, i64, P, P]
            lib.fp8_mx_norm_quantize.restype = i32
            lib.fp8_mx_norm_quantize.argtypes = [P, i32, i64, P, i32, i64, i64, i64, i32, f32, P, P, i32, P, i64, P,
                                                 P, i32, i32, P, P, P, i64, P, P]
            lib.fp8_residual_norm_backward.restype = i32
            lib.fp8_residual_norm_backward.argtypes = [P, i32, i64, P, i64, P, i64, P, i64, i32, P, i64, i64, i64,
                                                       i32, P, P, P, i32, P, i32, i64, P, P, P, i64, P]
            lib.fp8_swiglu_gemm.restype = i32
            lib.fp8_swiglu_gemm.argtypes = [P, i32, i64, P, i32, i64, i64, i64, i64, P, i32, P, i32, i32, i32, P, P,
                                            P, P, i64, P, P, i64, P, i64, i32, P, i64, P, i64, P]
            lib.fp8_mx_swiglu_gemm.restype = i32
            lib.fp8_mx_swiglu_gemm.argtypes = [P, i32, i64, P, P, i32, i64, P, i64, i64, i64, i32, i32, P, P, P, i64,
                                               P, P, i64, P, i64, i32, P, i64, P, i64, P]
            lib.fp8_swiglu_gemm_backward.restype = i32
            lib.fp8_swiglu_gemm_backward.argtypes = [P, i32, i64, P, i32, i64, i64, i64, i64, P, i32, P, i32, P, i64,
                                                     P, i64, P, i64, i32, i32, i32, P, P, P, P, i64, P, P, i64, P]
            lib.fp8_mx_swiglu_gemm_backward.restype = i32
            lib.fp8_mx_swiglu_gemm_backward.argtypes = [P, i32, i64, P, P, i32, i64, P, i64, i64, i64, P, i64, P,
                                                        i64, P, i64, i32, i32, i32, P, P, P, i64, P, P, i64, P]
            lib.fp8_mx_gemm.restype = i32
            lib.fp8_mx_gemm.argtypes = [P, i32, i64, P, P, i32, i64, P, i64, i64, i64, P, i64, P]
            lib.fp8_mx_grouped_gemm.restype = i32
            lib.fp8_mx_grouped_gemm.argtypes = [i32, P, i32, P, P, i32, P, P, i32, i64, i64, i64, P, i64, P]
            _lib = lib
    return _lib


# Addresses go to ctypes as plain integers (its c_void_p arguments take them);
# a c_void_p object around each costs a small call microseconds in all.
def _p(t):
    return t if t is None or isinstance(t, int) else t.data_ptr()


def _stream(stream):
    if stream is None:
        # the handle alone: torch.cuda.current_stream() builds a Stream object around it (3 us)
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _check(status: int, where: str):
    if status != 0:
        detail = load_library().fp8_last_cuda_error().decode() if status == 4 else ""
        raise Fp8Error(status, where, detail)


# --- the C entry points ------------------------------------------------------

def fp8_quantize(x, rows, cols, ld_x, fmt, recipe: Recipe, layouts, scale_in, amax_out, q_row, scale_inv_row,
                 q_colT, ld_colT, scale_inv_col, group_offsets=None, num_groups=0, stream=None, check=True):
    rc = load_library().fp8_quantize(_p(x), rows, cols, ld_x, fmt, ctypes.byref(recipe.c()), layouts,
                                     _p(scale_in), _p(amax_out), _p(q_row), _p(scale_inv_row), _p(q_colT),
                                     ld_colT, _p(scale_inv_col), _p(group_offsets), num_groups, _stream(stream))
    if check:
        _check(rc, "fp8_quantize")
    return rc


def fp8_update_amax_history(hist, scale, scale_inv, fmt, n, L, algo, margin, nonfinite_count=None, stream=None,
                            check=True):
    rc = load_library().fp8_update_amax_history(_p(hist), _p(scale), _p(scale_inv), _p(fmt), n, L, algo, margin,
                                                _p(nonfinite_count), _stream(stream))
    if check:
        _check(rc, "fp8_update_amax_history")
    return rc


def fp8_scaled_gemm(A, fa, lda, B, fb, ldb, M, N, K, sa, sa_mode, sb, sb_mode, C, ldc, stream=None, check=True):
    rc = load_library().fp8_scaled_gemm(_p(A), fa, lda, _p(B), fb, ldb, M, N, K, _p(sa), sa_mode, _p(sb), sb_mode,
                                        _p(C), ldc, _stream(stream))
    if check:
        _check(rc, "fp8_scaled_gemm")
    return rc


def fp8_grouped_gemm(mode, A, fa, B, fb, group_offsets, G, M_total, N, K, sa, sa_mode, sb, sb_mode, C, ld_T=0,
                     stream=None, check=True):
    rc = load_library().fp8_grouped_gemm(mode, _p(A), fa, _p(B), fb, _p(group_offsets), G, M_total, N, K, _p(sa),
                                         sa_mode, _p(sb), sb_mode, _p(C), ld_T, _stream(stream))
    if check:
        _check(rc, "fp8_grouped_gemm")
    return rc


def fp8_group_padded_offsets(host_offsets, align: int = 32):
    """int32 CPU offsets [G+1] -> (total, int64 CPU padded offsets [G+1])."""
    off = torch.as_tensor(host_offsets, dtype=torch.int32).contiguous().cpu()
    G = off.numel() - 1
    out = torch.zeros(G + 1, dtype=torch.int64)
    total = load_library().fp8_group_padded_offsets(_p(off), G, align, _p(out))
    if total < 0:
        raise Fp8Error(1, "fp8_group_padded_offsets")
    return int(total), out


def fp8_mx_scale_bytes(scale_rows: int, blocks: int) -> int:
    return int(load_library().fp8_mx_scale_bytes(scale_rows, blocks))


def fp8_mx_quantize(x, rows, cols, ld_x, fmt, layouts, q_row, s_row, q_colT, ld_colT, s_col, group_offsets=None,
                    num_groups=0, stream=None, check=True):
    rc = load_library().fp8_mx_quantize(_p(x), rows, cols, ld_x, fmt, layouts, _p(q_row), _p(s_row), _p(q_colT),
                                        ld_colT, _p(s_col), _p(group_offsets), num_groups, _stream(stream))
    if check:
        _check(rc, "fp8_mx_quantize")
    return rc


def fp8_mx_permute_quantize(x, x_rows, cols, ld_x, src_rows, rows, fmt, layouts, q_row, s_row, q_colT, ld_colT,
                            s_col, group_offsets=None, num_groups=0, stream=None, check=True):
    rc = load_library().fp8_mx_permute_quantize(_p(x), x_rows, cols, ld_x, _p(src_rows), rows, fmt, layouts,
                                                _p(q_row), _p(s_row), _p(q_colT), ld_colT, _p(s_col),
                                                _p(group_offsets), num_groups, _stream(stream))
    if check:
        _check(rc, "fp8_mx_permute_quantize")
    return rc


def fp8_mx_swiglu_quantize(gate_up, rows, F, ld, fmt, layouts, h, ld_h, q_row, s_row, q_colT, ld_colT, s_col,
                           group_offsets=None, num_groups=0, stream=None, check=True):
    rc = load_library().fp8_mx_swiglu_quantize(_p(gate_up), rows, F, ld, fmt, layouts, _p(h), ld_h, _p(q_row),
                                               _p(s_row), _p(q_colT), ld_colT, _p(s_col), _p(group_offsets),
                                               num_groups, _stream(stream))
    if check:
        _check(rc, "fp8_mx_swiglu_quantize")
    return rc


def fp8_quantize_rowwise_resident(x, rows, cols, ld_x, fmt, margin, layouts, amax_out, q_row, scale_inv_row, q_colT,
                                  ld_colT, scale_inv_col, stream=None, check=True):
    rc = load_library().fp8_quantize_rowwise_resident(_p(x), rows, cols, ld_x, fmt, margin, layouts, _p(amax_out),
                                                      _p(q_row), _p(scale_inv_row), _p(q_colT), ld_colT,
                                                      _p(scale_inv_col), _stream(stream))
    if check:
        _check(rc, "fp8_quantize_rowwise_resident")
    return rc


def fp8_permute_quantize(x, x_rows, cols, ld_x, src_rows, rows, fmt, margin, layouts, amax_out, q_row,
                         scale_inv_row, q_colT, ld_colT, scale_inv_col, group_offsets, num_groups, stream=None,
                         check=True):
    rc = load_library().fp8_permute_quantize(_p(x), x_rows, cols, ld_x, _p(src_rows), rows, fmt, margin, layouts,
                                             _p(amax_out), _p(q_row), _p(scale_inv_row), _p(q_colT), ld_colT,
                                             _p(scale_inv_col), _p(group_offsets), num_groups, _stream(stream))
    if check:
        _check(rc, "fp8_permute_quantize")
    return rc


def fp8_swiglu_quantize(gate_up, rows, F, ld, fmt, margin, layouts, h, ld_h, amax_out, q_row, scale_inv_row,
                        q_colT, ld_colT, scale_inv_col, group_offsets, num_groups, stream=None, check=True):
    rc = load_library().fp8_swiglu_quantize(_p(gate_up), rows, F, ld, fmt, margin, layouts, _p(h), ld_h,
                                            _p(amax_out), _p(q_row), _p(scale_inv_row), _p(q_colT), ld_colT,
                                            _p(scale_inv_col), _p(group_offsets), num_groups, _stream(stream))
    if check:
        _check(rc, "fp8_swiglu_quantize")
    return rc


def fp8_blockwise_quantize(x, rows, cols, ld_x, fmt, block_rows, layouts, q_row, s_row, q_colT, ld_colT, s_col,
                           stream=None, check=True):
    rc = load_library().fp8_blockwise_quantize(_p(x), rows, cols, ld_x, fmt, block_rows, layouts, _p(q_row),
                                               _p(s_row), _p(q_colT), ld_colT, _p(s_col), _stream(stream))
    if check:
        _check(rc, "fp8_blockwise_quantize")
    return rc


def fp8_mx_gemm(A, fa, lda, sA, B, fb, ldb, sB, M, N, K, C, ldc, stream=None, check=True):
    rc = load_library().fp8_mx_gemm(_p(A), fa, lda, _p(sA), _p(B), fb, ldb, _p(sB), M, N, K, _p(C), ldc,
                                    _stream(stream))
    if check:
        _check(rc, "fp8_mx_gemm")
    return rc


def fp8_mx_grouped_gemm(mode, A, fa, sA, B, fb, sB, group_offsets, G, M_total, N, K, C, ld_T=0, stream=None,
                        check=True):
    rc = load_library().fp8_mx_grouped_gemm(mode, _p(A), fa, _p(sA), _p(B), fb, _p(sB), _p(group_offsets), G,
                                            M_total, N, K, _p(C), ld_T, _stream(stream))
    if check:
        _check(rc, "fp8_mx_grouped_gemm")
    return rc


def fp8_checkpoint(x, dtype, rows, cols, ld_x, parts, fmt, q, ld_q, s, ld_s, stream=None, check=True):
    rc = load_library().fp8_checkpoint(_p(x), dtype, rows, cols, ld_x, parts, fmt, _p(q), ld_q, _p(s), ld_s,
                                       _stream(stream))
    if check:
        _check(rc, "fp8_checkpoint")
    return rc


def fp8_checkpoint_restore(q, ld_q, s, ld_s, fmt, rows, cols, parts, x, dtype, ld_x, stream=None, check=True):
    rc = load_library().fp8_checkpoint_restore(_p(q), ld_q, _p(s), ld_s, fmt, rows, cols, parts, _p(x), dtype, ld_x,
                                               _stream(stream))
    if check:
        _check(rc, "fp8_checkpoint_restore")
    return rc


def fp8_swiglu_checkpoint(gate_up, rows, F, ld, fmt, h, ld_h, q, ld_q, s, ld_s, stream=None, check=True):
    rc = load_library().fp8_swiglu_checkpoint(_p(gate_up), rows, F, ld, fmt, _p(h), ld_h, _p(q), ld_q, _p(s), ld_s,
                                              _stream(stream))
    if check:
        _check(rc, "fp8_swiglu_checkpoint")
    return rc


def fp8_swiglu_backward(dh, ld_dh, gate_up, ld, q, ld_q, s, ld_s, fmt, rows, F, d_gate_up, ld_d, h=None, ld_h=0,
                        stream=None, check=True):
    rc = load_library().fp8_swiglu_backward(_p(dh), ld_dh, _p(gate_up), ld, _p(q), ld_q, _p(s), ld_s, fmt, rows, F,
                                            _p(d_gate_up), ld_d, _p(h), ld_h, _stream(stream))
    if check:
        _check(rc, "fp8_swiglu_backward")
    return rc


def fp8_norm_forward(x, x_dtype, ld_x, rows, cols, kind, eps, weight, bias, w_dtype, y, y_dtype, ld_y, mean, rstd,
                     fmt=0, q=None, ld_q=0, s=None, ld_s=0, stream=None, check=True):
    rc = load_library().fp8_norm_forward(_p(x), x_dtype, ld_x, rows, cols, kind, eps, _p(weight), _p(bias), w_dtype,
                                         _p(y), y_dtype, ld_y, _p(mean), _p(rstd), fmt, _p(q), ld_q, _p(s), ld_s,
                                         _stream(stream))
    if check:
        _check(rc, "fp8_norm_forward")
    return rc


def fp8_norm_workspace_bytes(rows: int, cols: int) -> int:
    return int(load_library().fp8_norm_workspace_bytes(rows, cols))


def fp8_norm_backward(dy, y_dtype, ld_dy, x, ld_x, q, ld_q, s, ld_s, fmt, rows, cols, kind, mean, rstd, weight,
                      w_dtype, dx, x_dtype, ld_dx, dweight, dbias, workspace, workspace_bytes, stream=None,
                      check=True):
    rc = load_library().fp8_norm_backward(_p(dy), y_dtype, ld_dy, _p(x), ld_x, _p(q), ld_q, _p(s), ld_s, fmt, rows,
                                          cols, kind, _p(mean), _p(rstd), _p(weight), w_dtype, _p(dx), x_dtype, ld_dx,
                                          _p(dweight), _p(dbias), _p(workspace), workspace_bytes, _stream(stream))
    if check:
        _check(rc, "fp8_norm_backward")
    return rc


def fp8_norm_quantize(x, x_dtype, ld_x, residual, r_dtype, ld_r, rows, cols, kind, eps, weight, bias, w_dtype, sum,
                      ld_sum, mean, rstd, fmt, recipe: Recipe, layouts, scale_in, amax_out, q_row, scale_inv_row,
                      q_colT, ld_colT, scale_inv_col, stream=None, check=True):
    rc = load_library().fp8_norm_quantize(_p(x), x_dtype, ld_x, _p(residual), r_dtype, ld_r, rows, cols, kind, eps,
                                          _p(weight), _p(bias), w_dtype, _p(sum), ld_sum, _p(mean), _p(rstd), fmt,
                                          ctypes.byref(recipe.c()), layouts, _p(scale_in), _p(amax_out), _p(q_row),
                                          _p(scale_inv_row), _p(q_colT), ld_colT, _p(scale_inv_col), _stream(stream))
    if check:
        _check(rc, "fp8_norm_quantize")
    return rc


def fp8_mx_norm_quantize(x, x_dtype, ld_x, residual, r_dtype, ld_r, rows, cols, kind, eps, weight, bias, w_dtype, sum,
                         ld_sum, mean, rstd, fmt, layouts, q_row, s_row, q_colT, ld_colT, s_col, stream=None,
                         check=True):
    rc = load_library().fp8_mx_norm_quantize(_p(x), x_dtype, ld_x, _p(residual), r_dtype, ld_r, rows, cols, kind, eps,
                                             _p(weight), _p(bias), w_dtype, _p(sum), ld_sum, _p(mean), _p(rstd), fmt,
                                             layouts, _p(q_row), _p(s_row), _p(q_colT), ld_colT, _p(s_col),
                                             _stream(stream))
    if check:
        _check(rc, "fp8_mx_norm_quantize")
    return rc


def fp8_residual_norm_backward(dy, y_dtype, ld_dy, x, ld_x, q, ld_q, s, ld_s, fmt, dsum, ld_dsum, rows, cols, kind,
                               mean, rstd, weight, w_dtype, dx, x_dtype, ld_dx, dweight, dbias, workspace,
                               workspace_bytes, stream=None, check=True):
    rc = load_library().fp8_residual_norm_backward(_p(dy), y_dtype, ld_dy, _p(x), ld_x, _p(q), ld_q, _p(s), ld_s, fmt,
                                                   _p(dsum), ld_dsum, rows, cols, kind, _p(mean), _p(rstd),
                                                   _p(weight), w_dtype, _p(dx), x_dtype, ld_dx, _p(dweight),
                                                   _p(dbias), _p(workspace), workspace_bytes, _stream(stream))
    if check:
        _check(rc, "fp8_residual_norm_backward")
    return rc


def fp8_swiglu_gemm(A, fa, lda, W, fw, ldw, M, F, K, sa, sa_mode, sw, sw_mode, fmt=0, layouts=0, scale_in=None,
                    amax_out=None, q_row=None, q_colT=None, ld_colT=0, scale_inv=None, h=None, ld_h=0, gate_up=None,
                    ld_gu=0, ckpt_fmt=0, q=None, ld_q=0, s=None, ld_s=0, stream=None, check=True):
    rc = load_library().fp8_swiglu_gemm(_p(A), fa, lda, _p(W), fw, ldw, M, F, K, _p(sa), sa_mode, _p(sw), sw_mode,
                                        fmt, layouts, _p(scale_in), _p(amax_out), _p(q_row), _p(q_colT), ld_colT,
                                        _p(scale_inv), _p(h), ld_h, _p(gate_up), ld_gu, ckpt_fmt, _p(q), ld_q, _p(s),
                                        ld_s, _stream(stream))
    if check:
        _check(rc, "fp8_swiglu_gemm")
    return rc


def fp8_mx_swiglu_gemm(A, fa, lda, sA, W, fw, ldw, sW, M, F, K, fmt=0, layouts=0, q_row=None, s_row=None, q_colT=None,
                       ld_colT=0, s_col=None, h=None, ld_h=0, gate_up=None, ld_gu=0, ckpt_fmt=0, q=None, ld_q=0,
                       s=None, ld_s=0, stream=None, check=True):
    rc = load_library().fp8_mx_swiglu_gemm(_p(A), fa, lda, _p(sA), _p(W), fw, ldw, _p(sW), M, F, K, fmt, layouts,
                                           _p(q_row), _p(s_row), _p(q_colT), ld_colT, _p(s_col), _p(h), ld_h,
                                           _p(gate_up), ld_gu, ckpt_fmt, _p(q), ld_q, _p(s), ld_s, _stream(stream))
    if check:
        _check(rc, "fp8_mx_swiglu_gemm")
    return rc


def fp8_swiglu_gemm_backward(A, fa, lda, B, fb, ldb, M, F, K, sa, sa_mode, sb, sb_mode, gate_up=None, ld_gu=0, q=None,
                             ld_q=0, s=None, ld_s=0, ckpt_fmt=0, fmt=0, layouts=0, scale_in=None, amax_out=None,
                             q_row=None, q_colT=None, ld_colT=0, scale_inv=None, d_gate_up=None, ld_d=0, stream=None,
                             check=True):
    rc = load_library().fp8_swiglu_gemm_backward(_p(A), fa, lda, _p(B), fb, ldb, M, F, K, _p(sa), sa_mode, _p(sb),
                                                 sb_mode, _p(gate_up), ld_gu, _p(q), ld_q, _p(s), ld_s, ckpt_fmt, fmt,
                                                 layouts, _p(scale_in), _p(amax_out), _p(q_row), _p(q_colT), ld_colT,
                                                 _p(scale_inv), _p(d_gate_up), ld_d, _stream(stream))
    if check:
        _check(rc, "fp8_swiglu_gemm_backward")
    return rc


def fp8_mx_swiglu_gemm_backward(A, fa, lda, sA, B, fb, ldb, sB, M, F, K, gate_up=None, ld_gu=0, q=None, ld_q=0,
                                s=None, ld_s=0, ckpt_fmt=0, fmt=0, layouts=0, q_row=None, s_row=None, q_colT=None,
                                ld_colT=0, s_col=None, d_gate_up=None, ld_d=0, stream=None, check=True):
    rc = load_library().fp8_mx_swiglu_gemm_backward(_p(A), fa, lda, _p(sA), _p(B), fb, ldb, _p(sB), M, F, K,
                                                    _p(gate_up), ld_gu, _p(q), ld_q, _p(s), ld_s, ckpt_fmt, fmt,
                                                    layouts, _p(q_row), _p(s_row), _p(q_colT), ld_colT, _p(s_col),
                                                    _p(d_gate_up), ld_d, _stream(stream))
    if check:
        _check(rc, "fp8_mx_swiglu_gemm_backward")
    return rc


def fp8_sync_status(stream=None) -> int:
    return load_library().fp8_sync_status(_stream(stream))


def fp8_selftest_bounded_wait(wait_ns: int, stream=None) -> int:
    return load_library().fp8_selftest_bounded_wait(int(wait_ns), _stream(stream))


def version() -> str:
    return load_library().fp8_version().decode()


# --- convenience wrappers (allocate outputs with torch) -----------------------

@dataclass
class Quantized:
    q_row: torch.Tensor | None
    scale_inv_row: torch.Tensor | None
    q_colT: torch.Tensor | None
    scale_inv_col: torch.Tensor | None
    ld_colT: int


def quantize(x: torch.Tensor, fmt: int, recipe: Recipe, layouts: int = LAYOUT_ROW | LAYOUT_COLT, scale_in=None,
             amax_out=None, group_offsets=None, host_offsets=None, stream=None, equal_groups: int = 0) -> Quantized:
    """Quantize a CUDA bf16 [rows, cols] tensor (row stride x.stride(0)).

    Grouped (MoE) tensors pass the device offsets and their CPU copy
    (host_offsets) so the padded colwise width can be sized here; a stack of
    equal groups (expert weights) may pass equal_groups = the number of
    groups instead (rows / equal_groups a multiple of 64).
    """
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    rows, cols = x.shape
    dev = x.device
    G = 0
    if group_offsets is not None:
        G = group_offsets.numel() - 1
        ld_colT, _ = fp8_group_padded_offsets(host_offsets)
        ld_colT = max(16, (ld_colT + 15) // 16 * 16)
    else:
        G = equal_groups
        ld_colT = max(16, (rows + 15) // 16 * 16)
    q_row = sr = q_colT = sc = None
    if layouts & LAYOUT_ROW:
        q_row = torch.empty((rows, cols), dtype=torch.uint8, device=dev)
        sr = torch.empty(rows if recipe.kind == ROWWISE else 1, dtype=torch.float32, device=dev)
    if layouts & LAYOUT_COLT:
        q_colT = torch.empty((cols, ld_colT), dtype=torch.uint8, device=dev)
        nsc = (cols * (G if G else 1)) if recipe.kind == ROWWISE else 1
        sc = torch.empty(nsc, dtype=torch.float32, device=dev)
    fp8_quantize(x, rows, cols, x.stride(0), fmt, recipe, layouts, scale_in, amax_out, q_row, sr, q_colT, ld_colT,
                 sc, group_offsets, G, stream)
    return Quantized(q_row, sr, q_colT, sc, ld_colT)


def quantize_rowwise_resident(x: torch.Tensor, fmt: int, margin: int = 0, layouts: int = LAYOUT_ROW | LAYOUT_COLT,
                              amax_out=None, stream=None) -> Quantized:
    """The rowwise recipe of quantize() for a plain CUDA bf16 [rows, cols]
    tensor in one cooperative launch (same results; fewer launches, and the
    second read of x comes from L2)."""
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    rows, cols = x.shape
    dev = x.device
    ld_colT = max(16, (rows + 15) // 16 * 16)
    q_row = sr = q_colT = sc = None
    if layouts & LAYOUT_ROW:
        q_row = torch.empty((rows, cols), dtype=torch.uint8, device=dev)
        sr = torch.empty(max(rows, 1), dtype=torch.float32, device=dev)
    if layouts & LAYOUT_COLT:
        q_colT = torch.empty((cols, ld_colT), dtype=torch.uint8, device=dev)
        sc = torch.empty(cols, dtype=torch.float32, device=dev)
    fp8_quantize_rowwise_resident(x, rows, cols, x.stride(0), fmt, margin, layouts, amax_out, q_row, sr, q_colT,
                                  ld_colT, sc, stream)
    return Quantized(q_row, sr, q_colT, sc, ld_colT)


def _rowwise_outputs(rows, cols, dev, layouts, host_offsets):
    G = len(host_offsets) - 1
    ld_colT, _ = fp8_group_padded_offsets(host_offsets)
    ld_colT = max(16, (ld_colT + 15) // 16 * 16)
    q_row = sr = q_colT = sc = None
    if layouts & LAYOUT_ROW:
        q_row = torch.empty((rows, cols), dtype=torch.uint8, device=dev)
        sr = torch.empty(max(rows, 1), dtype=torch.float32, device=dev)
    if layouts & LAYOUT_COLT:
        q_colT = torch.empty((cols, ld_colT), dtype=torch.uint8, device=dev)
        sc = torch.empty(cols * G, dtype=torch.float32, device=dev)
    return Quantized(q_row, sr, q_colT, sc, ld_colT)


def permute_quantize(x: torch.Tensor, src_rows: torch.Tensor, fmt: int, group_offsets, host_offsets,
                     layouts: int = LAYOUT_ROW | LAYOUT_COLT, margin: int = 0, amax_out=None,
                     stream=None) -> Quantized:
    """Gather x[src_rows] (routed token rows in expert order) and quantize it
    with the rowwise recipe, per-expert column scales, in one pass."""
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1 and src_rows.dtype == torch.int32
    rows, cols = src_rows.numel(), x.shape[1]
    q = _rowwise_outputs(rows, cols, x.device, layouts, host_offsets)
    fp8_permute_quantize(x, x.shape[0], cols, x.stride(0), src_rows, rows, fmt, margin, layouts, amax_out, q.q_row,
                         q.scale_inv_row, q.q_colT, q.ld_colT, q.scale_inv_col, group_offsets,
                         group_offsets.numel() - 1, stream)
    return q


def swiglu_quantize(gate_up: torch.Tensor, fmt: int, group_offsets, host_offsets,
                    layouts: int = LAYOUT_ROW | LAYOUT_COLT, h_out=None, margin: int = 0, amax_out=None,
                    stream=None) -> Quantized:
    """h = bf16(silu(gate) * up) of a [rows, 2F] gate|up tensor, quantized
    with the rowwise recipe, per-expert column scales, in one pass (h also
    written to h_out when given)."""
    assert gate_up.dtype == torch.bfloat16 and gate_up.dim() == 2 and gate_up.stride(1) == 1
    rows, F = gate_up.shape[0], gate_up.shape[1] // 2
    q = _rowwise_outputs(rows, F, gate_up.device, layouts, host_offsets)
    fp8_swiglu_quantize(gate_up, rows, F, gate_up.stride(0), fmt, margin, layouts, h_out,
                        h_out.stride(0) if h_out is not None else 0, amax_out, q.q_row, q.scale_inv_row, q.q_colT,
                        q.ld_colT, q.scale_inv_col, group_offsets, group_offsets.numel() - 1, stream)
    return q


def scaled_gemm(A: torch.Tensor, fa: int, B: torch.Tensor, fb: int, sa: torch.Tensor, sb: torch.Tensor, K=None,
                out=None, stream=None) -> torch.Tensor:
    """C = bf16(A[:, :K] . B[:, :K]^T * sa * sb); sa/sb of size 1 are per-tensor."""
    M, lda = A.shape
    N, ldb = B.shape
    K = lda if K is None else K
    C = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16, device=A.device)
    fp8_scaled_gemm(A, fa, A.stride(0), B, fb, B.stride(0), M, N, K, sa, int(sa.numel() > 1), sb,
                    int(sb.numel() > 1), C, C.stride(0), stream)
    return C


def grouped_gemm(mode: int, A, fa, B, fb, group_offsets, M_total, N, K, sa, sb, ld_T=0, out=None, stream=None):
    G = group_offsets.numel() - 1
    if out is None:
        shape = (G, N, K) if mode == GROUPED_K else (M_total, N)
        out = torch.empty(shape, dtype=torch.bfloat16, device=A.device)
    fp8_grouped_gemm(mode, A, fa, B, fb, group_offsets, G, M_total, N, K, sa, int(sa.numel() > 1), sb,
                     int(sb.numel() > 1), out, ld_T, stream)
    return out


@dataclass
class MxQuantized:
    q_row: torch.Tensor | None     # [rows, cols] u8
    s_row: torch.Tensor | None     # MX scale layout, R = rows (grouped: padded total)
    q_colT: torch.Tensor | None    # [cols, ld_colT] u8
    s_col: torch.Tensor | None     # MX scale layout, R = cols, KB = ld_colT / 32
    ld_colT: int
    scale_rows: int                # R of s_row


def mx_quantize(x: torch.Tensor, fmt: int, layouts: int = LAYOUT_ROW | LAYOUT_COLT, group_offsets=None,
                host_offsets=None, stream=None) -> MxQuantized:
    """MX quantize of a CUDA bf16 [rows, cols] tensor (cols % 32 == 0).

    Grouped (MoE) tensors pass the device offsets and their CPU copy; every
    group is padded to MX_GROUP_ALIGN rows in the padded layouts.
    """
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    rows, cols = x.shape
    dev = x.device
    G = 0
    if group_offsets is not None:
        G = group_offsets.numel() - 1
        P, _ = fp8_group_padded_offsets(host_offsets, MX_GROUP_ALIGN)
    else:
        P = rows
    ld_colT = max(16, (P + 15) // 16 * 16)
    def buf(n):  # never a zero-byte (null) allocation
        return torch.empty(max(16, n), dtype=torch.uint8, device=dev)

    q_row = s_row = q_colT = s_col = None
    if layouts & LAYOUT_ROW:
        q_row = buf(rows * cols)[:rows * cols].view(rows, cols)
        s_row = buf(fp8_mx_scale_bytes(P, cols // MX_BLOCK))
    if layouts & LAYOUT_COLT:
        q_colT = buf(cols * ld_colT)[:cols * ld_colT].view(cols, ld_colT)
        s_col = buf(fp8_mx_scale_bytes(cols, P // MX_BLOCK))
    fp8_mx_quantize(x, rows, cols, x.stride(0), fmt, layouts, q_row, s_row, q_colT, ld_colT, s_col, group_offsets,
                    G, stream)
    return MxQuantized(q_row, s_row, q_colT, s_col, ld_colT, P)


def _mx_outputs(rows, cols, dev, layouts, host_offsets):
    P = fp8_group_padded_offsets(host_offsets, MX_GROUP_ALIGN)[0] if host_offsets is not None else rows
    ld_colT = max(16, (P + 15) // 16 * 16)

    def buf(n):  # never a zero-byte (null) allocation
        return torch.empty(max(16, n), dtype=torch.uint8, device=dev)

    q_row = s_row = q_colT = s_col = None
    if layouts & LAYOUT_ROW:
        q_row = buf(rows * cols)[:rows * cols].view(rows, cols)
        s_row = buf(fp8_mx_scale_bytes(P, cols // MX_BLOCK))
    if layouts & LAYOUT_COLT:
        q_colT = buf(cols * ld_colT)[:cols * ld_colT].view(cols, ld_colT)
        s_col = buf(fp8_mx_scale_bytes(cols, P // MX_BLOCK))
    return MxQuantized(q_row, s_row, q_colT, s_col, ld_colT, P)


def mx_permute_quantize(x: torch.Tensor, src_rows: torch.Tensor, fmt: int, layouts: int = LAYOUT_ROW | LAYOUT_COLT,
                        group_offsets=None, host_offsets=None, stream=None) -> MxQuantized:
    """Gather x[src_rows] (routed token rows in expert order) and MX-quantize
    them in one pass."""
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1 and src_rows.dtype == torch.int32
    rows, cols = src_rows.numel(), x.shape[1]
    q = _mx_outputs(rows, cols, x.device, layouts, host_offsets)
    G = 0 if group_offsets is None else group_offsets.numel() - 1
    fp8_mx_permute_quantize(x, x.shape[0], cols, x.stride(0), src_rows, rows, fmt, layouts, q.q_row, q.s_row,
                            q.q_colT, q.ld_colT, q.s_col, group_offsets, G, stream)
    return q


def mx_swiglu_quantize(gate_up: torch.Tensor, fmt: int, layouts: int = LAYOUT_ROW | LAYOUT_COLT, h_out=None,
                       group_offsets=None, host_offsets=None, stream=None) -> MxQuantized:
    """h = bf16(silu(gate) * up) of a [rows, 2F] gate|up tensor, MX-quantized
    in one pass (h also written to h_out when given)."""
    assert gate_up.dtype == torch.bfloat16 and gate_up.dim() == 2 and gate_up.stride(1) == 1
    rows, F = gate_up.shape[0], gate_up.shape[1] // 2
    q = _mx_outputs(rows, F, gate_up.device, layouts, host_offsets)
    G = 0 if group_offsets is None else group_offsets.numel() - 1
    fp8_mx_swiglu_quantize(gate_up, rows, F, gate_up.stride(0), fmt, layouts, h_out,
                           h_out.stride(0) if h_out is not None else 0, q.q_row, q.s_row, q.q_colT, q.ld_colT,
                           q.s_col, group_offsets, G, stream)
    return q


def mx_gemm(A: torch.Tensor, fa: int, sA: torch.Tensor, B: torch.Tensor, fb: int, sB: torch.Tensor, K=None,
            out=None, stream=None) -> torch.Tensor:
    """C = bf16(MX-scaled A[:, :K] . B[:, :K]^T)."""
    M, lda = A.shape
    N, ldb = B.shape
    K = lda if K is None else K
    C = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16, device=A.device)
    fp8_mx_gemm(A, fa, A.stride(0), sA, B, fb, B.stride(0), sB, M, N, K, C, C.stride(0), stream)
    return C


def mx_grouped_gemm(mode: int, A, fa, sA, B, fb, sB, group_offsets, M_total, N, K, ld_T=0, out=None, stream=None):
    G = group_offsets.numel() - 1
    if out is None:
        shape = (G, N, K) if mode == GROUPED_K else (M_total, N)
        out = torch.empty(shape, dtype=torch.bfloat16, device=A.device)
    fp8_mx_grouped_gemm(mode, A, fa, sA, B, fb, sB, group_offsets, G, M_total, N, K, out, ld_T, stream)
    return out


def blockwise_quantize(x: torch.Tensor, fmt: int, block_rows: int, layouts: int = LAYOUT_ROW | LAYOUT_COLT,
                       stream=None) -> MxQuantized:
    """Blockwise quantize of a CUDA bf16 [rows, cols] tensor: block_rows 1 for
    activations / gradients (1 x 128 blocks), 128 for weights (128 x 128).
    The scales are in the MX scale layout, ready for mx_gemm."""
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    rows, cols = x.shape
    q = _mx_outputs(rows, cols, x.device, layouts, None)
    fp8_blockwise_quantize(x, rows, cols, x.stride(0), fmt, block_rows, layouts, q.q_row, q.s_row, q.q_colT,
                           q.ld_colT, q.s_col, stream)
    return q


# --- norms, SwiGLU backward and 8-bit checkpoints -------------------------------
# These call the library directly with addresses, not through the mirrors of the
# entry points above: for a few tokens the host's time is what a call costs, and
# the extra layer is a fifth of it.  A call runs on the current device (that of
# `stream`, where one is given as a torch stream), and its tensors lie there.

def _ptr(t):
    return None if t is None else t.data_ptr()


def _refuse(where: str, detail: str):
    raise Fp8Error(1, where, detail)


def _on(stream):
    """Context that makes `stream` current: torch then allocates for it, and
    what is dropped at return (a workspace) is reused in that stream's order."""
    if not isinstance(stream, torch.cuda.Stream):
        handle = int(stream)
        # ExternalStream takes 0, the default stream's handle, as none given and makes a stream of its own
        stream = torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def _elsewhere(t: torch.Tensor, where: str, name: str):
    """A tensor of another device than the current one, on which the call
    launches: a kernel cannot count on reaching its memory."""
    _refuse(where, f"{name} is on cuda:{t.get_device()}, the current device is {torch._C._cuda_getDevice()}")


def _matrix(t: torch.Tensor, where: str, name: str, rows=None, cols=None, dtype=None) -> int:
    """Check a CUDA matrix; returns its row stride."""
    if not t.is_cuda or t.dim() != 2:
        _refuse(where, f"{name} must be a CUDA matrix")
    if t.get_device() != torch._C._cuda_getDevice():
        _elsewhere(t, where, name)
    if t.dtype not in DTYPES if dtype is None else t.dtype != dtype:
        _refuse(where, f"{name} has type {t.dtype}")
    n, c = t.shape
    if (rows is not None and n != rows) or (cols is not None and c != cols):
        _refuse(where, f"{name} is {n} x {c}, not {rows} x {cols}")
    ld, col = t.stride()
    if c == 0 or (col != 1 and c > 1):
        _refuse(where, f"{name} must have consecutive columns")
    return ld if n > 1 else max(c, ld)


def _vector(t, where: str, name: str, n: int, dtype=None):
    if not t.is_cuda or t.dim() != 1 or t.numel() != n or not t.is_contiguous():
        _refuse(where, f"{name} must be a contiguous CUDA vector of {n} elements")
    if t.get_device() != torch._C._cuda_getDevice():
        _elsewhere(t, where, name)
    if t.dtype not in DTYPES if dtype is None else t.dtype != dtype:
        _refuse(where, f"{name} has type {t.dtype}")


@dataclass
class Checkpoint:
    """An activation of `parts` side-by-side tensors of `cols` columns each,
    kept in 8 bits (format in include/fp8gb.h): q u8 [rows, parts * W], W =
    cols rounded up to 32, and one scale byte per 32 columns in s u8
    [rows, parts * W / 32]."""
    q: torch.Tensor
    s: torch.Tensor
    fmt: int
    cols: int
    parts: int = 1

    @property
    def rows(self) -> int:
        return self.q.shape[0]


def _blocks(cols: int) -> int:
    return (cols + MX_BLOCK - 1) // MX_BLOCK


def _new_checkpoint(rows, cols, parts, dev, fmt) -> Checkpoint:
    nb = _blocks(cols) * parts
    return Checkpoint(torch.empty((rows, nb * MX_BLOCK), dtype=torch.uint8, device=dev),
                      torch.empty((rows, nb), dtype=torch.uint8, device=dev), fmt, cols, parts)


def _checkpoint_strides(c: Checkpoint, where: str, rows=None, cols=None, parts=None):
    n = c.q.shape[0]
    if (rows is not None and n != rows) or (cols is not None and c.cols != cols) or \
            (parts is not None and c.parts != parts):
        _refuse(where, f"the checkpoint holds {n} x {c.parts} x {c.cols}, not {rows} x {parts} x {cols}")
    nb = _blocks(c.cols) * c.parts
    return (_matrix(c.q, where, "checkpoint codes", n, nb * MX_BLOCK, torch.uint8),
            _matrix(c.s, where, "checkpoint scales", n, nb, torch.uint8))


def checkpoint(x: torch.Tensor, fmt: int = E4M3FN, parts: int = 1, stream=None) -> Checkpoint:
    """Keep a [rows, parts * cols] bf16 / fp16 / fp32 activation in 8 bits."""
    if stream is not None:
        with _on(stream):
            return checkpoint(x, fmt, parts)
    where = "checkpoint"
    ld = _matrix(x, where, "x")
    rows, total = x.shape
    if parts < 1 or total % parts:
        _refuse(where, f"{total} columns are not {parts} equal parts")
    c = _new_checkpoint(rows, total // parts, parts, x.device, fmt)
    nb = _blocks(c.cols) * parts
    _check(load_library().fp8_checkpoint(x.data_ptr(), DTYPES[x.dtype], rows, c.cols, ld, parts, fmt, c.q.data_ptr(),
                                         nb * MX_BLOCK, c.s.data_ptr(), nb, _stream(None)), where)
    return c


def checkpoint_restore(c: Checkpoint, dtype: torch.dtype = torch.bfloat16, out=None, stream=None) -> torch.Tensor:
    """The [rows, parts * cols] activation a checkpoint stands for."""
    if stream is not None:
        with _on(stream):
            return checkpoint_restore(c, dtype, out)
    where = "checkpoint_restore"
    ld_q, ld_s = _checkpoint_strides(c, where)
    rows = c.q.shape[0]
    if out is None:
        if dtype not in DTYPES:
            _refuse(where, f"cannot restore to {dtype}")
        out, ld = torch.empty((rows, c.parts * c.cols), dtype=dtype, device=c.q.device), c.parts * c.cols
    else:
        ld = _matrix(out, where, "out", rows, c.parts * c.cols)
    _check(load_library().fp8_checkpoint_restore(c.q.data_ptr(), ld_q, c.s.data_ptr(), ld_s, c.fmt, rows, c.cols,
                                                 c.parts, out.data_ptr(), DTYPES[out.dtype], ld, _stream(None)), where)
    return out


def swiglu_checkpoint(gate_up: torch.Tensor, fmt: int = E4M3FN, h_out=None, stream=None):
    """h = bf16(silu(gate) * up) of a bf16 [rows, 2F] gate|up tensor, and its
    2-part 8-bit checkpoint, from one read.  Returns (h, checkpoint)."""
    if stream is not None:
        with _on(stream):
            return swiglu_checkpoint(gate_up, fmt, h_out)
    where = "swiglu_checkpoint"
    ld = _matrix(gate_up, where, "gate_up", dtype=torch.bfloat16)
    rows, total = gate_up.shape
    if total % 2:
        _refuse(where, "gate_up must have an even number of columns")
    F = total // 2
    if h_out is None:
        h, ld_h = torch.empty((rows, F), dtype=torch.bfloat16, device=gate_up.device), F
    else:
        h, ld_h = h_out, _matrix(h_out, where, "h_out", rows, F, torch.bfloat16)
    c = _new_checkpoint(rows, F, 2, gate_up.device, fmt)
    nb = 2 * _blocks(F)
    _check(load_library().fp8_swiglu_checkpoint(gate_up.data_ptr(), rows, F, ld, fmt, h.data_ptr(), ld_h,
                                                c.q.data_ptr(), nb * MX_BLOCK, c.s.data_ptr(), nb, _stream(None)),
           where)
    return h, c


def swiglu_backward(dh: torch.Tensor, src, out=None, return_h: bool = False, stream=None):
    """Gradient of gate|up from dh (bf16 [rows, F]) and src: the bf16
    [rows, 2F] gate|up tensor or its checkpoint.  With return_h also
    h = bf16(silu(gate) * up) of what src holds: (d_gate_up, h)."""
    if stream is not None:
        with _on(stream):
            return swiglu_backward(dh, src, out, return_h)
    where = "swiglu_backward"
    ld_dh = _matrix(dh, where, "dh", dtype=torch.bfloat16)
    rows, F = dh.shape
    gate_up = q = s = h = None
    ld = ld_q = ld_s = fmt = 0
    if isinstance(src, Checkpoint):
        ld_q, ld_s = _checkpoint_strides(src, where, rows, F, 2)
        q, s, fmt = src.q, src.s, src.fmt
    else:
        gate_up, ld = src, _matrix(src, where, "gate_up", rows, 2 * F, torch.bfloat16)
    if out is None:
        out, ld_d = torch.empty((rows, 2 * F), dtype=torch.bfloat16, device=dh.device), 2 * F
    else:
        ld_d = _matrix(out, where, "out", rows, 2 * F, torch.bfloat16)
    if return_h:
        h = torch.empty((rows, F), dtype=torch.bfloat16, device=dh.device)
    _check(load_library().fp8_swiglu_backward(dh.data_ptr(), ld_dh, _ptr(gate_up), ld, _ptr(q), ld_q, _ptr(s), ld_s,
                                              fmt, rows, F, out.data_ptr(), ld_d, _ptr(h), F, _stream(None)), where)
    return (out, h) if return_h else out


@dataclass
class NormForward:
    y: torch.Tensor
    mean: torch.Tensor | None        # fp32 [rows]; None for RMS_NORM
    rstd: torch.Tensor               # fp32 [rows]
    checkpoint: Checkpoint | None    # of the normalized rows


@dataclass
class NormBackward:
    dx: torch.Tensor
    dweight: torch.Tensor | None
    dbias: torch.Tensor | None


def norm_forward(x: torch.Tensor, weight=None, bias=None, kind: int = LAYER_NORM, eps: float = 1e-5, out_dtype=None,
                 checkpoint_fmt=None, out=None, stream=None) -> NormForward:
    """Layer or RMS norm of the rows of x (bf16 / fp16 / fp32 [rows, cols]),
    y = xhat * weight + bias, in x's type or, for an fp32 x, out_dtype.  With
    checkpoint_fmt (E4M3FN or E5M2) xhat is kept in 8 bits for norm_backward,
    which then needs neither x nor the mean."""
    if stream is not None:
        with _on(stream):
            return norm_forward(x, weight, bias, kind, eps, out_dtype, checkpoint_fmt, out)
    where = "norm_forward"
    ld = _matrix(x, where, "x")
    rows, cols = x.shape
    dev = x.device
    w_dtype = 0
    if weight is not None:
        _vector(weight, where, "weight", cols)
        w_dtype = DTYPES[weight.dtype]
    if bias is not None:
        _vector(bias, where, "bias", cols, None if weight is None else weight.dtype)
        w_dtype = DTYPES[bias.dtype]
    if out is None:
        out_dtype = out_dtype or x.dtype
        if out_dtype not in DTYPES:
            _refuse(where, f"cannot write {out_dtype}")
        out, ld_y = torch.empty((rows, cols), dtype=out_dtype, device=dev), cols
    else:
        ld_y = _matrix(out, where, "out", rows, cols)
        out_dtype = out.dtype
    mean = torch.empty(rows, dtype=torch.float32, device=dev) if kind == LAYER_NORM else None
    rstd = torch.empty(rows, dtype=torch.float32, device=dev)
    c = q = s = None
    nb = fmt = 0
    if checkpoint_fmt is not None:
        c = _new_checkpoint(rows, cols, 1, dev, checkpoint_fmt)
        q, s, fmt, nb = c.q, c.s, checkpoint_fmt, _blocks(cols)
    _check(load_library().fp8_norm_forward(x.data_ptr(), DTYPES[x.dtype], ld, rows, cols, kind, eps, _ptr(weight),
                                           _ptr(bias), w_dtype, out.data_ptr(), DTYPES[out_dtype], ld_y, _ptr(mean),
                                           rstd.data_ptr(), fmt, _ptr(q), nb * MX_BLOCK, _ptr(s), nb, _stream(None)),
           where)
    return NormForward(out, mean, rstd, c)


def norm_backward(dy: torch.Tensor, src, mean, rstd: torch.Tensor, weight=None, kind: int = LAYER_NORM, dx_dtype=None,
                  weight_grad: bool = True, bias_grad=None, out=None, stream=None, dsum=None) -> NormBackward:
    """Backward of norm_forward and the norm of norm_quantize from src: the forward's x, or the checkpoint
    it made (mean is then not read and may be None).  dweight and dbias have
    the weight's type (fp32 without a weight); bias_grad defaults to whether
    the norm is a layer norm.  dx has x's type; from a checkpoint, dx_dtype,
    by default dy's type.  dsum (of dx's type) is the gradient that reaches x
    past the norm and is added to dx before its rounding."""
    if stream is not None:
        with _on(stream):
            return norm_backward(dy, src, mean, rstd, weight, kind, dx_dtype, weight_grad, bias_grad, out, dsum=dsum)
    where = "norm_backward"
    ld_dy = _matrix(dy, where, "dy")
    rows, cols = dy.shape
    dev = dy.device
    _vector(rstd, where, "rstd", rows, torch.float32)
    if mean is not None:
        _vector(mean, where, "mean", rows, torch.float32)
    w_dtype = torch.float32
    if weight is not None:
        _vector(weight, where, "weight", cols)
        w_dtype = weight.dtype
    x = q = s = None
    ld_x = ld_q = ld_s = fmt = 0
    if isinstance(src, Checkpoint):
        ld_q, ld_s = _checkpoint_strides(src, where, rows, cols, 1)
        q, s, fmt = src.q, src.s, src.fmt
        dx_dtype = dx_dtype or (dy.dtype if out is None else out.dtype)
        if dx_dtype not in DTYPES:
            _refuse(where, f"cannot write {dx_dtype}")
    else:
        x, ld_x = src, _matrix(src, where, "x", rows, cols)
        if dx_dtype is not None and dx_dtype != x.dtype:
            _refuse(where, f"dx of a {x.dtype} x cannot be {dx_dtype}")
        if kind == LAYER_NORM and mean is None:
            _refuse(where, "a layer norm's backward from x needs its mean")
        dx_dtype = x.dtype
    ld_dsum = 0 if dsum is None else _matrix(dsum, where, "dsum", rows, cols, dx_dtype)
    if out is None:
        out, ld_dx = torch.empty((rows, cols), dtype=dx_dtype, device=dev), cols
    else:
        ld_dx = _matrix(out, where, "out", rows, cols, dx_dtype)
    dw = torch.empty(cols, dtype=w_dtype, device=dev) if weight_grad else None
    db = torch.empty(cols, dtype=w_dtype, device=dev) \
        if (kind == LAYER_NORM if bias_grad is None else bias_grad) else None
    ws, n = None, 0
    if dw is not None or db is not None:
        n = load_library().fp8_norm_workspace_bytes(rows, cols)
        if n > 0:  # -1: a shape that the call refuses
            ws = torch.empty(n, dtype=torch.uint8, device=dev)
    if dsum is None:
        _check(load_library().fp8_norm_backward(dy.data_ptr(), DTYPES[dy.dtype], ld_dy, _ptr(x), ld_x, _ptr(q), ld_q,
                                                _ptr(s), ld_s, fmt, rows, cols, kind, _ptr(mean), rstd.data_ptr(),
                                                _ptr(weight), DTYPES[w_dtype], out.data_ptr(), DTYPES[dx_dtype],
                                                ld_dx, _ptr(dw), _ptr(db), _ptr(ws), n, _stream(None)), where)
    else:
        _check(load_library().fp8_residual_norm_backward(
            dy.data_ptr(), DTYPES[dy.dtype], ld_dy, _ptr(x), ld_x, _ptr(q), ld_q, _ptr(s), ld_s, fmt, dsum.data_ptr(),
            ld_dsum, rows, cols, kind, _ptr(mean), rstd.data_ptr(), _ptr(weight), DTYPES[w_dtype], out.data_ptr(),
            DTYPES[dx_dtype], ld_dx, _ptr(dw), _ptr(db), _ptr(ws), n, _stream(None)), where)
    return NormBackward(out, dw, db)


# --- joined with the quantizes and products around them -------------------------

@dataclass
class NormQuantize:
    q: Quantized | MxQuantized       # the norm's result in 8 bits
    sum: torch.Tensor                # x + residual as stored (x without a residual): norm_backward's src
    mean: torch.Tensor | None        # fp32 [rows]; None for RMS_NORM
    rstd: torch.Tensor               # fp32 [rows]


def _u8(rows, cols, dev):
    """u8 [rows, cols], never a zero-byte (null) allocation."""
    if rows:
        return torch.empty((rows, cols), dtype=torch.uint8, device=dev)
    return torch.empty(16, dtype=torch.uint8, device=dev)[:0].view(0, cols)


def _mx_scale_buffer(rows, blocks, dev):
    """Buffer of fp8_mx_scale_bytes(rows, blocks) bytes (computed here: a call into the library costs microseconds)."""
    n = (blocks + 3) // 4 * 4 * ((rows + 127) // 128 * 128)
    return torch.empty(n or 16, dtype=torch.uint8, device=dev)


def _stored_inverse(rows, dev, scale_in):
    """Where the call leaves 1 / scale_in; with no rows it writes nothing, and the value is put here."""
    return torch.empty(1, dtype=torch.float32, device=dev) if rows else scale_in.reciprocal()


def _scaled_outputs(rows, cols, dev, layouts, scale_in, per_row) -> Quantized:
    ld_colT = max(16, (rows + 15) // 16 * 16)
    q = Quantized(None, None, None, None, ld_colT)
    scale = torch.empty(rows, dtype=torch.float32, device=dev) if per_row else _stored_inverse(rows, dev, scale_in)
    if layouts & LAYOUT_ROW:
        q.q_row, q.scale_inv_row = _u8(rows, cols, dev), scale
    if layouts & LAYOUT_COLT:
        q.q_colT, q.scale_inv_col = _u8(cols, ld_colT, dev), scale
    return q


def _mx_split_outputs(rows, row_cols, col_rows, dev, layouts) -> MxQuantized:
    """MX outputs whose row layout may be wider than the transposed one is tall."""
    ld_colT = max(16, (rows + 15) // 16 * 16)
    q = MxQuantized(None, None, None, None, ld_colT, rows)
    if layouts & LAYOUT_ROW:
        q.q_row = _u8(rows, row_cols, dev)
        q.s_row = _mx_scale_buffer(rows, row_cols // MX_BLOCK, dev)
    if layouts & LAYOUT_COLT:
        q.q_colT = _u8(col_rows, ld_colT, dev)
        q.s_col = _mx_scale_buffer(col_rows, rows // MX_BLOCK, dev)
    return q


def _norm_inputs(x, residual, weight, bias, kind, out, where):
    """Checks of norm_quantize and mx_norm_quantize: what the C call wants of
    them, and the tensors it writes besides the 8 bits."""
    ld_x = _matrix(x, where, "x")
    rows, cols = x.shape
    dev = x.device
    w_dtype = 0
    if weight is not None:
        _vector(weight, where, "weight", cols)
        w_dtype = DTYPES[weight.dtype]
    if bias is not None:
        _vector(bias, where, "bias", cols, None if weight is None else weight.dtype)
        w_dtype = DTYPES[bias.dtype]
    ld_r = ld_sum = r_dtype = 0
    if residual is not None:
        ld_r = _matrix(residual, where, "residual", rows, cols)
        r_dtype = DTYPES[residual.dtype]
        if out is None:
            out, ld_sum = torch.empty((rows, cols), dtype=residual.dtype, device=dev), cols
        else:
            ld_sum = _matrix(out, where, "out", rows, cols, residual.dtype)
    elif out is not None:
        _refuse(where, "out receives x + residual: there is no residual")
    mean = torch.empty(rows, dtype=torch.float32, device=dev) if kind == LAYER_NORM else None
    rstd = torch.empty(rows, dtype=torch.float32, device=dev)
    front = (x.data_ptr(), DTYPES[x.dtype], ld_x, _ptr(residual), r_dtype, ld_r, rows, cols)
    params = (_ptr(weight), _ptr(bias), w_dtype, _ptr(out), ld_sum, _ptr(mean), rstd.data_ptr())
    return front, params, out, mean, rstd


def norm_quantize(x: torch.Tensor, residual=None, weight=None, bias=None, kind: int = LAYER_NORM, eps: float = 1e-5,
                  fmt: int = E4M3FN, recipe: Recipe | None = None, layouts: int = LAYOUT_ROW, scale_in=None,
                  amax_out=None, out=None, stream=None) -> NormQuantize:
    """sum = x + residual (stored, in the residual's type: x's or fp32), its layer
    or RMS norm, and that in 8 bits, in one read.  out receives the sum, not in
    place of an input.  recipe: ROWWISE (the default; one scale per row, row layout)
    or DELAYED (scale_in, amax_out; either layout)."""
    if stream is not None:
        with _on(stream):
            return norm_quantize(x, residual, weight, bias, kind, eps, fmt, recipe, layouts, scale_in, amax_out, out)
    where = "norm_quantize"
    recipe = recipe or Recipe(kind=ROWWISE)
    _delayed_scales(fmt if recipe.kind == DELAYED else None, scale_in, amax_out, where)
    front, params, total, mean, rstd = _norm_inputs(x, residual, weight, bias, kind, out, where)
    rows, cols = x.shape
    q = _scaled_outputs(rows, cols, x.device, layouts, scale_in, recipe.kind != DELAYED)
    _check(load_library().fp8_norm_quantize(*front, kind, eps, *params, fmt, ctypes.byref(recipe.c()), layouts,
                                            _ptr(scale_in), _ptr(amax_out), _ptr(q.q_row), _ptr(q.scale_inv_row),
                                            _ptr(q.q_colT), q.ld_colT, _ptr(q.scale_inv_col), _stream(None)), where)
    return NormQuantize(q, x if residual is None else total, mean, rstd)


def mx_norm_quantize(x: torch.Tensor, residual=None, weight=None, bias=None, kind: int = LAYER_NORM,
                     eps: float = 1e-5, fmt: int = E4M3FN, layouts: int = LAYOUT_ROW | LAYOUT_COLT, out=None,
                     stream=None) -> NormQuantize:
    """norm_quantize with MX block scales (mx_quantize's layouts and limits)."""
    if stream is not None:
        with _on(stream):
            return mx_norm_quantize(x, residual, weight, bias, kind, eps, fmt, layouts, out)
    where = "mx_norm_quantize"
    front, params, total, mean, rstd = _norm_inputs(x, residual, weight, bias, kind, out, where)
    rows, cols = x.shape
    q = _mx_split_outputs(rows, cols, cols, x.device, layouts)
    _check(load_library().fp8_mx_norm_quantize(*front, kind, eps, *params, fmt, layouts, _ptr(q.q_row), _ptr(q.s_row),
                                               _ptr(q.q_colT), q.ld_colT, _ptr(q.s_col), _stream(None)), where)
    return NormQuantize(q, x if residual is None else total, mean, rstd)


@dataclass
class SwigluGemm:
    q: Quantized | MxQuantized | None  # h in 8 bits
    h: torch.Tensor | None             # bf16 [M, F]
    gate_up: torch.Tensor | None       # bf16 [M, 2F]
    checkpoint: Checkpoint | None      # of gate|up


@dataclass
class SwigluGemmBackward:
    q: Quantized | MxQuantized | None  # d_gate | d_up in 8 bits
    d_gate_up: torch.Tensor | None     # bf16 [M, 2F]


def _codes(t: torch.Tensor, where: str, name: str, K: int) -> int:
    """Check an FP8 operand of at least K columns; returns its row stride."""
    ld = _matrix(t, where, name, dtype=torch.uint8)
    if t.shape[1] < K:
        _refuse(where, f"{name} has {t.shape[1]} columns, not {K}")
    return ld if ld % 16 == 0 or t.shape[0] > 1 else (ld + 15) // 16 * 16


def _scale(t: torch.Tensor, where: str, name: str, n: int) -> int:
    """Check an operand's scales: one, or one for each of its n rows (none for no rows)."""
    _vector(t, where, name, 1 if t.numel() == 1 else n, torch.float32)
    return SCALE_TENSOR if t.numel() == 1 else SCALE_PER_ROW


def _mx_scales(t: torch.Tensor, where: str, name: str, rows: int, K: int):
    """MX scales must be as many as the operand's products read."""
    _vector(t, where, name, t.numel(), torch.uint8)
    need = (K + 127) // 128 * 4 * ((rows + 127) // 128 * 128)
    if t.numel() < need:
        _refuse(where, f"{name} holds {t.numel()} bytes, {need} are needed")


def _groups_of(F: int) -> int:
    """Rows of a half in the MX layouts of gate|up: padded to whole groups."""
    return (F + MX_GROUP_ALIGN - 1) // MX_GROUP_ALIGN * MX_GROUP_ALIGN


def _kept(src, M, F, where):
    """gate|up for the backward as the C call takes it."""
    if isinstance(src, Checkpoint):
        ld_q, ld_s = _checkpoint_strides(src, where, M, F, 2)
        return None, 0, src.q.data_ptr(), ld_q, src.s.data_ptr(), ld_s, src.fmt
    ld = _matrix(src, where, "gate_up", M, 2 * F, torch.bfloat16)
    return src.data_ptr(), ld, None, 0, None, 0, 0


def _swiglu_gemm_outputs(M, F, dev, h, gate_up, checkpoint_fmt):
    h = torch.empty((M, F), dtype=torch.bfloat16, device=dev) if h else None
    gate_up = torch.empty((M, 2 * F), dtype=torch.bfloat16, device=dev) if gate_up else None
    c = None if checkpoint_fmt is None else _new_checkpoint(M, F, 2, dev, checkpoint_fmt)
    nb = 2 * _blocks(F)
    return h, gate_up, c, (_ptr(h), F, _ptr(gate_up), 2 * F, checkpoint_fmt or 0, _ptr(c and c.q), nb * MX_BLOCK,
                           _ptr(c and c.s), nb)


def swiglu_gemm(A: torch.Tensor, fa: int, W: torch.Tensor, fw: int, sa: torch.Tensor, sw: torch.Tensor, K=None,
                fmt=None, layouts: int = LAYOUT_ROW | LAYOUT_COLT, scale_in=None, amax_out=None, h: bool = False,
                gate_up: bool = False, checkpoint_fmt=None, stream=None) -> SwigluGemm:
    """h = silu(gate) * up with gate | up = A[:, :K] . W[:, :K]^T, W u8 [2F, K]
    the gate's rows, then the up's; sa / sw of size 1 are per-tensor, else per
    row.  Leaves what is asked for: h in 8 bits (fmt given: the delayed recipe,
    scale_in and amax_out), h in bf16, gate|up in bf16 or as a checkpoint."""
    if stream is not None:
        with _on(stream):
            return swiglu_gemm(A, fa, W, fw, sa, sw, K, fmt, layouts, scale_in, amax_out, h, gate_up, checkpoint_fmt)
    where = "swiglu_gemm"
    M, K = A.shape[0], A.shape[1] if K is None else K
    lda, ldw = _codes(A, where, "A", K), _codes(W, where, "W", K)
    if W.shape[0] % 2:
        _refuse(where, "W must have an even number of rows")
    F, dev = W.shape[0] // 2, A.device
    modes = _scale(sa, where, "sa", M), _scale(sw, where, "sw", 2 * F)
    _delayed_scales(fmt, scale_in, amax_out, where)
    q, quant = _delayed_outputs(M, F, F, dev, fmt, layouts, scale_in, amax_out)
    h, gate_up, c, rest = _swiglu_gemm_outputs(M, F, dev, h, gate_up, checkpoint_fmt)
    _check(load_library().fp8_swiglu_gemm(A.data_ptr(), fa, lda, W.data_ptr(), fw, ldw, M, F, K, sa.data_ptr(),
                                          modes[0], sw.data_ptr(), modes[1], *quant, *rest, _stream(None)), where)
    return SwigluGemm(q, h, gate_up, c)


def _delayed_scales(fmt, scale_in, amax_out, where):
    for t, name in ((scale_in, "scale_in"), (amax_out, "amax_out")):
        if t is not None:
            _vector(t, where, name, 1, torch.float32)
        elif fmt is not None:
            _refuse(where, f"8-bit results need {name}")


def _delayed_outputs(M, row_cols, col_rows, dev, fmt, layouts, scale_in, amax_out):
    """The delayed recipe's 8-bit outputs, and the C call's arguments for them."""
    if fmt is None:
        return None, (0, 0, None, None, None, None, 0, None)
    q = Quantized(None, None, None, None, max(16, (M + 15) // 16 * 16))
    scale = _stored_inverse(M, dev, scale_in)
    if layouts & LAYOUT_ROW:
        q.q_row, q.scale_inv_row = _u8(M, row_cols, dev), scale
    if layouts & LAYOUT_COLT:
        q.q_colT, q.scale_inv_col = _u8(col_rows, q.ld_colT, dev), scale
    return q, (fmt, layouts, scale_in.data_ptr(), amax_out.data_ptr(), _ptr(q.q_row), _ptr(q.q_colT), q.ld_colT,
               scale.data_ptr())


def mx_swiglu_gemm(A: torch.Tensor, fa: int, sA: torch.Tensor, W: torch.Tensor, fw: int, sW: torch.Tensor, K=None,
                   fmt=None, layouts: int = LAYOUT_ROW | LAYOUT_COLT, h: bool = False, gate_up: bool = False,
                   checkpoint_fmt=None, stream=None) -> SwigluGemm:
    """swiglu_gemm on MX operands; fmt: h in 8 bits with MX scales.  W quantized
    as two groups of F rows (host_offsets [0, F, 2 F]), which for F % 128 == 0 is
    what a plain mx_quantize gives."""
    if stream is not None:
        with _on(stream):
            return mx_swiglu_gemm(A, fa, sA, W, fw, sW, K, fmt, layouts, h, gate_up, checkpoint_fmt)
    where = "mx_swiglu_gemm"
    M, K = A.shape[0], A.shape[1] if K is None else K
    lda, ldw = _codes(A, where, "A", K), _codes(W, where, "W", K)
    if W.shape[0] % 2:
        _refuse(where, "W must have an even number of rows")
    F, dev = W.shape[0] // 2, A.device
    _mx_scales(sA, where, "sA", M, K)
    _mx_scales(sW, where, "sW", 2 * _groups_of(F), K)
    q, quant = _mx_gemm_outputs(M, F, F, dev, fmt, layouts)
    h, gate_up, c, rest = _swiglu_gemm_outputs(M, F, dev, h, gate_up, checkpoint_fmt)
    _check(load_library().fp8_mx_swiglu_gemm(A.data_ptr(), fa, lda, sA.data_ptr(), W.data_ptr(), fw, ldw,
                                             sW.data_ptr(), M, F, K, *quant, *rest, _stream(None)), where)
    return SwigluGemm(q, h, gate_up, c)


def _mx_gemm_outputs(M, row_cols, col_rows, dev, fmt, layouts):
    if fmt is None:
        return None, (0, 0, None, None, None, 0, None)
    q = _mx_split_outputs(M, row_cols, col_rows, dev, layouts)
    return q, (fmt, layouts, _ptr(q.q_row), _ptr(q.s_row), _ptr(q.q_colT), q.ld_colT, _ptr(q.s_col))


def swiglu_gemm_backward(A: torch.Tensor, fa: int, B: torch.Tensor, fb: int, sa: torch.Tensor, sb: torch.Tensor, src,
                         K=None, fmt=None, layouts: int = LAYOUT_ROW | LAYOUT_COLT, scale_in=None, amax_out=None,
                         d_gate_up: bool = False, stream=None) -> SwigluGemmBackward:
    """Gradient of gate|up from dh = A[:, :K] . B[:, :K]^T (A the output gradient's
    row layout, B u8 [F, K] the down weight's transposed layout) and src: bf16
    gate|up or its checkpoint.  Leaves it in 8 bits (fmt given: the delayed
    recipe) and / or in bf16."""
    if stream is not None:
        with _on(stream):
            return swiglu_gemm_backward(A, fa, B, fb, sa, sb, src, K, fmt, layouts, scale_in, amax_out, d_gate_up)
    where = "swiglu_gemm_backward"
    M, K = A.shape[0], A.shape[1] if K is None else K
    lda, ldb = _codes(A, where, "A", K), _codes(B, where, "B", K)
    F, dev = B.shape[0], A.device
    modes = _scale(sa, where, "sa", M), _scale(sb, where, "sb", F)
    _delayed_scales(fmt, scale_in, amax_out, where)
    kept = _kept(src, M, F, where)
    q, quant = _delayed_outputs(M, 2 * F, 2 * F, dev, fmt, layouts, scale_in, amax_out)
    d = torch.empty((M, 2 * F), dtype=torch.bfloat16, device=dev) if d_gate_up else None
    _check(load_library().fp8_swiglu_gemm_backward(A.data_ptr(), fa, lda, B.data_ptr(), fb, ldb, M, F, K,
                                                   sa.data_ptr(), modes[0], sb.data_ptr(), modes[1], *kept, *quant,
                                                   _ptr(d), 2 * F, _stream(None)), where)
    return SwigluGemmBackward(q, d)


def mx_swiglu_gemm_backward(A: torch.Tensor, fa: int, sA: torch.Tensor, B: torch.Tensor, fb: int, sB: torch.Tensor,
                            src, K=None, fmt=None, layouts: int = LAYOUT_ROW | LAYOUT_COLT, d_gate_up: bool = False,
                            stream=None) -> SwigluGemmBackward:
    """swiglu_gemm_backward on MX operands.  The row layout's halves are padded to
    whole groups of 128 columns, as the columns of W quantized in two groups are
    (its transposed layout is the other operand of the input's gradient); the
    transposed layout's rows are the 2 F of W."""
    if stream is not None:
        with _on(stream):
            return mx_swiglu_gemm_backward(A, fa, sA, B, fb, sB, src, K, fmt, layouts, d_gate_up)
    where = "mx_swiglu_gemm_backward"
    M, K = A.shape[0], A.shape[1] if K is None else K
    lda, ldb = _codes(A, where, "A", K), _codes(B, where, "B", K)
    F, dev = B.shape[0], A.device
    _mx_scales(sA, where, "sA", M, K)
    _mx_scales(sB, where, "sB", F, K)
    kept = _kept(src, M, F, where)
    q, quant = _mx_gemm_outputs(M, 2 * _groups_of(F), 2 * F, dev, fmt, layouts)
    d = torch.empty((M, 2 * F), dtype=torch.bfloat16, device=dev) if d_gate_up else None
    _check(load_library().fp8_mx_swiglu_gemm_backward(A.data_ptr(), fa, lda, sA.data_ptr(), B.data_ptr(), fb, ldb,
                                                      sB.data_ptr(), M, F, K, *kept, *quant, _ptr(d), 2 * F,
                                                      _stream(None)), where)
    return SwigluGemmBackward(q, d)
