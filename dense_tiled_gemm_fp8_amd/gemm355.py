"""ctypes binding of libgemm355 (include/gemm355.h): argument marshalling only.

Every function here has the name of the C entry point it wraps and does no
arithmetic of its own: all work runs in the library's HIP kernels.  Pointers
may be passed as torch tensors (their ``data_ptr()``) or plain integers;
``stream=None`` means torch's current stream on the current device.

Importing this module loads ``libgemm355.so`` and raises ImportError if it
has not been built (``python -m dense_tiled_gemm_fp8_amd.build``).
"""
from __future__ import annotations

import ctypes
import os
from typing import Any, Dict, Optional

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgemm355.so")

if not os.path.exists(LIB_PATH):
    raise ImportError("libgemm355.so is not built; run python -m dense_tiled_gemm_fp8_amd.build")
# One HIP runtime per process: PyTorch's ROCm wheels carry their own
# libamdhip64, which they load under a name the dynamic loader does not match
# to a runtime already loaded from the system ROCm, so loading this library
# first would leave two runtimes (and torch's device memory foreign to the
# one this library launches on).  Loaded after torch, the library binds to
# torch's runtime.
try:
    import torch  # noqa: F401
except ImportError:   # no PyTorch in the process: the system runtime is the only one
    pass
_lib = ctypes.CDLL(LIB_PATH)

# status codes
OK, EINVAL, EALIGN, EUNSUPPORTED, ENOMEM, EHIP, ETOOBIG = range(7)
# dtypes (input -> output)
(BF16_F32, BF16_BF16, E4M3_F32, E4M3_BF16, E5M2_F32, E5M2_BF16, E4M3_E5M2_F32,
 E4M3_E5M2_BF16, MXE4M3_F32, MXE4M3_BF16, MXE5M2_F32, MXE5M2_BF16, MXE4M3_E5M2_F32,
 MXE4M3_E5M2_BF16, MXFP4_F32, MXFP4_BF16, MXFP6_E2M3_F32, MXFP6_E2M3_BF16, MXFP6_E3M2_F32,
 MXFP6_E3M2_BF16) = range(20)
# 8-bit formats and source types of the quantiser
FP8_E4M3, FP8_E5M2 = range(2)
SRC_F32, SRC_BF16 = range(2)
# formats of a matrix held in 4 bits
W4_INT, W4_MXFP4 = range(2)
# activations of the gated pair of products
ACT_SILU, ACT_GELU_TANH = range(2)
# layouts
A_ROW_B_COL, A_ROW_B_ROW, A_COL_B_COL, A_COL_B_ROW = range(4)

_i64, _i32, _vp, _f64, _sz = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_double, ctypes.c_size_t


class gemm355_args(ctypes.Structure):
    _fields_ = [
        ("M", _i64), ("N", _i64), ("K", _i64),
        ("A", _vp), ("lda", _i64), ("stride_a", _i64),
        ("B", _vp), ("ldb", _i64), ("stride_b", _i64),
        ("C", _vp), ("ldc", _i64), ("stride_c", _i64),
        ("batch", _i64),
        ("scale_a", _vp), ("scale_b", _vp),
        ("dtype", ctypes.c_int), ("layout", ctypes.c_int),
        ("split_k", _i32), ("persistent", _i32), ("tile", _i32), ("cus", _i32),
        ("workspace", _vp), ("workspace_bytes", _sz),
        ("unit_stamps", _vp),
        ("block_scale_a", _vp), ("block_scale_b", _vp),
    ]


class gemm355_plan_t(ctypes.Structure):
    _fields_ = [
        ("tile", _i32), ("T_M", _i32), ("T_N", _i32), ("T_K", _i32),
        ("stages", _i32), ("waves", _i32), ("lds_bytes", _i32), ("vgpr_budget", _i32),
        ("S", _i32), ("b", _i32),
        ("G", _i64), ("nK", _i64), ("M_pad", _i64), ("N_pad", _i64), ("K_pad", _i64),
        ("split", _i32), ("persistent", _i32),
        ("tail_tiles", _i64), ("tail_split", _i32), ("repack", _i32),
        ("units", _i64), ("grid", _i64),
        ("eta_wave_num", _i64), ("eta_wave_den", _i64),
        ("eta_pad_num", _i64), ("eta_pad_den", _i64),
        ("eta_sched_num", _i64), ("eta_sched_den", _i64),
        ("workspace_bytes", _sz),
        ("model_seconds", ctypes.c_double),
        ("model_mfma_peak_seconds", ctypes.c_double), ("model_mfma_eff", ctypes.c_double),
        ("model_bytes", ctypes.c_double), ("model_spread", ctypes.c_double),
        ("model_stream_eff", ctypes.c_double), ("model_copy_seconds", ctypes.c_double),
        ("model_fixed_seconds", ctypes.c_double), ("model_units_in_turn", _i64),
    ]


class gemm355_conv_args(ctypes.Structure):
    _fields_ = [
        ("N", _i64), ("H", _i64), ("W", _i64), ("C", _i64),
        ("K", _i64), ("R", _i64), ("S", _i64),
        ("pad_h", _i64), ("pad_w", _i64), ("stride_h", _i64), ("stride_w", _i64),
        ("dil_h", _i64), ("dil_w", _i64),
        ("x", _vp), ("w", _vp), ("y", _vp),
        ("dtype", ctypes.c_int),
        ("split_k", _i32), ("persistent", _i32), ("tile", _i32), ("cus", _i32),
        ("workspace", _vp), ("workspace_bytes", _sz),
    ]


class gemm355_w4_matrix(ctypes.Structure):
    _fields_ = [
        ("N", _i64), ("K", _i64), ("codes", _vp), ("ldw", _i64), ("scales", _vp), ("zeros", _vp),
        ("fmt", ctypes.c_int), ("group", _i32),
    ]


class gemm355_kv_cache(ctypes.Structure):
    _fields_ = [
        ("k", _vp), ("v", _vp), ("k_scale", _vp), ("v_scale", _vp),
        ("pages", _i64), ("heads", _i32), ("head_dim", _i32), ("page", _i32),
        ("batch", _i64), ("table", _vp), ("table_ld", _i64), ("lens", _vp), ("q_start", _vp),
        ("tokens", _i64), ("max_new", _i64), ("max_len", _i64),
    ]


class gemm355_kv_append_args(ctypes.Structure):
    _fields_ = [
        ("cache", gemm355_kv_cache),
        ("k", _vp), ("ldk", _i64), ("v", _vp), ("ldv", _i64), ("q", _vp), ("ldq", _i64),
        ("q_out", _vp), ("ldqo", _i64),
        ("q_heads", _i32), ("rot_dim", _i32), ("interleaved", _i32),
        ("cos", _vp), ("sin", _vp), ("rot_len", _i64),
    ]


class gemm355_attention_args(ctypes.Structure):
    _fields_ = [
        ("cache", gemm355_kv_cache),
        ("q", _vp), ("ldq", _i64), ("o", _vp), ("ldo", _i64), ("lse", _vp),
        ("q_heads", _i32), ("scale", ctypes.c_float), ("window", _i64), ("sinks", _i64), ("splits", _i32),
        ("workspace", _vp), ("workspace_bytes", _sz),
    ]


class gemm355_block_matrix(ctypes.Structure):
    _fields_ = [
        ("rows", _i64), ("K", _i64), ("codes", _vp), ("ld", _i64), ("scales", _vp), ("ld_scale", _i64), ("block_rows", _i32),
    ]


class gemm355_rmsnorm_args(ctypes.Structure):
    _fields_ = [
        ("rows", _i64), ("width", _i64),
        ("x", _vp), ("ldx", _i64), ("x_type", ctypes.c_int),
        ("residual", _vp), ("ldr", _i64), ("r_type", ctypes.c_int),
        ("sum", _vp), ("lds", _i64),
        ("weight", _vp), ("w_type", ctypes.c_int),
        ("eps", ctypes.c_float),
        ("y", _vp), ("ldy", _i64), ("y_type", ctypes.c_int),
        ("q", ctypes.POINTER(gemm355_block_matrix)),
    ]


class gemm355_block_gemm_args(ctypes.Structure):
    _fields_ = [
        ("x", gemm355_block_matrix), ("w", gemm355_block_matrix),
        ("y", _vp), ("ldy", _i64), ("out", ctypes.c_int), ("splits", _i32),
        ("workspace", _vp), ("workspace_bytes", _sz),
    ]


class gemm355_block_gated_args(ctypes.Structure):
    _fields_ = [
        ("x", gemm355_block_matrix), ("gate", gemm355_block_matrix), ("up", gemm355_block_matrix), ("act", ctypes.c_int),
        ("y", _vp), ("ldy", _i64), ("out", ctypes.c_int), ("q", gemm355_block_matrix), ("splits", _i32),
        ("workspace", _vp), ("workspace_bytes", _sz),
    ]


_lib.gemm355_gemm.restype = ctypes.c_int
_lib.gemm355_gemm.argtypes = [_i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64,
                              ctypes.c_int, ctypes.c_int, _i32, _i32, _vp]
_lib.gemm355_gemm_ex.restype = ctypes.c_int
_lib.gemm355_gemm_ex.argtypes = [ctypes.POINTER(gemm355_args), _vp]
_lib.gemm355_gemm_noalloc.restype = ctypes.c_int
_lib.gemm355_gemm_noalloc.argtypes = [ctypes.POINTER(gemm355_args), _vp]
_lib.gemm355_plan.restype = ctypes.c_int
_lib.gemm355_plan.argtypes = [ctypes.POINTER(gemm355_args), ctypes.POINTER(gemm355_plan_t)]
_lib.gemm355_eta_wave.restype = _f64
_lib.gemm355_eta_wave.argtypes = [_i64, _i32, _i32]
_lib.gemm355_eta_pad.restype = _f64
_lib.gemm355_eta_pad.argtypes = [_i64] * 6
_lib.gemm355_kslice.restype = ctypes.c_int
_lib.gemm355_kslice.argtypes = [_i64, _i32, _i32, ctypes.POINTER(_i64), ctypes.POINTER(_i64)]
_lib.gemm355_unit.restype = ctypes.c_int
_lib.gemm355_unit.argtypes = [ctypes.POINTER(gemm355_args), _i64] + [ctypes.POINTER(_i64)] * 5
_lib.gemm355_num_tiles.restype = _i32
_lib.gemm355_num_tiles.argtypes = []
_lib.gemm355_tile_info.restype = ctypes.c_int
_lib.gemm355_tile_info.argtypes = [_i32] + [ctypes.POINTER(_i32)] * 10
_lib.gemm355_tile_occupancy.restype = ctypes.c_int
_lib.gemm355_tile_occupancy.argtypes = [_i32, ctypes.POINTER(_i32)]
_lib.gemm355_quantize.restype = ctypes.c_int
_lib.gemm355_quantize.argtypes = [_vp, _i64, _i64, ctypes.c_int, ctypes.c_int, _vp, _vp, _vp]
_lib.gemm355_conv2d.restype = ctypes.c_int
_lib.gemm355_conv2d.argtypes = [ctypes.POINTER(gemm355_conv_args), _vp]
_lib.gemm355_conv2d_plan.restype = ctypes.c_int
_lib.gemm355_conv2d_plan.argtypes = [ctypes.POINTER(gemm355_conv_args), ctypes.POINTER(gemm355_plan_t)]
_lib.gemm355_conv2d_out_size.restype = ctypes.c_int
_lib.gemm355_conv2d_out_size.argtypes = [ctypes.POINTER(gemm355_conv_args), ctypes.POINTER(_i64),
                                         ctypes.POINTER(_i64)]
_lib.gemm355_set_scratch_limit.restype = ctypes.c_int
_lib.gemm355_set_scratch_limit.argtypes = [ctypes.c_uint64, ctypes.POINTER(ctypes.c_uint64)]
_w4p = ctypes.POINTER(gemm355_w4_matrix)
_lib.gemm355_w4_quantize.restype = ctypes.c_int
_lib.gemm355_w4_quantize.argtypes = [_vp, _i64, ctypes.c_int, _w4p, _vp]
_lib.gemm355_w4_dequantize.restype = ctypes.c_int
_lib.gemm355_w4_dequantize.argtypes = [_w4p, _vp, _i64, ctypes.c_int, _vp]
_lib.gemm355_w4_gemm.restype = ctypes.c_int
_lib.gemm355_w4_gemm.argtypes = [_i64, _vp, _i64, _w4p, _vp, _i64, ctypes.c_int, _vp]
_lib.gemm355_kv_append.restype = ctypes.c_int
_lib.gemm355_kv_append.argtypes = [ctypes.POINTER(gemm355_kv_append_args), _vp]
_lib.gemm355_attention.restype = ctypes.c_int
_lib.gemm355_attention.argtypes = [ctypes.POINTER(gemm355_attention_args), _vp]
_lib.gemm355_attention_workspace.restype = ctypes.c_int
_lib.gemm355_attention_workspace.argtypes = [ctypes.POINTER(gemm355_attention_args), ctypes.POINTER(_sz)]
_lib.gemm355_block_quantize.restype = ctypes.c_int
_lib.gemm355_block_quantize.argtypes = [_vp, _i64, ctypes.c_int, ctypes.POINTER(gemm355_block_matrix), _vp]
_lib.gemm355_rmsnorm.restype = ctypes.c_int
_lib.gemm355_rmsnorm.argtypes = [ctypes.POINTER(gemm355_rmsnorm_args), _vp]
_lib.gemm355_block_gemm.restype = ctypes.c_int
_lib.gemm355_block_gemm.argtypes = [ctypes.POINTER(gemm355_block_gemm_args), _vp]
_lib.gemm355_block_gemm_workspace.restype = ctypes.c_int
_lib.gemm355_block_gemm_workspace.argtypes = [ctypes.POINTER(gemm355_block_gemm_args), ctypes.POINTER(_sz)]
_lib.gemm355_block_gated.restype = ctypes.c_int
_lib.gemm355_block_gated.argtypes = [ctypes.POINTER(gemm355_block_gated_args), _vp]
_lib.gemm355_block_gated_workspace.restype = ctypes.c_int
_lib.gemm355_block_gated_workspace.argtypes = [ctypes.POINTER(gemm355_block_gated_args), ctypes.POINTER(_sz)]
_lib.gemm355_status_string.restype = ctypes.c_char_p
_lib.gemm355_status_string.argtypes = [ctypes.c_int]

EXPORTED = ("gemm355_gemm", "gemm355_gemm_ex", "gemm355_gemm_noalloc",
            "gemm355_plan", "gemm355_eta_wave",
            "gemm355_eta_pad", "gemm355_kslice", "gemm355_unit", "gemm355_num_tiles",
            "gemm355_tile_info", "gemm355_tile_occupancy", "gemm355_quantize",
            "gemm355_conv2d", "gemm355_conv2d_plan", "gemm355_conv2d_out_size", "gemm355_set_scratch_limit",
            "gemm355_w4_quantize", "gemm355_w4_dequantize", "gemm355_w4_gemm", "gemm355_kv_append",
            "gemm355_attention", "gemm355_attention_workspace", "gemm355_block_quantize", "gemm355_rmsnorm",
            "gemm355_block_gemm", "gemm355_block_gemm_workspace", "gemm355_block_gated", "gemm355_block_gated_workspace",
            "gemm355_status_string")


class Gemm355Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s: %s (status %d)" % (where, gemm355_status_string(status), status))


def _ptr(x: Any) -> Optional[int]:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return int(x.data_ptr())


_raw_stream = None   # handle of torch's current stream on the current device, once a device is known


def _find_raw_stream():
    """torch's own lookup of the current stream's handle where it has one (0.3 us;
    building the stream object takes 3 us, as long as a launch)."""
    global _raw_stream
    import torch
    if not torch.cuda.is_available():
        return None
    torch.cuda.init()
    raw, device = getattr(torch._C, "_cuda_getCurrentRawStream", None), getattr(torch._C, "_cuda_getDevice", None)
    if raw is not None and device is not None:
        _raw_stream = lambda: raw(device())  # noqa: E731
    else:
        _raw_stream = lambda: int(torch.cuda.current_stream().cuda_stream)  # noqa: E731
    return _raw_stream


def _stream(stream: Any) -> Optional[int]:
    if stream is None:
        find = _raw_stream or _find_raw_stream()
        return find() if find is not None else None
    if isinstance(stream, int):
        return stream
    return int(stream.cuda_stream)


def _check(status: int, where: str) -> None:
    if status != OK:
        raise Gemm355Error(status, where)


def gemm355_status_string(status: int) -> str:
    return _lib.gemm355_status_string(status).decode()


def gemm355_gemm(M, N, K, A, lda, B, ldb, C, ldc, dtype, layout=A_ROW_B_COL, split_k=0,
                 persistent=-1, stream=None) -> None:
    _check(_lib.gemm355_gemm(M, N, K, _ptr(A), lda, _ptr(B), ldb, _ptr(C), ldc, dtype, layout,
                             split_k, persistent, _stream(stream)), "gemm355_gemm")


def make_args(M, N, K, A=None, lda=None, B=None, ldb=None, C=None, ldc=None, dtype=BF16_F32,
              layout=A_ROW_B_COL, batch=1, stride_a=0, stride_b=0, stride_c=0, scale_a=None,
              scale_b=None, split_k=0, persistent=-1, tile=-1, cus=0, workspace=None,
              workspace_bytes=0, unit_stamps=None, block_scale_a=None,
              block_scale_b=None) -> gemm355_args:
    """Fill a gemm355_args; leading dimensions default to the packed ones."""
    a_row = layout in (A_ROW_B_COL, A_ROW_B_ROW)
    b_col = layout in (A_ROW_B_COL, A_COL_B_COL)
    if lda is None:
        lda = max(1, K if a_row else M)
    if ldb is None:
        ldb = max(1, K if b_col else N)
    if ldc is None:
        ldc = max(1, N)
    return gemm355_args(M, N, K, _ptr(A), lda, stride_a, _ptr(B), ldb, stride_b, _ptr(C), ldc,
                        stride_c, batch, _ptr(scale_a), _ptr(scale_b), dtype, layout, split_k,
                        persistent, tile, cus, _ptr(workspace), workspace_bytes, _ptr(unit_stamps),
                        _ptr(block_scale_a), _ptr(block_scale_b))


def gemm355_gemm_ex(args: gemm355_args, stream=None) -> None:
    _check(_lib.gemm355_gemm_ex(ctypes.byref(args), _stream(stream)), "gemm355_gemm_ex")


def gemm355_gemm_noalloc(args: gemm355_args, stream=None) -> None:
    _check(_lib.gemm355_gemm_noalloc(ctypes.byref(args), _stream(stream)), "gemm355_gemm_noalloc")


def gemm355_plan(args: gemm355_args) -> Dict[str, int]:
    out = gemm355_plan_t()
    _check(_lib.gemm355_plan(ctypes.byref(args), ctypes.byref(out)), "gemm355_plan")
    return {name: getattr(out, name) for name, _ in gemm355_plan_t._fields_}


def gemm355_eta_wave(G: int, S: int, b: int) -> float:
    return _lib.gemm355_eta_wave(G, S, b)


def gemm355_eta_pad(M: int, N: int, K: int, T_M: int, T_N: int, T_K: int) -> float:
    return _lib.gemm355_eta_pad(M, N, K, T_M, T_N, T_K)


def gemm355_kslice(nK: int, s: int, i: int):
    b, e = _i64(), _i64()
    _check(_lib.gemm355_kslice(nK, s, i, ctypes.byref(b), ctypes.byref(e)), "gemm355_kslice")
    return b.value, e.value


def gemm355_unit(args: gemm355_args, u: int):
    vals = [_i64() for _ in range(5)]
    _check(_lib.gemm355_unit(ctypes.byref(args), u, *[ctypes.byref(v) for v in vals]),
           "gemm355_unit")
    return tuple(v.value for v in vals)   # batch, tile_m, tile_n, kt_begin, kt_end


def gemm355_num_tiles() -> int:
    return _lib.gemm355_num_tiles()


def gemm355_tile_info(tile: int) -> Dict[str, int]:
    vals = [_i32() for _ in range(10)]
    _check(_lib.gemm355_tile_info(tile, *[ctypes.byref(v) for v in vals]), "gemm355_tile_info")
    names = ("dtype_class", "T_M", "T_N", "T_K", "stages", "waves", "lds_bytes", "b_max", "op", "schedule")
    return dict(zip(names, (v.value for v in vals)))


SCRATCH_UNLIMITED = (1 << 64) - 1


def gemm355_set_scratch_limit(nbytes: int) -> int:
    """Cap on library-owned scratch (SCRATCH_UNLIMITED: none); returns the previous cap."""
    prev = ctypes.c_uint64()
    _check(_lib.gemm355_set_scratch_limit(nbytes, ctypes.byref(prev)), "gemm355_set_scratch_limit")
    return prev.value


def gemm355_tile_occupancy(tile: int) -> int:
    n = _i32()
    _check(_lib.gemm355_tile_occupancy(tile, ctypes.byref(n)), "gemm355_tile_occupancy")
    return n.value


def make_conv_args(N, H, W, C, K, R, S, x=None, w=None, y=None, pad_h=0, pad_w=0, stride_h=1,
                   stride_w=1, dil_h=1, dil_w=1, dtype=BF16_F32, split_k=0, persistent=-1, tile=-1,
                   cus=0, workspace=None, workspace_bytes=0) -> gemm355_conv_args:
    return gemm355_conv_args(N, H, W, C, K, R, S, pad_h, pad_w, stride_h, stride_w, dil_h, dil_w,
                             _ptr(x), _ptr(w), _ptr(y), dtype, split_k, persistent, tile, cus,
                             _ptr(workspace), workspace_bytes)


def gemm355_conv2d(args: gemm355_conv_args, stream=None) -> None:
    _check(_lib.gemm355_conv2d(ctypes.byref(args), _stream(stream)), "gemm355_conv2d")


def gemm355_conv2d_out_size(args: gemm355_conv_args):
    """(P, Q): the output extent the library gives this convolution."""
    P, Q = _i64(), _i64()
    _check(_lib.gemm355_conv2d_out_size(ctypes.byref(args) if args is not None else None, ctypes.byref(P),
                                        ctypes.byref(Q)), "gemm355_conv2d_out_size")
    return P.value, Q.value


def gemm355_conv2d_plan(args: gemm355_conv_args) -> Dict[str, int]:
    out = gemm355_plan_t()
    _check(_lib.gemm355_conv2d_plan(ctypes.byref(args) if args is not None else None, ctypes.byref(out)),
           "gemm355_conv2d_plan")
    return {name: getattr(out, name) for name, _ in gemm355_plan_t._fields_}


def gemm355_quantize(x, n, batch, src, fmt, q, scale, stream=None) -> None:
    """Per-tensor scaling of `batch` tensors of n elements to 8-bit codes q,
    dequantisation factors into scale[batch] (device pointers or tensors)."""
    _check(_lib.gemm355_quantize(_ptr(x), n, batch, src, fmt, _ptr(q), _ptr(scale), _stream(stream)),
           "gemm355_quantize")


def make_w4_matrix(N, K, codes=None, scales=None, zeros=None, fmt=W4_INT, group=128, ldw=0) -> gemm355_w4_matrix:
    """Descriptor of an N x K matrix in 4 bits; it holds addresses, so the
    tensors must outlive it.  ldw = 0: rows of K rounded up to 32 codes."""
    return gemm355_w4_matrix(N, K, _ptr(codes), ldw, _ptr(scales), _ptr(zeros), fmt, group)


def gemm355_w4_quantize(w, matrix: gemm355_w4_matrix, src=SRC_BF16, ld=0, stream=None) -> None:
    """Codes, scales and zero points (if any) of `matrix` from the rows of w."""
    _check(_lib.gemm355_w4_quantize(_ptr(w), ld, src, ctypes.byref(matrix), _stream(stream)), "gemm355_w4_quantize")


def gemm355_w4_dequantize(matrix: gemm355_w4_matrix, w, dst=SRC_BF16, ld=0, stream=None) -> None:
    """The values that `matrix` stands for, into the rows of w."""
    _check(_lib.gemm355_w4_dequantize(ctypes.byref(matrix), _ptr(w), ld, dst, _stream(stream)),
           "gemm355_w4_dequantize")


def gemm355_w4_gemm(M, x, matrix: gemm355_w4_matrix, y, out=SRC_BF16, ldx=0, ldy=0, stream=None) -> None:
    """y (M x N, type `out`) = x (M x K, bf16) times the transpose of `matrix`."""
    _check(_lib.gemm355_w4_gemm(M, _ptr(x), ldx, ctypes.byref(matrix), _ptr(y), ldy, out, _stream(stream)),
           "gemm355_w4_gemm")


def make_kv_cache(k=None, v=None, k_scale=None, v_scale=None, pages=0, heads=0, head_dim=0, page=0, table=None,
                  lens=None, batch=0, max_len=0, q_start=None, tokens=0, max_new=1, table_ld=0) -> gemm355_kv_cache:
    """Descriptor of a paged cache and one step on it (addresses only)."""
    return gemm355_kv_cache(_ptr(k), _ptr(v), _ptr(k_scale), _ptr(v_scale), pages, heads, head_dim, page, batch,
                            _ptr(table), table_ld, _ptr(lens), _ptr(q_start), tokens, max_new, max_len)


def make_kv_append_args(cache: gemm355_kv_cache, k=None, v=None, q=None, q_out=None, q_heads=0, cos=None, sin=None,
                        rot_dim=0, rot_len=0, interleaved=False, ldk=0, ldv=0, ldq=0,
                        ldqo=0) -> gemm355_kv_append_args:
    return gemm355_kv_append_args(cache, _ptr(k), ldk, _ptr(v), ldv, _ptr(q), ldq, _ptr(q_out), ldqo, q_heads,
                                  rot_dim, 1 if interleaved else 0, _ptr(cos), _ptr(sin), rot_len)


def gemm355_kv_append(args: gemm355_kv_append_args, stream=None) -> None:
    """The step's keys (rotated) and values into the cache, and the rotated queries."""
    _check(_lib.gemm355_kv_append(ctypes.byref(args), _stream(stream)), "gemm355_kv_append")


def make_attention_args(cache: gemm355_kv_cache, q=None, o=None, q_heads=0, lse=None, scale=0.0, window=0, sinks=0,
                        splits=0, ldq=0, ldo=0, workspace=None, workspace_bytes=0) -> gemm355_attention_args:
    return gemm355_attention_args(cache, _ptr(q), ldq, _ptr(o), ldo, _ptr(lse), q_heads, scale, window, sinks, splits,
                                  _ptr(workspace), workspace_bytes)


def gemm355_attention(args: gemm355_attention_args, stream=None) -> None:
    """Attention of the step's queries over the cache."""
    _check(_lib.gemm355_attention(ctypes.byref(args), _stream(stream)), "gemm355_attention")


def gemm355_attention_workspace(args: gemm355_attention_args) -> int:
    """Scratch bytes of that call (0: none)."""
    n = _sz()
    _check(_lib.gemm355_attention_workspace(ctypes.byref(args), ctypes.byref(n)), "gemm355_attention_workspace")
    return n.value


def make_block_matrix(rows, K, codes=None, scales=None, block_rows=1, ld=0, ld_scale=0) -> gemm355_block_matrix:
    """Descriptor of a rows x K matrix of E4M3 codes with a scale for each 128
    K-values of `block_rows` rows; it holds addresses, so the tensors must
    outlive it."""
    return gemm355_block_matrix(rows, K, _ptr(codes), ld, _ptr(scales), ld_scale, block_rows)


def gemm355_block_quantize(x, matrix: gemm355_block_matrix, src=SRC_BF16, ld=0, stream=None) -> None:
    """Codes and scales of `matrix` from the rows of x."""
    _check(_lib.gemm355_block_quantize(_ptr(x), ld, src, ctypes.byref(matrix), _stream(stream)), "gemm355_block_quantize")


def make_rmsnorm_args(rows, width, x=None, x_type=SRC_BF16, residual=None, sum=None, r_type=SRC_BF16, weight=None,
                      w_type=SRC_BF16, eps=1e-5, y=None, y_type=SRC_BF16, q: Optional[gemm355_block_matrix] = None, ldx=0,
                      ldr=0, lds=0, ldy=0) -> gemm355_rmsnorm_args:
    return gemm355_rmsnorm_args(rows, width, _ptr(x), ldx, x_type, _ptr(residual), ldr, r_type, _ptr(sum), lds, _ptr(weight),
                                w_type, eps, _ptr(y), ldy, y_type, ctypes.pointer(q) if q is not None else None)


def gemm355_rmsnorm(args: gemm355_rmsnorm_args, stream=None) -> None:
    """The residual's addition and the norm of its rows, as rows, codes or both."""
    _check(_lib.gemm355_rmsnorm(ctypes.byref(args), _stream(stream)), "gemm355_rmsnorm")


def make_block_gemm_args(x: gemm355_block_matrix, w: gemm355_block_matrix, y=None, out=SRC_BF16, ldy=0, splits=0,
                         workspace=None, workspace_bytes=0) -> gemm355_block_gemm_args:
    return gemm355_block_gemm_args(x, w, _ptr(y), ldy, out, splits, _ptr(workspace), workspace_bytes)


def gemm355_block_gemm(args: gemm355_block_gemm_args, stream=None) -> None:
    """y = x times the transpose of w, both with a scale for each block of 128."""
    _check(_lib.gemm355_block_gemm(ctypes.byref(args), _stream(stream)), "gemm355_block_gemm")


def gemm355_block_gemm_workspace(args: gemm355_block_gemm_args) -> int:
    """Scratch bytes of that call (0: none)."""
    n = _sz()
    _check(_lib.gemm355_block_gemm_workspace(ctypes.byref(args), ctypes.byref(n)), "gemm355_block_gemm_workspace")
    return n.value


def make_block_gated_args(x: gemm355_block_matrix, gate: gemm355_block_matrix, up: gemm355_block_matrix, act=ACT_SILU, y=None,
                          out=SRC_BF16, ldy=0, q: Optional[gemm355_block_matrix] = None, splits=0, workspace=None,
                          workspace_bytes=0) -> gemm355_block_gated_args:
    return gemm355_block_gated_args(x, gate, up, act, _ptr(y), ldy, out, q if q is not None else gemm355_block_matrix(), splits,
                                    _ptr(workspace), workspace_bytes)


def gemm355_block_gated(args: gemm355_block_gated_args, stream=None) -> None:
    """act(x gate^T) * (x up^T), as rows or as codes with scales."""
    _check(_lib.gemm355_block_gated(ctypes.byref(args), _stream(stream)), "gemm355_block_gated")


def gemm355_block_gated_workspace(args: gemm355_block_gated_args) -> int:
    """Scratch bytes of that call (0: none)."""
    n = _sz()
    _check(_lib.gemm355_block_gated_workspace(ctypes.byref(args), ctypes.byref(n)), "gemm355_block_gated_workspace")
    return n.value
