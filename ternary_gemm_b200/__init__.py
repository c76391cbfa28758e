"""B200-native H-BitLinear forward (BitNet v2): CUDA kernels behind a C ABI.

The functions below carry the names of the C entry points in include/hbl.h and
only marshal arguments: torch tensors supply device memory and the current
CUDA stream, every step of the computation runs in libhbl.so.  Outputs that
the caller does not pass are allocated here with torch (the library itself
never allocates).  With `stream=` a call runs on that stream and its own
allocations belong to it; tensors that are passed in must be ready there, and
be kept (or marked, Tensor.record_stream) until the stream is done with them.
If libhbl.so is missing or fails to load, every call raises -- there is no CPU
fallback.
"""
from __future__ import annotations

import ctypes
import os
import re
import threading

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libhbl.so")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "hbl.h")

HBL_OK, HBL_ERR_INVALID_ARG, HBL_ERR_UNSUPPORTED, HBL_ERR_WORKSPACE, HBL_ERR_CUDA, HBL_ERR_TIMEOUT = range(6)
HBL_F32, HBL_BF16 = 0, 1
HBL_NORM_LAYER, HBL_NORM_RMS = 0, 1

_lock = threading.Lock()
_lib = None


class HBLError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        self.cuda_error = None
        msg = "%s failed: %s" % (where, status_string(status))
        if status == HBL_ERR_CUDA:
            self.cuda_error = int(lib().hbl_last_cuda_error())
            msg += " (%s)" % lib().hbl_cuda_error_name(self.cuda_error).decode()
        super().__init__(msg)


def declared_symbols():
    """Names of the functions declared in include/hbl.h."""
    text = open(HEADER_PATH).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(hbl_[a-z0-9_]+)\s*\(", text)))


def lib():
    """The loaded libhbl.so (ctypes); raises if it is not built."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise ImportError("libhbl.so is not built (run python -m ternary_gemm_b200.build); "
                                  "there is no fallback path")
            L = ctypes.CDLL(LIB_PATH)
            p, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
            L.hbl_packed_ternary_bytes.argtypes = [i64, i64]
            L.hbl_packed_ternary_bytes.restype = sz
            L.hbl_codes_bytes.argtypes = [i64, i64, i32]
            L.hbl_codes_bytes.restype = sz
            L.hbl_pack_ternary_workspace_bytes.argtypes = [i64, i64]
            L.hbl_pack_ternary_workspace_bytes.restype = sz
            L.hbl_forward_workspace_bytes.argtypes = [i64, i64, i64, i32]
            L.hbl_forward_workspace_bytes.restype = sz
            L.hbl_pack_ternary.argtypes = [p, i32, i64, i64, p, p, p, sz, p]
            L.hbl_pack_ternary.restype = i32
            L.hbl_fht_quant.argtypes = [p, i32, i64, i64, i32, p, p, p]
            L.hbl_fht_quant.restype = i32
            L.hbl_forward.argtypes = [p, i32, i64, i64, p, p, i64, i32, p, i32, p, sz, p]
            L.hbl_forward.restype = i32
            L.hbl_fht.argtypes = [p, i32, i64, i64, p, p]
            L.hbl_fht.restype = i32
            L.hbl_backward_workspace_bytes.argtypes = [i64, i64, i64, i32]
            L.hbl_backward_workspace_bytes.restype = sz
            L.hbl_backward.argtypes = [p, i32, i64, i64, p, p, i64, i32, p, i32, p, p, p, sz, p]
            L.hbl_backward.restype = i32
            L.hbl_gemm_bf16_f32.argtypes = [p, i32, p, i64, i64, i64, p, p, p]
            L.hbl_gemm_bf16_f32.restype = i32
            L.hbl_ln_backward.argtypes = [p, i32, i64, i64, p, p, p]
            L.hbl_ln_backward.restype = i32
            L.hbl_fht_ln_backward.argtypes = [p, p, i32, i64, i64, p, p]
            L.hbl_fht_ln_backward.restype = i32
            L.hbl_kv_quant.argtypes = [p, i32, i64, i64, i32, p, p, p]
            L.hbl_kv_quant.restype = i32
            L.hbl_pack_ternary_rotated_workspace_bytes.argtypes = [i64, i64]
            L.hbl_pack_ternary_rotated_workspace_bytes.restype = sz
            L.hbl_pack_ternary_rotated.argtypes = [p, i32, i64, i64, p, p, p, sz, p]
            L.hbl_pack_ternary_rotated.restype = i32
            L.hbl_norm_quant.argtypes = [p, i32, i64, i64, i32, i32, p, p, p]
            L.hbl_norm_quant.restype = i32
            L.hbl_debug_norm.argtypes = [p, i32, i64, i64, i32, p, p]
            L.hbl_debug_norm.restype = i32
            L.hbl_forward_noalloc.argtypes = [p, i32, i64, i64, p, p, i64, i32, p, i32, p]
            L.hbl_forward_noalloc.restype = i32
            L.hbl_fht_quant_i8.argtypes = [p, i32, i64, i64, i32, p, p, p]
            L.hbl_fht_quant_i8.restype = i32
            L.hbl_widen_ternary.argtypes = [p, i64, i64, p, p]
            L.hbl_widen_ternary.restype = i32
            L.hbl_gemm_dequant.argtypes = [p, p, i64, i64, i64, p, p, p, i32, p]
            L.hbl_gemm_dequant.restype = i32
            L.hbl_gemm_tern_dequant.argtypes = [p, p, i64, i64, i64, p, p, p, i32, p]
            L.hbl_gemm_tern_dequant.restype = i32
            L.hbl_gemv_ternary_dequant.argtypes = [p, p, i64, i64, i64, p, p, p, i32, p]
            L.hbl_gemv_ternary_dequant.restype = i32
            L.hbl_debug_ln_fht.argtypes = [p, i32, i64, i64, p, p]
            L.hbl_debug_ln_fht.restype = i32
            L.hbl_quant_from_f32.argtypes = [p, i64, i64, i32, p, p, p]
            L.hbl_quant_from_f32.restype = i32
            L.hbl_gemm_i8_i32.argtypes = [p, p, i64, i64, i64, p, p]
            L.hbl_gemm_i8_i32.restype = i32
            L.hbl_kv_plan.argtypes = [p, p, i64, i64, p, i64, p, p, i64, i64, p, p, p, p, p, p]
            L.hbl_kv_plan.restype = i32
            L.hbl_kv_append.argtypes = [p, p, i32, i64, i64, i64, i64, i64, p, i32, i64, i64, p, p, p, p, p]
            L.hbl_kv_append.restype = i32
            L.hbl_kv_attention_workspace_bytes.argtypes = [i64, i64, i64, i64, i64]
            L.hbl_kv_attention_workspace_bytes.restype = sz
            L.hbl_kv_attention.argtypes = [p, i32, i64, i64, i64, i64, i64, p, p, i64, p, i64, i64, i64, i32, p, p, p, p,
                                           p, p, i32, p, sz, p]
            L.hbl_kv_attention.restype = i32
            L.hbl_add_rms_quant.argtypes = [p, p, i32, i64, i64, p, i32, p, p, p, p]
            L.hbl_add_rms_quant.restype = i32
            L.hbl_add_rms_quant_backward_workspace_bytes.argtypes = [i64, i64]
            L.hbl_add_rms_quant_backward_workspace_bytes.restype = sz
            L.hbl_add_rms_quant_backward.argtypes = [p, i32, i64, i64, p, p, i32, p, p, p, p, sz, p]
            L.hbl_add_rms_quant_backward.restype = i32
            L.hbl_last_device_error.argtypes = [p]
            L.hbl_last_device_error.restype = i32
            L.hbl_debug_raise_device_error.argtypes = [p]
            L.hbl_debug_raise_device_error.restype = i32
            L.hbl_debug_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
            L.hbl_debug_set_wait_limit_ns.restype = i32
            L.hbl_status_string.argtypes = [i32]
            L.hbl_status_string.restype = ctypes.c_char_p
            L.hbl_last_cuda_error.argtypes = []
            L.hbl_last_cuda_error.restype = ctypes.c_int
            L.hbl_cuda_error_name.argtypes = [ctypes.c_int]
            L.hbl_cuda_error_name.restype = ctypes.c_char_p
            _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().hbl_status_string(int(status)).decode()


def _check(status: int, where: str):
    if status != HBL_OK:
        raise HBLError(status, where)


def _torch():
    import torch
    return torch


def _stream(stream):
    torch = _torch()
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.float32:
        return HBL_F32
    if t.dtype == torch.bfloat16:
        return HBL_BF16
    raise TypeError("expected float32 or bfloat16, got %s" % t.dtype)


def _ptr(t) -> ctypes.c_void_p:
    return ctypes.c_void_p(t.data_ptr())


def _new(stream, shape, dtype, like, zero=False, scratch=False):
    """A buffer that the caller did not pass, on the device of `like`, made (and filled) on the stream of the call, so
    that neither the fill nor a later owner of its memory can come between.  A result (not scratch, which is dropped on
    return) is marked as used on the caller's current stream too."""
    torch = _torch()
    make = torch.zeros if zero else torch.empty
    if stream is None:
        return make(shape, dtype=dtype, device=like.device)
    here = torch.cuda.current_stream(like.device)
    with torch.cuda.stream(stream):
        t = make(shape, dtype=dtype, device=like.device)
    if not scratch:
        t.record_stream(here)
    return t


def _need_cuda(*ts):
    for t in ts:
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("tensors must be contiguous CUDA tensors")


# ------------------------------------------------------------------ sizes

def hbl_packed_ternary_bytes(K: int, N: int) -> int:
    return int(lib().hbl_packed_ternary_bytes(K, N))


def hbl_codes_bytes(M: int, K: int, bits: int) -> int:
    return int(lib().hbl_codes_bytes(M, K, bits))


def hbl_pack_ternary_workspace_bytes(K: int, N: int) -> int:
    return int(lib().hbl_pack_ternary_workspace_bytes(K, N))


def hbl_forward_workspace_bytes(M: int, K: int, N: int, bits: int) -> int:
    return int(lib().hbl_forward_workspace_bytes(M, K, N, bits))


# ------------------------------------------------------------------ compute

def hbl_pack_ternary(W, packed=None, alpha=None, workspace=None, stream=None):
    """W [N][K] (float32/bf16) -> (packed uint8 [N][K/4], alpha float32 [1])."""
    torch = _torch()
    _need_cuda(W)
    N, K = W.shape
    if packed is None:
        packed = _new(stream, (N, K // 4), torch.uint8, W)
    if alpha is None:
        alpha = _new(stream, (1,), torch.float32, W)
    if workspace is None:
        workspace = _new(stream, (max(1, hbl_pack_ternary_workspace_bytes(K, N)),), torch.uint8, W, scratch=True)
    _check(lib().hbl_pack_ternary(_ptr(W), _dtype_code(W), K, N, _ptr(packed), _ptr(alpha), _ptr(workspace),
                                  workspace.numel(), _stream(stream)), "hbl_pack_ternary")
    return packed, alpha


def hbl_fht_quant(x, bits: int, codes=None, scales=None, stream=None):
    """x [M][K] -> (codes uint8 [M][K/2] (bits 4) or int8 [M][K] (bits 8), scales float32 [M])."""
    torch = _torch()
    _need_cuda(x)
    M, K = x.shape
    if codes is None:
        codes = _new(stream, (M, K // 2), torch.uint8, x) if bits == 4 else _new(stream, (M, K), torch.int8, x)
    if scales is None:
        scales = _new(stream, (M,), torch.float32, x)
    _check(lib().hbl_fht_quant(_ptr(x), _dtype_code(x), M, K, bits, _ptr(codes), _ptr(scales), _stream(stream)),
           "hbl_fht_quant")
    return codes, scales


def hbl_forward(x, packed, alpha, N: int, bits: int, y=None, y_dtype=None, workspace=None, stream=None):
    """x [M][K], packed ternary [N][K/4], alpha [1] -> y [M][N] (dtype of x unless y_dtype)."""
    torch = _torch()
    _need_cuda(x, packed, alpha)
    M, K = x.shape
    if y is None:
        y = _new(stream, (M, N), y_dtype or x.dtype, x)
    if workspace is None:
        workspace = _new(stream, (hbl_forward_workspace_bytes(M, K, N, bits),), torch.uint8, x, scratch=True)
    _check(lib().hbl_forward(_ptr(x), _dtype_code(x), M, K, _ptr(packed), _ptr(alpha), N, bits, _ptr(y),
                             _dtype_code(y), _ptr(workspace), workspace.numel(), _stream(stream)), "hbl_forward")
    return y


def hbl_backward_workspace_bytes(M: int, K: int, N: int, bits: int) -> int:
    return int(lib().hbl_backward_workspace_bytes(M, K, N, bits))


def hbl_backward(x, packed, alpha, N: int, bits: int, g_y, g_x=None, g_W=None, workspace=None, stream=None):
    """Straight-through-estimator gradients of hbl_forward: (g_x [M][K] of x's dtype, g_W float32 [N][K])."""
    torch = _torch()
    _need_cuda(x, packed, alpha, g_y)
    M, K = x.shape
    if g_x is None:
        g_x = _new(stream, (M, K), x.dtype, x)
    if g_W is None:
        g_W = _new(stream, (N, K), torch.float32, x)
    if workspace is None:
        workspace = _new(stream, (hbl_backward_workspace_bytes(M, K, N, bits),), torch.uint8, x, scratch=True)
    _check(lib().hbl_backward(_ptr(x), _dtype_code(x), M, K, _ptr(packed), _ptr(alpha), N, bits, _ptr(g_y),
                              _dtype_code(g_y), _ptr(g_x), _ptr(g_W), _ptr(workspace), workspace.numel(),
                              _stream(stream)), "hbl_backward")
    return g_x, g_W


def hbl_gemm_bf16_f32(A, B, a_mn: bool = False, scale=None, D=None, stream=None):
    """D = scale * A B on the tensor cores.  A bf16 [R][Kc] (a_mn False) or [Kc][R] (a_mn True),
    B bf16 [Kc][C], D float32 [R][C]; scale a device float32 [1] or None."""
    torch = _torch()
    _need_cuda(A, B)
    Kc, C = B.shape
    R = A.shape[1] if a_mn else A.shape[0]
    if D is None:
        D = _new(stream, (R, C), torch.float32, A)
    _check(lib().hbl_gemm_bf16_f32(_ptr(A), 1 if a_mn else 0, _ptr(B), R, C, Kc, _ptr(D),
                                   _ptr(scale) if scale is not None else None, _stream(stream)),
           "hbl_gemm_bf16_f32")
    return D


def hbl_ln_backward(x, g_u, g_x=None, stream=None):
    """LayerNorm backward (no affine): g_x [M][K] of x's dtype from x and float32 g_u."""
    _need_cuda(x, g_u)
    M, K = x.shape
    if g_x is None:
        g_x = _new(stream, (M, K), x.dtype, x)
    _check(lib().hbl_ln_backward(_ptr(x), _dtype_code(x), M, K, _ptr(g_u), _ptr(g_x), _stream(stream)),
           "hbl_ln_backward")
    return g_x


def hbl_fht_ln_backward(g, x, g_x=None, stream=None):
    """g_x [M][K] (x's dtype) = LayerNorm backward at x of H g / sqrt(K), g float32 [M][K]."""
    _need_cuda(g, x)
    M, K = x.shape
    if g_x is None:
        g_x = _new(stream, (M, K), x.dtype, x)
    _check(lib().hbl_fht_ln_backward(_ptr(g), _ptr(x), _dtype_code(x), M, K, _ptr(g_x), _stream(stream)),
           "hbl_fht_ln_backward")
    return g_x


def hbl_kv_quant(x, bits: int, codes=None, scales=None, stream=None):
    """Post-RoPE head vectors x [rows][D] -> (unsigned codes uint8 [rows][D], gamma float32 [rows])."""
    torch = _torch()
    _need_cuda(x)
    rows, D = x.shape
    if codes is None:
        codes = _new(stream, (rows, D), torch.uint8, x)
    if scales is None:
        scales = _new(stream, (rows,), torch.float32, x)
    _check(lib().hbl_kv_quant(_ptr(x), _dtype_code(x), rows, D, bits, _ptr(codes), _ptr(scales), _stream(stream)),
           "hbl_kv_quant")
    return codes, scales


def hbl_fht(x, t=None, stream=None):
    """t = H_K x / sqrt(K) per row (the transform alone), float32 [M][K]."""
    torch = _torch()
    _need_cuda(x)
    M, K = x.shape
    if t is None:
        t = _new(stream, (M, K), torch.float32, x)
    _check(lib().hbl_fht(_ptr(x), _dtype_code(x), M, K, _ptr(t), _stream(stream)), "hbl_fht")
    return t


def hbl_pack_ternary_rotated_workspace_bytes(K: int, N: int) -> int:
    return int(lib().hbl_pack_ternary_rotated_workspace_bytes(K, N))


def hbl_pack_ternary_rotated(W, packed=None, alpha=None, workspace=None, stream=None):
    """Ternarise W H_K/sqrt(K) (weights rotated like the activations): (packed, alpha)."""
    torch = _torch()
    _need_cuda(W)
    N, K = W.shape
    if packed is None:
        packed = _new(stream, (N, K // 4), torch.uint8, W)
    if alpha is None:
        alpha = _new(stream, (1,), torch.float32, W)
    if workspace is None:
        workspace = _new(stream, (hbl_pack_ternary_rotated_workspace_bytes(K, N),), torch.uint8, W, scratch=True)
    _check(lib().hbl_pack_ternary_rotated(_ptr(W), _dtype_code(W), K, N, _ptr(packed), _ptr(alpha),
                                          _ptr(workspace), workspace.numel(), _stream(stream)),
           "hbl_pack_ternary_rotated")
    return packed, alpha


def hbl_norm_quant(x, bits: int, norm: int = HBL_NORM_LAYER, codes=None, scales=None, stream=None):
    """BitLinear activation path without the transform: LN or RMSNorm, then INT4/INT8 codes."""
    torch = _torch()
    _need_cuda(x)
    M, K = x.shape
    if codes is None:
        codes = _new(stream, (M, K // 2), torch.uint8, x) if bits == 4 else _new(stream, (M, K), torch.int8, x)
    if scales is None:
        scales = _new(stream, (M,), torch.float32, x)
    _check(lib().hbl_norm_quant(_ptr(x), _dtype_code(x), M, K, int(norm), bits, _ptr(codes), _ptr(scales),
                                _stream(stream)), "hbl_norm_quant")
    return codes, scales


def hbl_debug_norm(x, norm: int = HBL_NORM_LAYER, t=None, stream=None):
    torch = _torch()
    _need_cuda(x)
    M, K = x.shape
    if t is None:
        t = _new(stream, (M, K), torch.float32, x)
    _check(lib().hbl_debug_norm(_ptr(x), _dtype_code(x), M, K, int(norm), _ptr(t), _stream(stream)),
           "hbl_debug_norm")
    return t


def hbl_forward_noalloc(x, packed, alpha, N: int, bits: int, y=None, y_dtype=None, stream=None):
    """hbl_forward without a workspace, for callers that cannot allocate device memory: the library's
    fixed 32 MiB area is used instead (shapes needing more are rejected; concurrent calls race on it)."""
    _need_cuda(x, packed, alpha)
    M, K = x.shape
    if y is None:
        y = _new(stream, (M, N), y_dtype or x.dtype, x)
    _check(lib().hbl_forward_noalloc(_ptr(x), _dtype_code(x), M, K, _ptr(packed), _ptr(alpha), N, bits, _ptr(y),
                                     _dtype_code(y), _stream(stream)), "hbl_forward_noalloc")
    return y


def hbl_fht_quant_i8(x, bits: int, codes=None, scales=None, stream=None):
    """x [M][K] -> (int8 codes [M][K], one per byte, scales float32 [M])."""
    torch = _torch()
    _need_cuda(x)
    M, K = x.shape
    if codes is None:
        codes = _new(stream, (M, K), torch.int8, x)
    if scales is None:
        scales = _new(stream, (M,), torch.float32, x)
    _check(lib().hbl_fht_quant_i8(_ptr(x), _dtype_code(x), M, K, bits, _ptr(codes), _ptr(scales),
                                  _stream(stream)), "hbl_fht_quant_i8")
    return codes, scales


def hbl_widen_ternary(packed, K: int, w=None, stream=None):
    """Packed ternary [N][K/4] -> int8 codes [N][K]."""
    torch = _torch()
    _need_cuda(packed)
    N = packed.shape[0]
    if w is None:
        w = _new(stream, (N, K), torch.int8, packed)
    _check(lib().hbl_widen_ternary(_ptr(packed), K, N, _ptr(w), _stream(stream)), "hbl_widen_ternary")
    return w


def hbl_gemm_tern_dequant(codes, packed, scales, alpha, y=None, y_dtype=None, stream=None):
    """Packed INT4 codes [M][K/2] (uint8), packed ternary [N][K/4] ->
    y = (q w^T) * (scales[m] * alpha) [M][N] (M >= 256)."""
    torch = _torch()
    _need_cuda(codes, packed, scales, alpha)
    M, K = codes.shape[0], codes.shape[1] * 2
    N = packed.shape[0]
    if y is None:
        y = _new(stream, (M, N), y_dtype or torch.bfloat16, codes)
    _check(lib().hbl_gemm_tern_dequant(_ptr(codes), _ptr(packed), M, N, K, _ptr(scales), _ptr(alpha), _ptr(y),
                                       _dtype_code(y), _stream(stream)), "hbl_gemm_tern_dequant")
    return y


def hbl_gemm_dequant(A, w, scales, alpha, y=None, y_dtype=None, stream=None):
    """int8 A [M][K], int8 w [N][K] -> y = (A w^T) * (scales[m] * alpha) [M][N]."""
    torch = _torch()
    _need_cuda(A, w, scales, alpha)
    M, K = A.shape
    N = w.shape[0]
    if y is None:
        y = _new(stream, (M, N), y_dtype or torch.bfloat16, A)
    _check(lib().hbl_gemm_dequant(_ptr(A), _ptr(w), M, N, K, _ptr(scales), _ptr(alpha), _ptr(y), _dtype_code(y),
                                  _stream(stream)), "hbl_gemm_dequant")
    return y


def hbl_gemv_ternary_dequant(A, packed, scales, alpha, y=None, y_dtype=None, stream=None):
    """int8 A [M][K], packed ternary [N][K/4] -> y = (A w^T) * (scales[m] * alpha) [M][N]
    (decode-sized M: M <= 4, M * K <= 65536)."""
    torch = _torch()
    _need_cuda(A, packed, scales, alpha)
    M, K = A.shape
    N = packed.shape[0]
    if y is None:
        y = _new(stream, (M, N), y_dtype or torch.bfloat16, A)
    _check(lib().hbl_gemv_ternary_dequant(_ptr(A), _ptr(packed), M, N, K, _ptr(scales), _ptr(alpha), _ptr(y),
                                          _dtype_code(y), _stream(stream)), "hbl_gemv_ternary_dequant")
    return y


# ------------------------------------------------------------------ the paged 8-bit cache

# The calls below are made once per layer and token step, so their checks are few attribute reads per tensor.

def _here(t) -> int:
    """The device of t, which must be the current one (the kernels run there and take raw pointers)."""
    dev = t.get_device()
    if dev < 0 or dev != _torch().cuda.current_device():
        raise ValueError("tensors must be on the current CUDA device, got %s" % t.device)
    return dev


def _raw_stream(stream, dev: int) -> int:
    torch = _torch()
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _demand(dev: int, *wanted):
    """Each (name, tensor, dtype, shape) is contiguous, on device dev, of that dtype (None: any) and shape."""
    for name, t, dtype, shape in wanted:
        if t.get_device() != dev:
            raise ValueError("%s: expected a tensor on CUDA device %d, got %s" % (name, dev, t.device))
        if dtype is not None and t.dtype is not dtype:
            raise TypeError("%s: expected %s, got %s" % (name, dtype, t.dtype))
        if t.shape != shape:
            raise ValueError("%s: expected shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
        if not t.is_contiguous():
            raise ValueError("%s must be contiguous" % name)


def _demand_line(dev: int, dtype, *wanted):
    """Each (name, tensor, n): n contiguous values of the dtype on device dev (whatever their shape is called)."""
    for name, t, n in wanted:
        if t.numel() != n or t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
            raise (TypeError if t.dtype is not dtype else ValueError)(
                "%s: expected %d contiguous values of %s on CUDA device %d, got %s of %s on %s"
                % (name, n, dtype, dev, tuple(t.shape), t.dtype, t.device))


def _head_rows(name, t, dev: int) -> int:
    """Rows of heads [T][H][D], heads and values contiguous, any row stride (columns of a wider matrix): the stride."""
    if t.dim() != 3:
        raise ValueError("%s must be [rows][heads][head dimension]" % name)
    (T, H, D), (row, head, value) = t.shape, t.stride()
    if t.get_device() != dev:
        raise ValueError("%s: expected a tensor on CUDA device %d, got %s" % (name, dev, t.device))
    if (D > 1 and value != 1) or (H > 1 and head != D):
        raise ValueError("%s: heads and their values must be contiguous" % name)
    return row if T > 1 else H * D


def _cache_shape(dev: int, k_codes, k_scales, v_codes, v_scales):
    torch = _torch()
    if k_codes.dim() != 4:
        raise ValueError("k_codes must be [blocks][heads][block][head dimension]")
    shape = k_codes.shape
    n, H, block, D = shape
    _demand(dev, ("v_codes", v_codes, torch.uint8, shape))
    _demand_line(dev, torch.uint8, ("k_codes", k_codes, k_codes.numel()))
    _demand_line(dev, torch.float32, ("k_scales", k_scales, n * H), ("v_scales", v_scales, n * H))
    return n, H, block, D


def hbl_kv_plan(cached, added, free_blocks, taken, table, block: int, T: int, total=None, row_start=None, slots=None,
                positions=None, taken_out=None, stream=None):
    """One serving step's bookkeeping from int32 lengths cached, added [B]: writes the new entries of table
    [B][width] (blocks from free_blocks, from place taken[0] on) and returns (total [B], row_start [B + 1],
    slots [T], positions [T], taken_out [1]).  T, the rows of the batch, is at least the sum of added: a plan that cuts
    a request (total - cached sums to more than row_start[B]) is not for hbl_kv_append and hbl_kv_attention."""
    torch = _torch()
    dev, i32 = _here(table), torch.int32
    B, width = table.shape
    new = lambda n: _new(stream, (n,), i32, table)  # noqa: E731
    total = new(B) if total is None else total
    row_start = new(B + 1) if row_start is None else row_start
    slots = new(T) if slots is None else slots
    positions = new(T) if positions is None else positions
    taken_out = new(1) if taken_out is None else taken_out
    free = free_blocks.numel()
    _demand_line(dev, i32, ("table", table, B * width), ("cached", cached, B), ("added", added, B),
                 ("free_blocks", free_blocks, free), ("taken", taken, 1), ("total", total, B), ("row_start", row_start, B + 1),
                 ("slots", slots, T), ("positions", positions, T), ("taken_out", taken_out, 1))
    _check(lib().hbl_kv_plan(cached.data_ptr(), added.data_ptr(), B, block, free_blocks.data_ptr(), free,
                             taken.data_ptr(), table.data_ptr(), width, T, total.data_ptr(), row_start.data_ptr(),
                             slots.data_ptr(), positions.data_ptr(), taken_out.data_ptr(), _raw_stream(stream, dev)),
           "hbl_kv_plan")
    return total, row_start, slots, positions, taken_out


def hbl_kv_append(k, v, slots, k_codes, k_scales, v_codes, v_scales, bits: int = 8, stream=None):
    """Writes rows k, v [T][H][D] (float32/bf16; columns of a wider matrix are fine) into the cache at int32 slots [T]:
    codes uint8 [blocks][H][block][D], scales float32 [blocks][H], both in place.  Returns the four.  Rows of one block
    are neighbours with consecutive slots (hbl_kv_plan's are); rows with a slot outside the cache are passed over."""
    dev = _here(k_codes)
    n, H, block, D = _cache_shape(dev, k_codes, k_scales, v_codes, v_scales)
    ks, vs = _head_rows("k", k, dev), _head_rows("v", v, dev)
    T = k.shape[0]
    if k.shape != (T, H, D) or v.shape != (T, H, D):
        raise ValueError("k and v: expected shape %s, got %s and %s" % ((T, H, D), tuple(k.shape), tuple(v.shape)))
    if v.dtype is not k.dtype:
        raise TypeError("k and v must have one dtype, got %s and %s" % (k.dtype, v.dtype))
    _demand_line(dev, _torch().int32, ("slots", slots, T))
    _check(lib().hbl_kv_append(k.data_ptr(), v.data_ptr(), _dtype_code(k), T, H, D, ks, vs, slots.data_ptr(), bits, n,
                               block, k_codes.data_ptr(), k_scales.data_ptr(), v_codes.data_ptr(), v_scales.data_ptr(),
                               _raw_stream(stream, dev)), "hbl_kv_append")
    return k_codes, k_scales, v_codes, v_scales


def hbl_kv_attention_workspace_bytes(T: int, Hq: int, Hkv: int, D: int, B: int) -> int:
    return int(lib().hbl_kv_attention_workspace_bytes(T, Hq, Hkv, D, B))


def hbl_kv_attention(q, row_start, total, table, k_codes, k_scales, v_codes, v_scales, bits: int = 8, scale=None, o=None,
                     o_dtype=None, workspace=None, stream=None):
    """Causal attention of rows q [T][Hq][D] (columns of a wider matrix are fine) over the cache that holds them:
    row_start [B + 1], total [B] and table [B][width] as hbl_kv_plan gives them; scale a device float32 [1] or None
    for 1/sqrt(D).  Returns o [T][Hq][D] (q's dtype unless o_dtype), rows outside the requests left as they were
    (zero in an o made here)."""
    torch = _torch()
    dev, i32 = _here(q), torch.int32
    n, Hkv, block, D = _cache_shape(dev, k_codes, k_scales, v_codes, v_scales)
    qs = _head_rows("q", q, dev)
    T, Hq, Dq = q.shape
    if Dq != D:
        raise ValueError("q has head dimension %d, the cache %d" % (Dq, D))
    B, width = table.shape
    if o is None:
        o = _new(stream, (T, Hq, D), o_dtype or q.dtype, q, zero=True)
    if workspace is None:
        workspace = _new(stream, (hbl_kv_attention_workspace_bytes(T, Hq, Hkv, D, B),), torch.uint8, q, scratch=True)
    _demand_line(dev, i32, ("row_start", row_start, B + 1), ("total", total, B), ("table", table, B * width))
    _demand_line(dev, workspace.dtype, ("workspace", workspace, workspace.numel()))
    _demand(dev, ("o", o, None, (T, Hq, D)))
    if scale is not None:
        _demand_line(dev, torch.float32, ("scale", scale, 1))
    _check(lib().hbl_kv_attention(q.data_ptr(), _dtype_code(q), T, qs, Hq, Hkv, D, row_start.data_ptr(), total.data_ptr(),
                                  B, table.data_ptr(), width, n, block, bits, k_codes.data_ptr(), k_scales.data_ptr(),
                                  v_codes.data_ptr(), v_scales.data_ptr(), None if scale is None else scale.data_ptr(),
                                  o.data_ptr(), _dtype_code(o), workspace.data_ptr(), workspace.nbytes,
                                  _raw_stream(stream, dev)), "hbl_kv_attention")
    return o


# ------------------------------------------------------------------ residual, RMSNorm and quantizer

def _opt(t):
    return None if t is None else t.data_ptr()


def hbl_add_rms_quant(x, bits: int, residual=None, gain=None, h=None, codes=None, scales=None, stream=None):
    """h = x + residual, then RMSNorm with a float32 gain [K] and the per-token quantizer (bits 8 absmax, 4 absmean):
    (h [M][K] of x's dtype, int8 codes [M][K], float32 scales [M]).  h may be x or residual itself."""
    torch = _torch()
    dev, dtype = _here(x), x.dtype
    M, K = x.shape
    if h is None:
        h = _new(stream, (M, K), dtype, x)
    if codes is None:
        codes = _new(stream, (M, K), torch.int8, x)
    if scales is None:
        scales = _new(stream, (M,), torch.float32, x)
    n = M * K
    _demand_line(dev, dtype, ("x", x, n), ("h", h, n))
    _demand_line(dev, torch.int8, ("codes", codes, n))
    _demand_line(dev, torch.float32, ("scales", scales, M))
    if residual is not None:
        _demand_line(dev, dtype, ("residual", residual, n))
    if gain is not None:
        _demand_line(dev, torch.float32, ("gain", gain, K))
    _check(lib().hbl_add_rms_quant(x.data_ptr(), _opt(residual), _dtype_code(x), M, K, _opt(gain), bits, h.data_ptr(),
                                   codes.data_ptr(), scales.data_ptr(), _raw_stream(stream, dev)), "hbl_add_rms_quant")
    return h, codes, scales


def hbl_add_rms_quant_backward_workspace_bytes(M: int, K: int) -> int:
    return int(lib().hbl_add_rms_quant_backward_workspace_bytes(M, K))


def hbl_add_rms_quant_backward(h, g_t, gain=None, g_h=None, g_x=None, g_gain=None, workspace=None, stream=None):
    """Straight-through gradient of hbl_add_rms_quant at its output h: g_t [M][K] of the normalised value, g_h [M][K]
    (h's dtype) along the residual stream.  Returns (g_x [M][K] of h's dtype, for x and residual alike; g_gain
    float32 [K], None without a gain)."""
    torch = _torch()
    dev, dtype, f32 = _here(h), h.dtype, torch.float32
    M, K = h.shape
    if g_x is None:
        g_x = _new(stream, (M, K), dtype, h)
    if g_gain is None and gain is not None:
        g_gain = _new(stream, (K,), f32, h)
    if workspace is None:
        workspace = _new(stream, (hbl_add_rms_quant_backward_workspace_bytes(M, K),), torch.uint8, h, scratch=True)
    n = M * K
    _demand_line(dev, dtype, ("h", h, n), ("g_x", g_x, n))
    _demand_line(dev, g_t.dtype, ("g_t", g_t, n))
    _demand_line(dev, workspace.dtype, ("workspace", workspace, workspace.numel()))
    if g_h is not None:
        _demand_line(dev, dtype, ("g_h", g_h, n))
    for name, t in (("gain", gain), ("g_gain", g_gain)):
        if t is not None:
            _demand_line(dev, f32, (name, t, K))
    _check(lib().hbl_add_rms_quant_backward(h.data_ptr(), _dtype_code(h), M, K, _opt(gain), g_t.data_ptr(),
                                            _dtype_code(g_t), _opt(g_h), g_x.data_ptr(), _opt(g_gain),
                                            workspace.data_ptr(), workspace.nbytes, _raw_stream(stream, dev)),
           "hbl_add_rms_quant_backward")
    return g_x, g_gain


def hbl_debug_ln_fht(x, t=None, stream=None):
    torch = _torch()
    _need_cuda(x)
    M, K = x.shape
    if t is None:
        t = _new(stream, (M, K), torch.float32, x)
    _check(lib().hbl_debug_ln_fht(_ptr(x), _dtype_code(x), M, K, _ptr(t), _stream(stream)), "hbl_debug_ln_fht")
    return t


def hbl_quant_from_f32(t, bits: int, codes=None, scales=None, stream=None):
    torch = _torch()
    _need_cuda(t)
    M, K = t.shape
    if codes is None:
        codes = _new(stream, (M, K // 2), torch.uint8, t) if bits == 4 else _new(stream, (M, K), torch.int8, t)
    if scales is None:
        scales = _new(stream, (M,), torch.float32, t)
    _check(lib().hbl_quant_from_f32(_ptr(t), M, K, bits, _ptr(codes), _ptr(scales), _stream(stream)),
           "hbl_quant_from_f32")
    return codes, scales


def hbl_gemm_i8_i32(A, B, acc=None, stream=None):
    torch = _torch()
    _need_cuda(A, B)
    M, K = A.shape
    N = B.shape[0]
    if acc is None:
        acc = _new(stream, (M, N), torch.int32, A)
    _check(lib().hbl_gemm_i8_i32(_ptr(A), _ptr(B), M, N, K, _ptr(acc), _stream(stream)), "hbl_gemm_i8_i32")
    return acc


def hbl_last_device_error(stream=None) -> int:
    return int(lib().hbl_last_device_error(_stream(stream)))


def hbl_debug_raise_device_error(stream=None):
    _check(lib().hbl_debug_raise_device_error(_stream(stream)), "hbl_debug_raise_device_error")


def hbl_debug_set_wait_limit_ns(ns: int):
    """Limit of the kernels' pipeline waits on the current device (0: 2 s)."""
    _check(lib().hbl_debug_set_wait_limit_ns(int(ns)), "hbl_debug_set_wait_limit_ns")
