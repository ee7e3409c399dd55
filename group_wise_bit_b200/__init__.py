"""Python binding of the group-wise low-bit linear-layer library (libgwb.so).

Argument marshalling only: every function below checks dtypes, shapes,
devices and contiguity of torch CUDA tensors, allocates outputs that were not
given, and calls the C entry point of the same name (see include/gwb.h) on
torch's current CUDA stream.  All computation happens in the library's CUDA
kernels; there is no CPU fallback.  Errors from the library raise GwbError.

Packed uint32 words may be held in torch.int32 or torch.uint32 tensors (the
bits are what matters); bf16 / fp16 tensors are passed as such.
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libgwb.so")

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_INT = ctypes.c_int
_F32 = ctypes.c_float
_F64 = ctypes.c_double

# name -> argument types (all return int gwb_status)
SIGNATURES = {
    "gwb_qpack_affine": [_P, _I64, _I64, _INT, _INT, _P, _P, _P, _P],
    "gwb_dequant_affine": [_P, _P, _P, _I64, _I64, _INT, _INT, _P, _P],
    "gwb_qmm_affine": [_P, _I64, _P, _P, _P, _I64, _I64, _INT, _INT, _P, _P],
    "gwb_qmm_affine_noalloc": [_P, _I64, _P, _P, _P, _I64, _I64, _INT, _INT, _P, _P],
    "gwb_gptq_dequant": [_P, _P, _P, _P, _I64, _I64, _INT, _P, _P],
    "gwb_gptq_qmm": [_P, _I64, _P, _P, _P, _P, _I64, _I64, _INT, _P, _P],
    "gwb_gemv_gate_up": [_P, _I64, _P, _P, _P, _P, _P, _P, _I64, _I64, _INT, _INT, _P, _P, _P],
    "gwb_gemv_silu_gate": [_P, _P, _I64, _P, _P, _P, _I64, _I64, _INT, _INT, _P, _P],
    "gwb_gemv_silu_gate_resid": [_P, _P, _I64, _P, _P, _P, _I64, _I64, _INT, _INT, _P, _P, _P],
    "gwb_awq_dequant": [_P, _P, _P, _I64, _I64, _INT, _P, _P],
    "gwb_awq_qmm": [_P, _I64, _P, _P, _P, _I64, _I64, _INT, _P, _P],
    "gwb_quant_per_token_i8": [_P, _I64, _I64, _P, _P, _P],
    "gwb_qpack_sym_i4": [_P, _I64, _I64, _P, _P, _P],
    "gwb_gemm_i8i4": [_P, _P, _I64, _P, _P, _I64, _I64, _P, _P, _P],
    "gwb_gemv_w4a8": [_P, _I64, _P, _P, _I64, _I64, _P, _P],
    "gwb_qpack_sym_i8": [_P, _I64, _I64, _P, _P, _P],
    "gwb_gemm_i8i8": [_P, _P, _I64, _P, _P, _I64, _I64, _P, _P, _P],
    "gwb_rmsnorm_quant_i8": [_P, _P, _P, _I64, _I64, _F64, _INT, _P, _P, _P, _P],
    "gwb_dequant_per_token_i8": [_P, _P, _I64, _I64, _INT, _P, _P],
    "gwb_kv_block_bytes": [_I64, _INT, _INT, _INT, _P],
    "gwb_kv_write": [_P, _I64, _P, _I64, _P, _I64, _INT, _P, _I64, _I64, _I64, _INT, _INT, _INT, _P],
    "gwb_kv_read": [_P, _I64, _I64, _I64, _INT, _INT, _INT, _P, _I64, _INT, _P, _P, _P],
    "gwb_attn_decode_workspace": [_I64, _I64, _INT, _I64, _I64, _P],
    "gwb_attn_decode": [_P, _I64, _I64, _I64, _INT, _P, _I64, _I64, _I64, _INT, _INT, _INT, _P, _I64, _I64, _P, _F32,
                        _P, _P, _P, _I64, _P],
    "gwb_check_device_error": [_P],
    "gwb_debug_set_wait_cycles": [ctypes.c_ulonglong],
    "gwb_debug_inject_stream_k_stall": [_INT],
}

STATUS = {0: "OK", 1: "INVALID_ARG", 2: "SHAPE", 3: "UNSUPPORTED", 4: "ALIGN", 5: "CUDA", 6: "TIMEOUT"}


class GwbError(RuntimeError):
    def __init__(self, fn, status, msg):
        super().__init__(f"{fn}: {STATUS.get(status, status)}: {msg}")
        self.status = status


_lib = None


def lib() -> ctypes.CDLL:
    """Loads libgwb.so (built in-tree by `python -m group_wise_bit_b200.build`)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with `python -m group_wise_bit_b200.build`")
        l = ctypes.CDLL(LIB_PATH)
        for name, args in SIGNATURES.items():
            fn = getattr(l, name)
            fn.argtypes = args
            fn.restype = _INT
        l.gwb_last_error.restype = ctypes.c_char_p
        l.gwb_last_error.argtypes = []
        l.gwb_version.restype = ctypes.c_char_p
        l.gwb_version.argtypes = []
        _lib = l
    return _lib


def version() -> str:
    return lib().gwb_version().decode()


_fns = {}


def _call(name, *args):
    fn = _fns.get(name)
    if fn is None:
        fn = _fns[name] = getattr(lib(), name)
    st = fn(*args)
    if st != 0:
        raise GwbError(name, st, lib().gwb_last_error().decode())


try:   # the raw handle of the current stream, without building a Stream object per call
    _raw_stream = torch._C._cuda_getCurrentRawStream

    def _stream():
        return _raw_stream(torch.cuda.current_device())
except AttributeError:   # pragma: no cover - older torch
    def _raw_stream(device):
        return torch.cuda.current_stream(device).cuda_stream

    def _stream():
        return torch.cuda.current_stream().cuda_stream


def _ptr(t):
    return None if t is None else t.data_ptr()


def _dev(t, name, dtypes, shape=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)} != {tuple(shape)}")
    return t


_WORDS = (torch.int32, torch.uint32)


def _out(t, name, shape, dtype, device, dtypes=None):
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    return _dev(t, name, dtypes or (dtype,), shape)


# ------------------------------------------------------------------ MLX affine
def qpack_affine(w, bits, group_size, wq=None, scales=None, biases=None):
    """w fp32 [N, K] -> (wq int32 [N, K*bits/32], scales bf16 [N, K/gs], biases bf16 [N, K/gs])."""
    _dev(w, "w", (torch.float32,))
    N, K = w.shape
    wq = _out(wq, "wq", (N, K * bits // 32), torch.int32, w.device, _WORDS)
    scales = _out(scales, "scales", (N, K // group_size), torch.bfloat16, w.device)
    biases = _out(biases, "biases", (N, K // group_size), torch.bfloat16, w.device)
    _call("gwb_qpack_affine", _ptr(w), N, K, bits, group_size, _ptr(wq), _ptr(scales), _ptr(biases), _stream())
    return wq, scales, biases


def dequant_affine(wq, scales, biases, K, bits, group_size, out=None):
    """-> bf16 [N, K] with w = bf16(fp32(code*scale + bias))."""
    _dev(wq, "wq", _WORDS)
    N = wq.shape[0]
    _dev(wq, "wq", _WORDS, (N, K * bits // 32))
    _dev(scales, "scales", (torch.bfloat16,), (N, K // group_size))
    _dev(biases, "biases", (torch.bfloat16,), (N, K // group_size))
    out = _out(out, "out", (N, K), torch.bfloat16, wq.device)
    _call("gwb_dequant_affine", _ptr(wq), _ptr(scales), _ptr(biases), N, K, bits, group_size, _ptr(out), _stream())
    return out


def _affine_check(wq, scales, biases, bits, group_size):
    """(N, K) of a weight in the MLX affine layout, its three tensors checked."""
    _dev(wq, "wq", _WORDS)
    N, K = wq.shape[0], wq.shape[1] * 32 // bits
    _dev(scales, "scales", (torch.bfloat16,), (N, K // group_size))
    _dev(biases, "biases", (torch.bfloat16,), (N, K // group_size))
    return N, K


def qmm_affine(x, wq, scales, biases, bits, group_size, y=None):
    """y bf16 [M, N] = x bf16 [M, K] . W^T with W in the MLX affine layout."""
    _dev(x, "x", (torch.bfloat16,))
    M, K = x.shape
    N = wq.shape[0]
    _dev(wq, "wq", _WORDS, (N, K * bits // 32))
    _dev(scales, "scales", (torch.bfloat16,), (N, K // group_size))
    _dev(biases, "biases", (torch.bfloat16,), (N, K // group_size))
    y = _out(y, "y", (M, N), torch.bfloat16, x.device)
    _call("gwb_qmm_affine", _ptr(x), M, _ptr(wq), _ptr(scales), _ptr(biases), N, K, bits, group_size, _ptr(y),
          _stream())
    return y


def qmm_affine_noalloc(x, wq, scales, biases, bits, group_size, y=None):
    """As qmm_affine for M > 128, with the GEMM's scratch in the library's fixed
    device array instead of device memory it allocates (see gwb.h)."""
    _dev(x, "x", (torch.bfloat16,))
    M, K = x.shape
    N = wq.shape[0]
    _dev(wq, "wq", _WORDS, (N, K * bits // 32))
    _dev(scales, "scales", (torch.bfloat16,), (N, K // group_size))
    _dev(biases, "biases", (torch.bfloat16,), (N, K // group_size))
    y = _out(y, "y", (M, N), torch.bfloat16, x.device)
    _call("gwb_qmm_affine_noalloc", _ptr(x), M, _ptr(wq), _ptr(scales), _ptr(biases), N, K, bits, group_size,
          _ptr(y), _stream())
    return y


# ------------------------------------------------------------------ GPTQ
def _gptq_check(qweight, scales, qzeros, g_idx, group_size):
    _dev(qweight, "qweight", _WORDS)
    K8, N = qweight.shape
    K = K8 * 8
    _dev(scales, "scales", (torch.float16,), (K // group_size, N))
    _dev(qzeros, "qzeros", _WORDS, (K // group_size, N // 8))
    if g_idx is not None:
        _dev(g_idx, "g_idx", (torch.int32,), (K,))
    return K, N


def gptq_dequant(qweight, scales, qzeros, g_idx, group_size, out=None):
    """-> fp16 [N, K] (out-features major)."""
    K, N = _gptq_check(qweight, scales, qzeros, g_idx, group_size)
    out = _out(out, "out", (N, K), torch.float16, qweight.device)
    _call("gwb_gptq_dequant", _ptr(qweight), _ptr(scales), _ptr(qzeros), _ptr(g_idx), K, N, group_size, _ptr(out),
          _stream())
    return out


def gptq_qmm(x, qweight, scales, qzeros, g_idx, group_size, y=None):
    """y fp16 [M, N] = x fp16 [M, K] . W^T with W in the GPTQ layout."""
    K, N = _gptq_check(qweight, scales, qzeros, g_idx, group_size)
    _dev(x, "x", (torch.float16,))
    M = x.shape[0]
    _dev(x, "x", (torch.float16,), (M, K))
    y = _out(y, "y", (M, N), torch.float16, x.device)
    _call("gwb_gptq_qmm", _ptr(x), M, _ptr(qweight), _ptr(scales), _ptr(qzeros), _ptr(g_idx), K, N, group_size,
          _ptr(y), _stream())
    return y


# ------------------------------------------------------------------ fused decode products
def gemv_gate_up(x, gate_w, up_w, bits, group_size, y_gate=None, y_up=None):
    """(x W_gate^T, x W_up^T) in one launch; gate_w / up_w = (wq, scales, biases) of one shape."""
    wq, sc, bi = gate_w
    wq2, sc2, bi2 = up_w
    N, K = _affine_check(wq, sc, bi, bits, group_size)
    if _affine_check(wq2, sc2, bi2, bits, group_size) != (N, K):
        raise ValueError("gate and up weights differ in shape")
    _dev(x, "x", (torch.bfloat16,), (x.shape[0], K))
    M = x.shape[0]
    y_gate = _out(y_gate, "y_gate", (M, N), torch.bfloat16, x.device)
    y_up = _out(y_up, "y_up", (M, N), torch.bfloat16, x.device)
    _call("gwb_gemv_gate_up", _ptr(x), M, _ptr(wq), _ptr(sc), _ptr(bi), _ptr(wq2), _ptr(sc2), _ptr(bi2), N, K,
          bits, group_size, _ptr(y_gate), _ptr(y_up), _stream())
    return y_gate, y_up


def gemv_silu_gate(gate, up, wq, scales, biases, bits, group_size, x_resid=None, y=None):
    """y = (x_resid +) (silu(gate) * up) W^T; gate, up bf16 [M, K], x_resid bf16 [M, N]."""
    N, K = _affine_check(wq, scales, biases, bits, group_size)
    _dev(gate, "gate", (torch.bfloat16,), (gate.shape[0], K))
    M = gate.shape[0]
    _dev(up, "up", (torch.bfloat16,), (M, K))
    y = _out(y, "y", (M, N), torch.bfloat16, gate.device)
    if x_resid is None:
        _call("gwb_gemv_silu_gate", _ptr(gate), _ptr(up), M, _ptr(wq), _ptr(scales), _ptr(biases), N, K, bits,
              group_size, _ptr(y), _stream())
    else:
        _dev(x_resid, "x_resid", (torch.bfloat16,), (M, N))
        _call("gwb_gemv_silu_gate_resid", _ptr(gate), _ptr(up), M, _ptr(wq), _ptr(scales), _ptr(biases), N, K,
              bits, group_size, _ptr(x_resid), _ptr(y), _stream())
    return y


# ------------------------------------------------------------------ AWQ
def awq_dequant(qweight, scales, qzeros, group_size, out=None):
    """-> fp16 [N, K]: the GPTQ layout with the stored zero used as is (no "+1", no g_idx)."""
    K, N = _gptq_check(qweight, scales, qzeros, None, group_size)
    out = _out(out, "out", (N, K), torch.float16, qweight.device)
    _call("gwb_awq_dequant", _ptr(qweight), _ptr(scales), _ptr(qzeros), K, N, group_size, _ptr(out), _stream())
    return out


def awq_qmm(x, qweight, scales, qzeros, group_size, y=None):
    """y fp16 [M, N] = x fp16 [M, K] . W^T with W as awq_dequant defines it."""
    K, N = _gptq_check(qweight, scales, qzeros, None, group_size)
    _dev(x, "x", (torch.float16,), (x.shape[0], K))
    M = x.shape[0]
    y = _out(y, "y", (M, N), torch.float16, x.device)
    _call("gwb_awq_qmm", _ptr(x), M, _ptr(qweight), _ptr(scales), _ptr(qzeros), K, N, group_size, _ptr(y),
          _stream())
    return y


# ------------------------------------------------------------------ W4A8
def quant_per_token_i8(x, qx=None, sx=None):
    """x bf16 [M, K] -> (qx int8 [M, K], sx fp32 [M])."""
    _dev(x, "x", (torch.bfloat16,))
    M, K = x.shape
    qx = _out(qx, "qx", (M, K), torch.int8, x.device)
    sx = _out(sx, "sx", (M,), torch.float32, x.device)
    _call("gwb_quant_per_token_i8", _ptr(x), M, K, _ptr(qx), _ptr(sx), _stream())
    return qx, sx


def qpack_sym_i4(w, wq=None, sw=None):
    """w fp32 [N, K] -> (wq int32 [N, K/8] of two's-complement nibbles, sw fp32 [N])."""
    _dev(w, "w", (torch.float32,))
    N, K = w.shape
    wq = _out(wq, "wq", (N, K // 8), torch.int32, w.device, _WORDS)
    sw = _out(sw, "sw", (N,), torch.float32, w.device)
    _call("gwb_qpack_sym_i4", _ptr(w), N, K, _ptr(wq), _ptr(sw), _stream())
    return wq, sw


def gemm_i8i4(qx, sx, wq, sw, want_y=True, want_acc=False, y=None, acc=None):
    """-> (y bf16 [M, N] or None, acc int32 [M, N] or None)."""
    _dev(qx, "qx", (torch.int8,))
    M, K = qx.shape
    N = wq.shape[0]
    _dev(sx, "sx", (torch.float32,), (M,))
    _dev(wq, "wq", _WORDS, (N, K // 8))
    _dev(sw, "sw", (torch.float32,), (N,))
    if want_y or y is not None:
        y = _out(y, "y", (M, N), torch.bfloat16, qx.device)
    if want_acc or acc is not None:
        acc = _out(acc, "acc", (M, N), torch.int32, qx.device)
    _call("gwb_gemm_i8i4", _ptr(qx), _ptr(sx), M, _ptr(wq), _ptr(sw), N, K, _ptr(y), _ptr(acc), _stream())
    return y, acc


def gemv_w4a8(x, wq, sw, y=None):
    """y bf16 [M, N] = W4A8 product of x bf16 [M, K] (quantized per token inside the kernel, M <= 8)
    and the int4 weights (wq, sw) of qpack_sym_i4; bit-identical to quant_per_token_i8 + gemm_i8i4."""
    _dev(x, "x", (torch.bfloat16,))
    M, K = x.shape
    N = wq.shape[0]
    _dev(wq, "wq", _WORDS, (N, K // 8))
    _dev(sw, "sw", (torch.float32,), (N,))
    y = _out(y, "y", (M, N), torch.bfloat16, x.device)
    _call("gwb_gemv_w4a8", _ptr(x), M, _ptr(wq), _ptr(sw), N, K, _ptr(y), _stream())
    return y


# ------------------------------------------------------------------ W8A8
def qpack_sym_i8(w, wq=None, sw=None):
    """w fp32 [N, K] -> (wq int8 [N, K], sw fp32 [N])."""
    _dev(w, "w", (torch.float32,))
    N, K = w.shape
    wq = _out(wq, "wq", (N, K), torch.int8, w.device)
    sw = _out(sw, "sw", (N,), torch.float32, w.device)
    _call("gwb_qpack_sym_i8", _ptr(w), N, K, _ptr(wq), _ptr(sw), _stream())
    return wq, sw


def gemm_i8i8(qx, sx, wq, sw, want_y=True, want_acc=False, y=None, acc=None):
    """-> (y bf16 [M, N] or None, acc int32 [M, N] or None)."""
    _dev(qx, "qx", (torch.int8,))
    M, K = qx.shape
    N = wq.shape[0]
    _dev(sx, "sx", (torch.float32,), (M,))
    _dev(wq, "wq", (torch.int8,), (N, K))
    _dev(sw, "sw", (torch.float32,), (N,))
    if want_y or y is not None:
        y = _out(y, "y", (M, N), torch.bfloat16, qx.device)
    if want_acc or acc is not None:
        acc = _out(acc, "acc", (M, N), torch.int32, qx.device)
    _call("gwb_gemm_i8i8", _ptr(qx), _ptr(sx), M, _ptr(wq), _ptr(sw), N, K, _ptr(y), _ptr(acc), _stream())
    return y, acc


# ------------------------------------------------------------------ norm, quantized paged cache, decode attention
_HALF = {torch.bfloat16: 0, torch.float16: 1}   # gwb_dtype
_HALVES = tuple(_HALF)


def _stream_of(*tensors):
    """The current stream; all given tensors must lie on its device, the current one."""
    cur = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != cur:
            raise ValueError(f"a tensor is on {t.device}, the current device is cuda:{cur}")
    return _raw_stream(cur)


def _out_like(t, name, like, dtype):
    """_out for an output of like's shape (less host time than torch.empty)."""
    return torch.empty_like(like, dtype=dtype) if t is None else _dev(t, name, (dtype,), like.shape)


def _out_of(t, name, src, shape, dtype):
    """_out on src's device (less host time than torch.empty)."""
    return src.new_empty(shape, dtype=dtype) if t is None else _dev(t, name, (dtype,), shape)


def _token_rows(t, name, shape, dtypes):
    """Rows [T, heads, head_dim] whose heads are contiguous; returns the elements between tokens."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {dtypes}")
    if t.dim() != 3 or (shape is not None and t.shape != shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)} != {tuple(shape) if shape else '[tokens, heads, head_dim]'}")
    T, H, D = t.shape
    s = t.stride()
    if (D > 1 and s[2] != 1) or (H > 1 and s[1] != D):
        raise ValueError(f"{name}: the heads of a token must be contiguous (strides {s})")
    return s[0] if T > 1 else H * D


def rmsnorm_quant_i8(x, weight, eps, residual=None, residual_out=None, qx=None, sx=None):
    """RMS norm of x (+ residual) with a per-token int8 output: (qx int8 [M, K], sx fp32 [M], h or None).

    x, residual bf16 or fp16 [M, K], weight [K] of the same dtype; h = x + residual, rounded once, is
    written to residual_out (which may be x or residual).  qx and sx are what gemm_i8i8 / gemm_i8i4 take."""
    _dev(x, "x", _HALVES)
    M, K = x.shape
    dt = (x.dtype,)
    _dev(weight, "weight", dt, (K,))
    if residual is not None:
        _dev(residual, "residual", dt, (M, K))
        residual_out = _out_like(residual_out, "residual_out", x, x.dtype)
    elif residual_out is not None:
        raise ValueError("residual_out without residual: the sum would be x itself")
    qx = _out_like(qx, "qx", x, torch.int8)
    sx = _out_of(sx, "sx", x, (M,), torch.float32)
    stream = _stream_of(x, weight, residual, residual_out, qx, sx)
    _call("gwb_rmsnorm_quant_i8", _ptr(x), _ptr(residual), _ptr(weight), M, K, float(eps), _HALF[x.dtype],
          _ptr(residual_out), _ptr(qx), _ptr(sx), stream)
    return qx, sx, residual_out


def dequant_per_token_i8(qx, sx, dtype=torch.bfloat16, out=None):
    """The values qx int8 [M, K] with scales sx fp32 [M] stand for, as bf16 or fp16 [M, K]."""
    _dev(qx, "qx", (torch.int8,))
    M, K = qx.shape
    _dev(sx, "sx", (torch.float32,), (M,))
    if dtype not in _HALF:
        raise TypeError(f"dtype {dtype} not in {_HALVES}")
    out = _out_like(out, "out", qx, dtype)
    stream = _stream_of(qx, sx, out)
    _call("gwb_dequant_per_token_i8", _ptr(qx), _ptr(sx), M, K, _HALF[dtype], _ptr(out), stream)
    return out


_block_bytes = {}


def kv_block_bytes(page_size, head_dim, bits, group_size):
    """Bytes of one page of one head of a quantized cache."""
    key = (page_size, head_dim, bits, group_size)
    n = _block_bytes.get(key)
    if n is None:
        out = _I64(0)
        _call("gwb_kv_block_bytes", page_size, head_dim, bits, group_size, ctypes.byref(out))
        n = _block_bytes[key] = out.value
    return n


def kv_cache(num_pages, heads, head_dim, page_size, bits, group_size, device="cuda"):
    """An empty quantized paged cache: uint8 [num_pages, heads, block] (the block's layout: gwb.h).
    Its memory is zeroed, so that rows never written read back as zeros."""
    return torch.zeros(num_pages, heads, kv_block_bytes(page_size, head_dim, bits, group_size), dtype=torch.uint8,
                       device=device)


def _cache_check(cache, head_dim, bits, group_size):
    """(pages, heads, page_size) of a cache."""
    _dev(cache, "cache", (torch.uint8,))
    if cache.dim() != 3:
        raise ValueError(f"cache: shape {tuple(cache.shape)} != [pages, heads, block]")
    pages, heads, block = cache.shape
    granule = _block_bytes.get((16, head_dim, bits, group_size)) or kv_block_bytes(16, head_dim, bits, group_size)
    if block % granule != 0:
        raise ValueError(f"cache: a block of {block} bytes does not hold granules of {granule} bytes "
                         f"(head_dim {head_dim}, {bits} bits, group size {group_size})")
    return pages, heads, block // granule * 16


def kv_write(cache, slots, k, v, bits, group_size):
    """Quantizes k, v [T, heads, head_dim] (bf16 or fp16, any token stride) into the cache at slots
    (int64 [T], page * page_size + place; negative: the row is padding and left out)."""
    ks = _token_rows(k, "k", None, _HALVES)
    T, H, D = k.shape
    vs = _token_rows(v, "v", k.shape, (k.dtype,))
    pages, heads, page_size = _cache_check(cache, D, bits, group_size)
    if heads != H:
        raise ValueError(f"k has {H} heads, the cache {heads}")
    _dev(slots, "slots", (torch.int64,), (T,))
    stream = _stream_of(cache, slots, k, v)
    _call("gwb_kv_write", _ptr(k), ks, _ptr(v), vs, _ptr(slots), T, _HALF[k.dtype], _ptr(cache), pages, heads,
          page_size, D, bits, group_size, stream)
    return cache


def kv_read(cache, slots, head_dim, bits, group_size, dtype=torch.bfloat16, k=None, v=None):
    """The cache's rows at slots (int64 [T]) as dense k, v [T, heads, head_dim]; zeros for negative slots."""
    pages, heads, page_size = _cache_check(cache, head_dim, bits, group_size)
    if dtype not in _HALF:
        raise TypeError(f"dtype {dtype} not in {_HALVES}")
    _dev(slots, "slots", (torch.int64,))
    if slots.dim() != 1:
        raise ValueError(f"slots: shape {tuple(slots.shape)} != [tokens]")
    shape = (slots.shape[0], heads, head_dim)
    k = _out_of(k, "k", cache, shape, dtype)
    v = _out_like(v, "v", k, dtype)
    stream = _stream_of(cache, slots, k, v)
    _call("gwb_kv_read", _ptr(cache), pages, heads, page_size, head_dim, bits, group_size, _ptr(slots), shape[0],
          _HALF[dtype], _ptr(k), _ptr(v), stream)
    return k, v


_ws_bytes = {}


def attn_decode_workspace(q_heads, heads, head_dim, batch=0, max_tokens=0):
    """Bytes of attn_decode's workspace on the current device, for up to `batch` sequences whose page tables
    name max_tokens tokens (0: any); none where the tables are short."""
    key = (torch.cuda.current_device(), q_heads, heads, head_dim, batch, max_tokens)
    n = _ws_bytes.get(key)
    if n is None:
        out = _I64(0)
        _call("gwb_attn_decode_workspace", q_heads, heads, head_dim, batch, max_tokens, ctypes.byref(out))
        n = out.value
        if len(_ws_bytes) < 4096:
            _ws_bytes[key] = n
    return n


def attn_decode(q, cache, page_table, seq_lens, bits, group_size, scale=None, out=None, lse=None, workspace=None):
    """Attention of one new token a sequence over the quantized cache: [B, q_heads, head_dim] of q's dtype.

    q [B, q_heads, head_dim] (bf16 or fp16, any sequence stride), page_table int32 [B, max_pages] (rows may lie
    apart, not overlap), seq_lens int32 [B] (0: an empty row, zeros).  scale defaults to 1 / sqrt(head_dim).  lse, if
    given, is an fp32 [B, q_heads] output.  workspace: a uint8 tensor of attn_decode_workspace() bytes that
    no overlapping call uses; without one the call takes it from torch's allocator."""
    qs = _token_rows(q, "q", None, _HALVES)
    B, HQ, D = q.shape
    pages, heads, page_size = _cache_check(cache, D, bits, group_size)
    if not isinstance(page_table, torch.Tensor) or not page_table.is_cuda:
        raise ValueError("page_table must be a CUDA tensor (the library has no CPU path)")
    if page_table.dtype != torch.int32:
        raise TypeError(f"page_table: dtype {page_table.dtype} not in {(torch.int32,)}")
    if page_table.dim() != 2 or page_table.shape[0] != B:
        raise ValueError(f"page_table: shape {tuple(page_table.shape)} != [{B}, max_pages]")
    max_pages = page_table.shape[1]
    if max_pages > 1 and page_table.stride(1) != 1:
        raise ValueError("page_table: a row's page ids must be contiguous")
    ts = max(page_table.stride(0), max_pages) if B > 1 else max_pages
    if B > 1 and page_table.stride(0) < max_pages:
        raise ValueError("page_table: rows overlap")
    _dev(seq_lens, "seq_lens", (torch.int32,), (B,))
    out = _out_of(out, "out", q, (B, HQ, D), q.dtype)
    if lse is not None:
        _dev(lse, "lse", (torch.float32,), (B, HQ))
    if workspace is not None:
        _dev(workspace, "workspace", (torch.uint8,))
    stream = _stream_of(q, cache, page_table, seq_lens, out, lse, workspace)
    if workspace is not None:
        ws = workspace.numel()
    else:
        ws = attn_decode_workspace(HQ, heads, D, B, max_pages * page_size)
        if ws:
            workspace = cache.new_empty(ws)
    _call("gwb_attn_decode", _ptr(q), qs, B, HQ, _HALF[q.dtype], _ptr(cache), pages, heads, page_size, D, bits,
          group_size, _ptr(page_table), ts, max_pages, _ptr(seq_lens),
          float(1.0 / D ** 0.5 if scale is None else scale), _ptr(out), _ptr(lse), _ptr(workspace),
          ws, stream)
    return out


def check_device_error():
    """Synchronizes the current stream; raises GwbError(TIMEOUT) if a bounded device wait gave up, and
    GwbError(INVALID_ARG) if a slot, page id or length in device memory was out of range."""
    _call("gwb_check_device_error", _stream())


def debug_set_wait_cycles(cycles):
    """Failure-path testing: SM clock cycles after which device waits give up on the
    current device (0 restores the default, about 2 s)."""
    _call("gwb_debug_set_wait_cycles", int(cycles))


def debug_inject_stream_k_stall(armed=True):
    """Failure-path testing: the next stream-K launch of the persistent GEMM waits for
    partial tiles that nothing publishes, so its bounded waits run out (see gwb.h);
    armed=False disarms it."""
    _call("gwb_debug_inject_stream_k_stall", 1 if armed else 0)
