"""ctypes binding of ``libfp8q.so`` (the C ABI declared in ``include/fp8q.h``).

Argument marshalling only: every step runs in the HIP library.  torch provides device memory and the
current stream; outputs are allocated with torch when the caller does not pass them.  If the library
is not built, every call raises -- there is no fallback path.

Every call takes a ``stream`` (default: the current one) and launches there.  Ordering that stream behind the
inputs, and the readers of the outputs behind it, is the caller's; outputs and temporaries that the call allocates
are safe to drop at any time.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfp8q.so")

OUT_BF16 = 0
OUT_F32 = 1

_lock = threading.Lock()
_lib = None


def load_library(path: str = LIB_PATH):
    """Load libfp8q.so and declare the C signatures.  Raises if it has not been built."""
    global _lib
    if _lib is not None and path == LIB_PATH:
        return _lib
    with _lock:
        if _lib is not None and path == LIB_PATH:
            return _lib
        if not os.path.exists(path):
            raise RuntimeError(f"fp8q HIP library not found at {path}; build it with "
                               "`python -m fine_grained_quantization_amd.build`")
        lib = ctypes.CDLL(path)
        P, I64, I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
        lib.fp8q_quant_act_1x128.argtypes = [P, I64, I64, P, P, P]
        lib.fp8q_quant_w_128x128.argtypes = [P, I64, I64, P, P, P]
        lib.fp8q_swiglu_quant_act_1x128.argtypes = [P, P, I64, I64, I64, P, P, P]
        lib.fp8q_swiglu_bf16.argtypes = [P, P, I64, I64, I64, P, P]
        lib.fp8q_quant_act_dual.argtypes = [P, I64, I64, P, P, P, P, P]
        lib.fp8q_quant_act_fp4_1x128.argtypes = [P, I64, I64, P, P, P]
        lib.fp8q_quant_w_fp4_128x128.argtypes = [P, I64, I64, P, P, P]
        lib.fp8q_quant_w_per_channel.argtypes = [P, I64, I64, P, P, P]
        lib.fp8q_quant_act_e5m6_1x128.argtypes = [P, I64, I64, P, P, P]
        lib.fp8q_gemm_blockscaled.argtypes = [P, P, P, P, P, I, I64, I64, I64, P]
        lib.fp8q_grouped_gemm_blockscaled.argtypes = [P, P, P, P, P, I, P, I64, I64, I64, I64, P]
        lib.fp8q_dequant_w_128x128.argtypes = [P, P, I64, I64, P, P]
        lib.fp8q_grouped_gemm_blockscaled_gather.argtypes = [P, P, I64, P, P, P, P, I, P, I64, I64, I64, I64, P]
        lib.fp8q_moe_route_topk.argtypes = [P, I64, I64, I64, P, P, P, P, I64, P, I64, P]
        lib.fp8q_moe_gather_fp8.argtypes = [P, P, I64, I64, I64, P, P, P, I64, I64, P, P, P]
        lib.fp8q_moe_route_topk_noalloc.argtypes = [P, I64, I64, I64, P, P, P, P, I64, P]
        F = ctypes.c_float
        lib.fp8q_moe_gate_topk.argtypes = [P, I, I64, I64, I64, I64, I, P, I64, I64, I64, I, F, P, P, P, P, P, I64, P,
                                           P, I64, P]
        lib.fp8q_moe_gate_backward.argtypes = [P, I, I64, I64, I64, I64, I, I, F, P, P, P, P]
        lib.fp8q_moe_combine.argtypes = [P, I, I64, I64, P, P, I64, I64, P, P, P]
        lib.fp8q_moe_combine_backward.argtypes = [P, P, I, I64, I64, P, P, I64, I64, P, P, I64, P, P, P]
        lib.fp8q_quant_int8.argtypes = [P, I64, I64, I64, P, P, P]
        lib.fp8q_gemm_int8.argtypes = [P, P, P, P, P, I, I64, I64, I64, P]
        lib.fp8q_grouped_gemm_int8.argtypes = [P, P, P, P, P, I, P, I64, I64, I64, I64, P]
        lib.fp8q_grouped_gemm_int8_gather.argtypes = [P, P, I64, P, P, P, P, I, P, I64, I64, I64, I64, P]
        for f in (lib.fp8q_moe_gate_topk, lib.fp8q_moe_gate_backward, lib.fp8q_moe_combine,
                  lib.fp8q_moe_combine_backward, lib.fp8q_quant_int8, lib.fp8q_gemm_int8, lib.fp8q_grouped_gemm_int8,
                  lib.fp8q_grouped_gemm_int8_gather):
            f.restype = ctypes.c_int
        lib.fp8q_moe_gate_workspace_bytes.argtypes = [I64, I64]
        lib.fp8q_moe_gate_workspace_bytes.restype = I64
        for f in (lib.fp8q_quant_act_1x128, lib.fp8q_quant_w_128x128, lib.fp8q_swiglu_quant_act_1x128,
                  lib.fp8q_swiglu_bf16, lib.fp8q_quant_act_dual, lib.fp8q_quant_act_fp4_1x128,
                  lib.fp8q_quant_w_fp4_128x128, lib.fp8q_quant_w_per_channel, lib.fp8q_quant_act_e5m6_1x128,
                  lib.fp8q_gemm_blockscaled,
                  lib.fp8q_grouped_gemm_blockscaled, lib.fp8q_grouped_gemm_blockscaled_gather,
                  lib.fp8q_dequant_w_128x128, lib.fp8q_moe_route_topk, lib.fp8q_moe_route_topk_noalloc,
                  lib.fp8q_moe_gather_fp8):
            f.restype = ctypes.c_int
        lib.fp8q_moe_route_capacity.argtypes = [I64, I64, I64]
        lib.fp8q_moe_route_capacity.restype = I64
        lib.fp8q_moe_route_workspace_bytes.argtypes = [I64, I64]
        lib.fp8q_moe_route_workspace_bytes.restype = I64
        lib.fp8q_status_string.argtypes = [I]
        lib.fp8q_status_string.restype = ctypes.c_char_p
        lib.fp8q_version.argtypes = []
        lib.fp8q_version.restype = ctypes.c_int
        if path == LIB_PATH:
            _lib = lib
        return lib


def status_string(rc: int) -> str:
    return load_library().fp8q_status_string(rc).decode()


def _check(rc: int, name: str):
    if rc != 0:
        raise RuntimeError(f"{name}: {status_string(rc)}")


# The current stream's handle without building a Stream object (that costs ~3 us a call, a third of a
# call's host time); torch.cuda.current_stream() where this accessor does not exist.
_RAW_STREAM = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_GET_DEVICE = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


# Addresses go to ctypes as plain integers (the declared argument types make pointers of them).
def _stream_ptr(stream):
    if stream is None and _RAW_STREAM is not None:
        return _RAW_STREAM(_GET_DEVICE())
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


# Memory that a call allocates belongs to the stream that the call runs on.  torch hands a freed block to the
# stream that allocated it without waiting, so a block of the current stream's, used on another, could still have
# work of the current stream before it, and could be reused there while the other stream has not finished with it.
def _scratch(stream, nbytes, device):
    """A temporary of one call: freed on return, and reused only behind the call's own launches."""
    if stream is None:
        return torch.empty(max(nbytes, 4), dtype=torch.uint8, device=device)
    with torch.cuda.stream(_torch_stream(stream, device)):
        return torch.empty(max(nbytes, 4), dtype=torch.uint8, device=device)


def _empty(stream, shape, dtype, device):
    """An output of a call.  On a given stream it is that stream's, and kept from reuse until the current stream
    too is done with what was queued there before it was freed."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    current = torch.cuda.current_stream(device)
    with torch.cuda.stream(_torch_stream(stream, device)):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(current)
    return t


def _torch_stream(stream, device):
    return stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(stream.cuda_stream, device)


def _ptr(t):
    return t.data_ptr() if t is not None else None


def _need(t: torch.Tensor, name: str, dtypes, ndim=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}; expected one of {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() not in (ndim if isinstance(ndim, tuple) else (ndim,)):
        raise ValueError(f"{name} must have {ndim} dims, got {t.dim()}")


_BF16 = (torch.bfloat16, torch.int16, torch.uint16)
_FP8 = (torch.uint8, torch.float8_e4m3fn)


def fp8q_quant_act_1x128(x: torch.Tensor, q: torch.Tensor | None = None, s: torch.Tensor | None = None,
                         stream=None):
    """1x128 activation quantization.  ``x`` bf16 [M, K] -> ``(q uint8 [M, K], s float32 [K/128, M])``."""
    _need(x, "x", _BF16, 2)
    M, K = x.shape
    if q is None:
        q = _empty(stream, (M, K), dtype=torch.uint8, device=x.device)
    if s is None:
        s = _empty(stream, (K // 128, M), dtype=torch.float32, device=x.device)
    _need(q, "q", _FP8)
    _need(s, "s", (torch.float32,))
    if q.numel() != M * K or s.numel() != (K // 128) * M:
        raise ValueError("output tensors have the wrong size")
    _check(load_library().fp8q_quant_act_1x128(_ptr(x), M, K, _ptr(q), _ptr(s), _stream_ptr(stream)),
           "fp8q_quant_act_1x128")
    return q, s


def fp8q_quant_act_fp4_1x128(x: torch.Tensor, q: torch.Tensor | None = None, s: torch.Tensor | None = None,
                             stream=None):
    """1x128 FP4 (E2M1) activation quantization.  ``x`` bf16 [M, K] -> ``(q uint8 [M, K/2], s float32
    [K/128, M])``, two codes a byte (element 2i in the low nibble)."""
    _need(x, "x", _BF16, 2)
    M, K = x.shape
    if q is None:
        q = _empty(stream, (M, K // 2), dtype=torch.uint8, device=x.device)
    if s is None:
        s = _empty(stream, (K // 128, M), dtype=torch.float32, device=x.device)
    _need(q, "q", (torch.uint8,))
    _need(s, "s", (torch.float32,))
    if q.numel() != M * (K // 2) or s.numel() != (K // 128) * M:
        raise ValueError("output tensors have the wrong size")
    _check(load_library().fp8q_quant_act_fp4_1x128(_ptr(x), M, K, _ptr(q), _ptr(s), _stream_ptr(stream)),
           "fp8q_quant_act_fp4_1x128")
    return q, s


def fp8q_quant_w_fp4_128x128(w: torch.Tensor, q: torch.Tensor | None = None, s: torch.Tensor | None = None,
                             stream=None):
    """128x128 FP4 (E2M1) weight quantization.  ``w`` bf16 [N, K] -> ``(q uint8 [N, K/2], s float32
    [N/128, K/128])``."""
    _need(w, "w", _BF16, 2)
    N, K = w.shape
    if q is None:
        q = _empty(stream, (N, K // 2), dtype=torch.uint8, device=w.device)
    if s is None:
        s = _empty(stream, (N // 128, K // 128), dtype=torch.float32, device=w.device)
    _need(q, "q", (torch.uint8,))
    _need(s, "s", (torch.float32,))
    if q.numel() != N * (K // 2) or s.numel() != (N // 128) * (K // 128):
        raise ValueError("output tensors have the wrong size")
    _check(load_library().fp8q_quant_w_fp4_128x128(_ptr(w), N, K, _ptr(q), _ptr(s), _stream_ptr(stream)),
           "fp8q_quant_w_fp4_128x128")
    return q, s


def fp8q_quant_act_e5m6_1x128(x: torch.Tensor, q: torch.Tensor | None = None, s: torch.Tensor | None = None,
                              stream=None):
    """1x128 E5M6 activation quantization.  ``x`` bf16 [M, K] -> ``(q uint8 [M, 3K/2], s float32 [K/128, M])``,
    two 12-bit codes per 3 bytes (element j at bits 12j of its row)."""
    _need(x, "x", _BF16, 2)
    M, K = x.shape
    if q is None:
        q = _empty(stream, (M, K // 2 * 3), dtype=torch.uint8, device=x.device)
    if s is None:
        s = _empty(stream, (K // 128, M), dtype=torch.float32, device=x.device)
    _need(q, "q", (torch.uint8,))
    _need(s, "s", (torch.float32,))
    if q.numel() != M * (K // 2 * 3) or s.numel() != M * (K // 128):
        raise ValueError("output tensors have the wrong size")
    _check(load_library().fp8q_quant_act_e5m6_1x128(_ptr(x), M, K, _ptr(q), _ptr(s), _stream_ptr(stream)),
           "fp8q_quant_act_e5m6_1x128")
    return q, s


def fp8q_quant_w_per_channel(w: torch.Tensor, q: torch.Tensor | None = None, s: torch.Tensor | None = None,
                             stream=None):
    """Per-channel FP8 weight quantization, one scale per output channel.  ``w`` bf16 [N, K] (K a multiple of
    8) -> ``(q uint8 [N, K], s float32 [N])``."""
    _need(w, "w", _BF16, 2)
    N, K = w.shape
    if q is None:
        q = _empty(stream, (N, K), dtype=torch.uint8, device=w.device)
    if s is None:
        s = _empty(stream, (N,), dtype=torch.float32, device=w.device)
    _need(q, "q", (torch.uint8,))
    _need(s, "s", (torch.float32,))
    if q.numel() != N * K or s.numel() != N:
        raise ValueError("output tensors have the wrong size")
    _check(load_library().fp8q_quant_w_per_channel(_ptr(w), N, K, _ptr(q), _ptr(s), _stream_ptr(stream)),
           "fp8q_quant_w_per_channel")
    return q, s


def fp8q_quant_act_dual(x: torch.Tensor, q=None, s=None, qt=None, st=None, stream=None):
    """Forward and backward FP8 copies of a Linear input in one pass.  ``x`` bf16 [M, K] (M, K multiples of
    128) -> ``(q uint8 [M, K], s float32 [K/128, M], qt uint8 [K, M], st float32 [M/128, K])``: the 1x128
    quantization of x and of x^T (per channel, per 128 tokens).  Outputs not given are allocated."""
    _need(x, "x", _BF16, 2)
    M, K = x.shape
    dev = x.device
    q = _empty(stream, (M, K), dtype=torch.uint8, device=dev) if q is None else q
    s = _empty(stream, (K // 128, M), dtype=torch.float32, device=dev) if s is None else s
    qt = _empty(stream, (K, M), dtype=torch.uint8, device=dev) if qt is None else qt
    st = _empty(stream, (M // 128, K), dtype=torch.float32, device=dev) if st is None else st
    for t, name, dt, n in ((q, "q", torch.uint8, M * K), (s, "s", torch.float32, (K // 128) * M),
                           (qt, "qt", torch.uint8, M * K), (st, "st", torch.float32, (M // 128) * K)):
        _need(t, name, (dt,))
        if t.numel() != n:
            raise ValueError(f"{name} has the wrong size")
    _check(load_library().fp8q_quant_act_dual(_ptr(x), M, K, _ptr(q), _ptr(s), _ptr(qt), _ptr(st),
                                              _stream_ptr(stream)), "fp8q_quant_act_dual")
    return q, s, qt, st


def fp8q_swiglu_quant_act_1x128(x: torch.Tensor, y: torch.Tensor | None = None, q: torch.Tensor | None = None,
                                s: torch.Tensor | None = None, stream=None):
    """Fused SwiGLU + 1x128 quantization of h = bf16(SiLU(x) * y).  Either ``x`` (gate) and ``y`` (up) bf16
    [M, K] with equal row strides (views are fine), or ``x`` alone as one [M, 2K] tensor whose halves are the
    gate and the up projection -> ``(q uint8 [M, K], s float32 [K/128, M])``."""
    _need_rows(x, "x")
    if y is None:
        M, K2 = x.shape
        if K2 % 2:
            raise ValueError("a fused gate/up tensor needs an even number of columns")
        K = K2 // 2
        ld = x.stride(0)
        y = x[:, K:]
        x = x[:, :K]
    else:
        _need_rows(y, "y")
        if y.shape != x.shape or y.stride(0) != x.stride(0):
            raise ValueError("x and y must have the same shape and row stride")
        M, K = x.shape
        ld = x.stride(0)
    if q is None:
        q = _empty(stream, (M, K), dtype=torch.uint8, device=x.device)
    if s is None:
        s = _empty(stream, (K // 128, M), dtype=torch.float32, device=x.device)
    _need(q, "q", _FP8)
    _need(s, "s", (torch.float32,))
    if q.numel() != M * K or s.numel() != (K // 128) * M:
        raise ValueError("output tensors have the wrong size")
    _check(load_library().fp8q_swiglu_quant_act_1x128(_ptr(x), _ptr(y), ld, M, K, _ptr(q), _ptr(s),
                                                      _stream_ptr(stream)), "fp8q_swiglu_quant_act_1x128")
    return q, s


def fp8q_swiglu_bf16(x: torch.Tensor, y: torch.Tensor, h: torch.Tensor | None = None, stream=None):
    """h = bf16(SiLU(x) * y) written out (the intermediate the fused quantizer keeps in registers).  ``x``,
    ``y`` bf16 [M, K] with equal row strides -> ``h`` bf16 [M, K]."""
    _need_rows(x, "x")
    _need_rows(y, "y")
    if y.shape != x.shape or y.stride(0) != x.stride(0):
        raise ValueError("x and y must have the same shape and row stride")
    M, K = x.shape
    if h is None:
        h = _empty(stream, (M, K), dtype=torch.bfloat16, device=x.device)
    _need(h, "h", _BF16)
    if h.numel() != M * K:
        raise ValueError("h has the wrong size")
    _check(load_library().fp8q_swiglu_bf16(_ptr(x), _ptr(y), x.stride(0), M, K, _ptr(h), _stream_ptr(stream)),
           "fp8q_swiglu_bf16")
    return h


def _need_rows(t, name):
    """A bf16 [M, K] device view whose rows are contiguous (any row stride)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype not in _BF16 or t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D bf16 device tensor")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have contiguous rows")


def fp8q_quant_w_128x128(w: torch.Tensor, q: torch.Tensor | None = None, s: torch.Tensor | None = None,
                         stream=None):
    """128x128 weight quantization.  ``w`` bf16 [N, K] (or an expert stack [E, N, K]) ->
    ``(q uint8, s float32 [N/128, K/128])`` (``[E, N/128, K/128]`` for a stack)."""
    _need(w, "w", _BF16, (2, 3))
    lead = tuple(w.shape[:-2])
    N, K = w.shape[-2:]
    rows = N * (lead[0] if lead else 1)
    if q is None:
        q = _empty(stream, w.shape, dtype=torch.uint8, device=w.device)
    if s is None:
        s = _empty(stream, lead + (N // 128, K // 128), dtype=torch.float32, device=w.device)
    _need(q, "q", _FP8)
    _need(s, "s", (torch.float32,))
    if q.numel() != w.numel() or s.numel() != (rows // 128) * (K // 128):
        raise ValueError("output tensors have the wrong size")
    _check(load_library().fp8q_quant_w_128x128(_ptr(w), rows, K, _ptr(q), _ptr(s), _stream_ptr(stream)),
           "fp8q_quant_w_128x128")
    return q, s


def fp8q_dequant_w_128x128(q: torch.Tensor, s: torch.Tensor, w: torch.Tensor | None = None, stream=None):
    """FP8 -> BF16 weight conversion with 128x128 block scales.  ``q`` E4M3 codes [N, K] (or an expert stack
    [E, N, K]), ``s`` float32 [N/128, K/128] (``[E, N/128, K/128]``) -> ``w`` bf16 of ``q``'s shape."""
    _need(q, "q", _FP8, (2, 3))
    _need(s, "s", (torch.float32,))
    K = q.shape[-1]
    rows = q.numel() // K if K else 0
    if s.numel() != (rows // 128) * (K // 128):
        raise ValueError("s has the wrong size")
    if w is None:
        w = _empty(stream, q.shape, dtype=torch.bfloat16, device=q.device)
    _need(w, "w", _BF16)
    if w.numel() != q.numel():
        raise ValueError("w has the wrong size")
    _check(load_library().fp8q_dequant_w_128x128(_ptr(q), _ptr(s), rows, K, _ptr(w), _stream_ptr(stream)),
           "fp8q_dequant_w_128x128")
    return w


def _out_code(out_dtype):
    if out_dtype == torch.bfloat16:
        return OUT_BF16
    if out_dtype == torch.float32:
        return OUT_F32
    raise ValueError(f"out_dtype must be torch.bfloat16 or torch.float32, got {out_dtype}")


def fp8q_gemm_blockscaled(qa, sa, qw, sw, out_dtype=torch.bfloat16, c=None, stream=None):
    """Block-scaled FP8 GEMM ``C = A W^T``.  ``qa`` [M, K], ``sa`` [K/128, M], ``qw`` [N, K],
    ``sw`` [N/128, K/128] -> ``c`` [M, N] in ``out_dtype`` (bf16 or fp32)."""
    _need(qa, "qa", _FP8, 2)
    _need(qw, "qw", _FP8, 2)
    _need(sa, "sa", (torch.float32,))
    _need(sw, "sw", (torch.float32,))
    M, K = qa.shape
    N = qw.shape[0]
    if qw.shape[1] != K or sa.numel() != (K // 128) * M or sw.numel() != (N // 128) * (K // 128):
        raise ValueError("inconsistent GEMM operand shapes")
    code = _out_code(out_dtype)
    if c is None:
        c = _empty(stream, (M, N), dtype=out_dtype, device=qa.device)
    _need(c, "c", (out_dtype,))
    if c.numel() != M * N:
        raise ValueError("c has the wrong size")
    _check(load_library().fp8q_gemm_blockscaled(_ptr(qa), _ptr(sa), _ptr(qw), _ptr(sw), _ptr(c), code, M, N, K,
                                                _stream_ptr(stream)), "fp8q_gemm_blockscaled")
    return c


def fp8q_grouped_gemm_blockscaled(qa, sa, qw, sw, offsets, out_dtype=torch.bfloat16, c=None, stream=None):
    """Grouped (MoE) block-scaled FP8 GEMM.  ``qa`` [M_total, K], ``sa`` [K/128, M_total], ``qw`` [E, N, K],
    ``sw`` [E, N/128, K/128], ``offsets`` int32 device [E+1] -> ``c`` [M_total, N]."""
    _need(qa, "qa", _FP8, 2)
    _need(qw, "qw", _FP8, 3)
    _need(sa, "sa", (torch.float32,))
    _need(sw, "sw", (torch.float32,))
    _need(offsets, "offsets", (torch.int32,), 1)
    M, K = qa.shape
    E, N, K2 = qw.shape
    if K2 != K or sa.numel() != (K // 128) * M or sw.numel() != E * (N // 128) * (K // 128) or \
            offsets.numel() != E + 1:
        raise ValueError("inconsistent grouped GEMM operand shapes")
    code = _out_code(out_dtype)
    if c is None:
        c = _empty(stream, (M, N), dtype=out_dtype, device=qa.device)
    _need(c, "c", (out_dtype,))
    if c.numel() != M * N:
        raise ValueError("c has the wrong size")
    _check(load_library().fp8q_grouped_gemm_blockscaled(_ptr(qa), _ptr(sa), _ptr(qw), _ptr(sw), _ptr(c), code,
                                                        _ptr(offsets), E, M, N, K, _stream_ptr(stream)),
           "fp8q_grouped_gemm_blockscaled")
    return c


def fp8q_grouped_gemm_blockscaled_gather(q, s, row_token, qw, sw, offsets, out_dtype=torch.bfloat16, c=None,
                                         stream=None):
    """Grouped GEMM reading each row's token through ``row_token`` (the FP8 dispatch folded into the GEMM).
    ``q`` [T, K] token codes, ``s`` [K/128, T] token scales, ``row_token`` int32 device [M_total] (-1: empty
    row), ``qw`` [E, N, K], ``sw`` [E, N/128, K/128], ``offsets`` int32 device [E+1] -> ``c`` [M_total, N]."""
    _need(q, "q", _FP8, 2)
    _need(qw, "qw", _FP8, 3)
    _need(s, "s", (torch.float32,))
    _need(sw, "sw", (torch.float32,))
    _need(row_token, "row_token", (torch.int32,), 1)
    _need(offsets, "offsets", (torch.int32,), 1)
    T, K = q.shape
    E, N, K2 = qw.shape
    M = row_token.numel()
    if K2 != K or s.numel() != (K // 128) * T or sw.numel() != E * (N // 128) * (K // 128) or \
            offsets.numel() != E + 1:
        raise ValueError("inconsistent grouped GEMM operand shapes")
    code = _out_code(out_dtype)
    if c is None:
        c = _empty(stream, (M, N), dtype=out_dtype, device=qw.device)
    _need(c, "c", (out_dtype,))
    if c.numel() != M * N:
        raise ValueError("c has the wrong size")
    _check(load_library().fp8q_grouped_gemm_blockscaled_gather(
        _ptr(q), _ptr(s), T, _ptr(row_token), _ptr(qw), _ptr(sw), _ptr(c), code, _ptr(offsets), E, M, N, K,
        _stream_ptr(stream)), "fp8q_grouped_gemm_blockscaled_gather")
    return c


def fp8q_moe_route_capacity(T: int, E: int, k: int) -> int:
    """Rows any routing of T tokens to k of E experts fits in (T*k + 127*E, rounded up to 128)."""
    n = load_library().fp8q_moe_route_capacity(T, E, k)
    if n < 0:
        raise ValueError(f"invalid routing sizes T={T} E={E} k={k}")
    return n


def fp8q_moe_route_topk(logits, k: int, rows: int | None = None, workspace=None, out=None, stream=None):
    """Top-k gating and the expert-sorted, 128-padded layout.  ``logits`` float32 [T, E] ->
    ``(topk_idx int32 [T, k], offsets int32 [E+1], row_of int32 [T, k], row_token int32 [rows])``.
    ``rows`` defaults to :func:`fp8q_moe_route_capacity`; ``workspace`` (any device tensor of at least
    ``fp8q_moe_route_workspace_bytes(T, E)`` bytes) and ``out`` (the four outputs) are allocated when
    not given."""
    _need(logits, "logits", (torch.float32,), 2)
    T, E = logits.shape
    lib = load_library()
    cap = fp8q_moe_route_capacity(T, E, k)
    rows = cap if rows is None else rows
    wbytes = lib.fp8q_moe_route_workspace_bytes(T, E)
    if wbytes < 0:
        raise ValueError(f"invalid routing sizes T={T} E={E}")
    if workspace is None:
        workspace = _scratch(stream, wbytes, logits.device)
    if out is None:
        out = tuple(_empty(stream, shape, dtype=torch.int32, device=logits.device)
                    for shape in ((T, k), E + 1, (T, k), rows))
    topk_idx, offsets, row_of, row_token = out
    for t, n, size in ((topk_idx, "topk_idx", T * k), (offsets, "offsets", E + 1), (row_of, "row_of", T * k),
                       (row_token, "row_token", rows)):
        _need(t, n, (torch.int32,))
        if t.numel() != size:
            raise ValueError(f"{n} has {t.numel()} elements; expected {size}")
    if not workspace.is_cuda:
        raise ValueError("workspace must be a device tensor")
    _check(lib.fp8q_moe_route_topk(_ptr(logits), T, E, k, _ptr(topk_idx), _ptr(offsets), _ptr(row_of),
                                   _ptr(row_token), rows, _ptr(workspace),
                                   workspace.numel() * workspace.element_size(), _stream_ptr(stream)),
           "fp8q_moe_route_topk")
    return topk_idx, offsets, row_of, row_token


def fp8q_moe_route_topk_noalloc(logits, k: int, rows: int | None = None, out=None, stream=None):
    """:func:`fp8q_moe_route_topk` through the entry point that allocates nothing: its workspace is the
    library's fixed per-GPU array (calls that overlap on one GPU race).  ``out`` (the four outputs) is
    allocated here when not given; the C call itself allocates nothing."""
    _need(logits, "logits", (torch.float32,), 2)
    T, E = logits.shape
    lib = load_library()
    cap = fp8q_moe_route_capacity(T, E, k)
    rows = cap if rows is None else rows
    if out is None:
        out = tuple(_empty(stream, shape, dtype=torch.int32, device=logits.device)
                    for shape in ((T, k), E + 1, (T, k), rows))
    topk_idx, offsets, row_of, row_token = out
    for t, n, size in ((topk_idx, "topk_idx", T * k), (offsets, "offsets", E + 1), (row_of, "row_of", T * k),
                       (row_token, "row_token", rows)):
        _need(t, n, (torch.int32,))
        if t.numel() != size:
            raise ValueError(f"{n} has {t.numel()} elements; expected {size}")
    _check(lib.fp8q_moe_route_topk_noalloc(_ptr(logits), T, E, k, _ptr(topk_idx), _ptr(offsets), _ptr(row_of),
                                           _ptr(row_token), rows, _stream_ptr(stream)),
           "fp8q_moe_route_topk_noalloc")
    return topk_idx, offsets, row_of, row_token


def fp8q_moe_gather_fp8(q, s, row_of, row_token, offsets, qa=None, sa=None, stream=None):
    """Expert-sorted FP8 rows for the grouped GEMM.  ``q`` E4M3 [T, K] and ``s`` float32 [K/128, T] (the
    quantized tokens), ``row_of`` int32 [T, k], ``row_token`` int32 [rows] and ``offsets`` int32 [E+1] (one
    :func:`fp8q_moe_route_topk` call) -> ``(qa uint8 [rows, K], sa float32 [K/128, rows])``; rows from
    ``offsets[E]`` on are left as they were."""
    _need(q, "q", _FP8, 2)
    _need(s, "s", (torch.float32,))
    _need(row_of, "row_of", (torch.int32,), 2)
    _need(row_token, "row_token", (torch.int32,), 1)
    _need(offsets, "offsets", (torch.int32,), 1)
    T, K = q.shape
    if row_of.shape[0] != T:
        raise ValueError("row_of must have one row per token")
    k = row_of.shape[1]
    rows = row_token.numel()
    E = offsets.numel() - 1
    if s.numel() != (K // 128) * T:
        raise ValueError("s has the wrong size")
    if qa is None:
        qa = _empty(stream, (rows, K), dtype=torch.uint8, device=q.device)
    if sa is None:
        sa = _empty(stream, (K // 128, rows), dtype=torch.float32, device=q.device)
    _need(qa, "qa", _FP8)
    _need(sa, "sa", (torch.float32,))
    if qa.numel() != rows * K or sa.numel() != (K // 128) * rows:
        raise ValueError("output tensors have the wrong size")
    _check(load_library().fp8q_moe_gather_fp8(_ptr(q), _ptr(s), T, K, k, _ptr(row_of), _ptr(row_token),
                                              _ptr(offsets), E, rows, _ptr(qa), _ptr(sa), _stream_ptr(stream)),
           "fp8q_moe_gather_fp8")
    return qa, sa


_FLOAT = (torch.bfloat16, torch.float32)
_SCORES = {"sigmoid": 0, "softmax": 1}


def _score_code(score):
    if score not in _SCORES:
        raise ValueError(f"score must be one of {sorted(_SCORES)}, got {score!r}")
    return _SCORES[score]


def _need_out(t, name, dtype, size):
    """A contiguous device tensor of one dtype and element count (an output, or an input of known size)."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.is_cuda and t.is_contiguous() and t.numel() == size:
        return
    _need(t, name, (dtype,))
    if t.numel() != size:
        raise ValueError(f"{name} has {t.numel()} elements; expected {size}")


def _need_logits(x):
    """fp32 or bf16 logits [T, E] whose rows are contiguous (any row stride >= E); returns that stride."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda or x.dtype not in _FLOAT or x.dim() != 2:
        raise ValueError("logits must be a 2-D float32 or bfloat16 device tensor")
    T, E = x.shape
    if T > 0 and E > 1 and x.stride(1) != 1:
        raise ValueError("logits must have contiguous rows")
    ld = x.stride(0) if T > 1 else E
    if ld < E:
        raise ValueError("logits must not overlap between rows")
    return ld


def fp8q_moe_gate_topk(logits, k: int, score: str = "sigmoid", bias=None, n_group: int = 1, topk_group: int = 1,
                       group_top: int = 2, renormalize: bool = True, scale: float = 1.0, rows: int | None = None,
                       workspace=None, out=None, stream=None):
    """Gating with scores, bias, groups and weights, and the expert-sorted layout.  ``logits`` float32 or bf16
    [T, E] (rows may be strided), ``bias`` float32 [E] or None -> ``(topk_idx int32 [T, k], topk_weight float32
    [T, k], offsets int32 [E+1], row_of int32 [T, k], row_token int32 [rows], load int32 [E])``.

    ``score`` is "sigmoid" or "softmax"; the choice goes by score + bias within the ``topk_group`` best of
    ``n_group`` groups (a group's value is the sum of its ``group_top`` largest keys), the weights are the chosen
    scores, divided by their sum if ``renormalize``, times ``scale``.  Experts whose logit is -inf or NaN are never
    chosen; slots without an expert get expert -1, weight 0 and row -1.  ``rows`` defaults to
    :func:`fp8q_moe_route_capacity`; ``workspace`` (``fp8q_moe_gate_workspace_bytes(T, E)`` bytes, or that of more
    tokens) and ``out`` (the six outputs) are allocated when not given."""
    ld = _need_logits(logits)
    T, E = logits.shape
    lib = load_library()
    code = _score_code(score)
    if group_top not in (1, 2):
        raise ValueError(f"group_top must be 1 or 2, got {group_top}")
    if bias is not None:
        _need_out(bias, "bias", torch.float32, E)
    if rows is None:
        rows = fp8q_moe_route_capacity(T, E, k)
    wbytes = lib.fp8q_moe_gate_workspace_bytes(T, E)
    if wbytes < 0:
        raise ValueError(f"invalid gating sizes T={T} E={E}")
    if workspace is None:
        workspace = _scratch(stream, wbytes, logits.device)
    elif not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous device tensor")
    if out is None:
        i32 = dict(dtype=torch.int32, device=logits.device)
        out = (_empty(stream, (T, k), **i32), _empty(stream, (T, k), dtype=torch.float32, device=logits.device),
               _empty(stream, E + 1, **i32), _empty(stream, (T, k), **i32), _empty(stream, rows, **i32),
               _empty(stream, E, **i32))
    topk_idx, topk_weight, offsets, row_of, row_token, load = out
    _need_out(topk_idx, "topk_idx", torch.int32, T * k)
    _need_out(topk_weight, "topk_weight", torch.float32, T * k)
    _need_out(offsets, "offsets", torch.int32, E + 1)
    _need_out(row_of, "row_of", torch.int32, T * k)
    _need_out(row_token, "row_token", torch.int32, rows)
    _need_out(load, "load", torch.int32, E)
    _check(lib.fp8q_moe_gate_topk(_ptr(logits), _out_code(logits.dtype), ld, T, E, k, code, _ptr(bias), n_group,
                                  topk_group, group_top, 1 if renormalize else 0, scale, _ptr(topk_idx),
                                  _ptr(topk_weight), _ptr(offsets), _ptr(row_of), _ptr(row_token), rows, _ptr(load),
                                  _ptr(workspace), workspace.numel() * workspace.element_size(),
                                  _stream_ptr(stream)), "fp8q_moe_gate_topk")
    return topk_idx, topk_weight, offsets, row_of, row_token, load


def fp8q_moe_gate_backward(logits, topk_idx, grad_weight, score: str = "sigmoid", renormalize: bool = True,
                           scale: float = 1.0, grad_logits=None, stream=None):
    """Gradient of :func:`fp8q_moe_gate_topk`'s weights with respect to the logits, the choice held fixed.
    ``logits`` [T, E] float32 or bf16, ``topk_idx`` int32 [T, k], ``grad_weight`` float32 [T, k] -> ``grad_logits``
    [T, E] in the logits' dtype.  ``score``, ``renormalize`` and ``scale`` as in the forward call."""
    ld = _need_logits(logits)
    T, E = logits.shape
    code = _score_code(score)
    _need(topk_idx, "topk_idx", (torch.int32,), 2)
    if topk_idx.shape[0] != T:
        raise ValueError("topk_idx must have one row per token")
    k = topk_idx.shape[1]
    _need_out(grad_weight, "grad_weight", torch.float32, T * k)
    if grad_logits is None:
        grad_logits = _empty(stream, (T, E), dtype=logits.dtype, device=logits.device)
    _need_out(grad_logits, "grad_logits", logits.dtype, T * E)
    _check(load_library().fp8q_moe_gate_backward(
        _ptr(logits), _out_code(logits.dtype), ld, T, E, k, code, 1 if renormalize else 0, scale, _ptr(topk_idx),
        _ptr(grad_weight), _ptr(grad_logits), _stream_ptr(stream)), "fp8q_moe_gate_backward")
    return grad_logits


def fp8q_moe_combine(c, row_of, weight, add=None, y=None, stream=None):
    """Expert rows back to tokens: ``y[t] = add[t] + sum_j weight[t, j] * c[row_of[t, j]]``.  ``c`` bf16 or float32
    [rows, H], ``row_of`` int32 [T, k] (outside [0, rows): an empty slot), ``weight`` float32 [T, k], ``add`` [T, H]
    in ``c``'s dtype or None -> ``y`` [T, H] in ``c``'s dtype."""
    _need(c, "c", _FLOAT, 2)
    _need(row_of, "row_of", (torch.int32,), 2)
    rows, H = c.shape
    T, k = row_of.shape
    _need_out(weight, "weight", torch.float32, T * k)
    if add is not None:
        _need_out(add, "add", c.dtype, T * H)
    if y is None:
        y = _empty(stream, (T, H), dtype=c.dtype, device=c.device)
    _need_out(y, "y", c.dtype, T * H)
    _check(load_library().fp8q_moe_combine(_ptr(c), _out_code(c.dtype), rows, H, _ptr(row_of), _ptr(weight), T, k,
                                           _ptr(add), _ptr(y), _stream_ptr(stream)), "fp8q_moe_combine")
    return y


def fp8q_moe_combine_backward(grad_y, c, row_of, weight, row_token, offsets, grad_c=None, grad_weight=None,
                              stream=None):
    """Gradient of :func:`fp8q_moe_combine` -> ``(grad_c [rows, H], grad_weight float32 [T, k])``.  ``row_token`` int32
    [rows] and ``offsets`` int32 [E+1] are the layout ``row_of`` belongs to: rows below ``offsets[E]`` without a
    token get zeros, rows from there on are left as they were (uninitialized when ``grad_c`` is not given)."""
    _need(c, "c", _FLOAT, 2)
    _need(row_of, "row_of", (torch.int32,), 2)
    _need(offsets, "offsets", (torch.int32,), 1)
    rows, H = c.shape
    T, k = row_of.shape
    _need_out(grad_y, "grad_y", c.dtype, T * H)
    _need_out(weight, "weight", torch.float32, T * k)
    _need_out(row_token, "row_token", torch.int32, rows)
    if grad_c is None:
        grad_c = _empty(stream, c.shape, dtype=c.dtype, device=c.device)
    if grad_weight is None:
        grad_weight = _empty(stream, (T, k), dtype=torch.float32, device=c.device)
    _need_out(grad_c, "grad_c", c.dtype, rows * H)
    _need_out(grad_weight, "grad_weight", torch.float32, T * k)
    _check(load_library().fp8q_moe_combine_backward(
        _ptr(grad_y), _ptr(c), _out_code(c.dtype), rows, H, _ptr(row_of), _ptr(weight), T, k, _ptr(row_token),
        _ptr(offsets), offsets.numel() - 1, _ptr(grad_c), _ptr(grad_weight), _stream_ptr(stream)),
        "fp8q_moe_combine_backward")
    return grad_c, grad_weight


def fp8q_quant_int8(x, q=None, s=None, stream=None):
    """INT8 quantization with one scale per row (tokens, or a weight's output channels).  ``x`` bf16 [M, K] (rows
    may be strided; an expert stack is passed as [E * N, K]) -> ``(q int8 [M, K], s float32 [M])``."""
    _need_rows(x, "x")
    M, K = x.shape
    ld = x.stride(0) if M > 1 and K > 0 else (K + 7) // 8 * 8
    if q is None:
        q = _empty(stream, (M, K), dtype=torch.int8, device=x.device)
    if s is None:
        s = _empty(stream, (M,), dtype=torch.float32, device=x.device)
    _need_out(q, "q", torch.int8, M * K)
    _need_out(s, "s", torch.float32, M)
    _check(load_library().fp8q_quant_int8(_ptr(x), ld, M, K, _ptr(q), _ptr(s), _stream_ptr(stream)),
           "fp8q_quant_int8")
    return q, s


def fp8q_gemm_int8(qa, sa, qw, sw, out_dtype=torch.bfloat16, c=None, stream=None):
    """INT8 product with scales per token and channel: ``C[m, n] = sa[m] sw[n] sum_k qa[m, k] qw[n, k]``.  ``qa`` int8
    [M, K], ``sa`` float32 [M], ``qw`` int8 [N, K], ``sw`` float32 [N] -> ``c`` [M, N] in ``out_dtype``."""
    _need(qa, "qa", (torch.int8,), 2)
    _need(qw, "qw", (torch.int8,), 2)
    M, K = qa.shape
    N = qw.shape[0]
    if qw.shape[1] != K:
        raise ValueError("inconsistent GEMM operand shapes")
    _need_out(sa, "sa", torch.float32, M)
    _need_out(sw, "sw", torch.float32, N)
    code = _out_code(out_dtype)
    if c is None:
        c = _empty(stream, (M, N), dtype=out_dtype, device=qa.device)
    _need_out(c, "c", out_dtype, M * N)
    _check(load_library().fp8q_gemm_int8(_ptr(qa), _ptr(sa), _ptr(qw), _ptr(sw), _ptr(c), code, M, N, K,
                                         _stream_ptr(stream)), "fp8q_gemm_int8")
    return c


def fp8q_grouped_gemm_int8(qa, sa, qw, sw, offsets, out_dtype=torch.bfloat16, c=None, stream=None):
    """INT8 product per expert segment.  ``qa`` int8 [M_total, K], ``sa`` float32 [M_total], ``qw`` int8 [E, N, K],
    ``sw`` float32 [E, N], ``offsets`` int32 device [E+1] -> ``c`` [M_total, N]."""
    _need(qa, "qa", (torch.int8,), 2)
    _need(qw, "qw", (torch.int8,), 3)
    _need(offsets, "offsets", (torch.int32,), 1)
    M, K = qa.shape
    E, N, K2 = qw.shape
    if K2 != K or offsets.numel() != E + 1:
        raise ValueError("inconsistent grouped GEMM operand shapes")
    _need_out(sa, "sa", torch.float32, M)
    _need_out(sw, "sw", torch.float32, E * N)
    code = _out_code(out_dtype)
    if c is None:
        c = _empty(stream, (M, N), dtype=out_dtype, device=qa.device)
    _need_out(c, "c", out_dtype, M * N)
    _check(load_library().fp8q_grouped_gemm_int8(_ptr(qa), _ptr(sa), _ptr(qw), _ptr(sw), _ptr(c), code, _ptr(offsets),
                                                 E, M, N, K, _stream_ptr(stream)), "fp8q_grouped_gemm_int8")
    return c


def fp8q_grouped_gemm_int8_gather(q, s, row_token, qw, sw, offsets, out_dtype=torch.bfloat16, c=None, stream=None):
    """:func:`fp8q_grouped_gemm_int8` reading each row's token through ``row_token``.  ``q`` int8 [T, K] token codes,
    ``s`` float32 [T], ``row_token`` int32 device [M_total] (outside [0, T): an empty row, output 0), ``qw`` int8
    [E, N, K], ``sw`` float32 [E, N], ``offsets`` int32 device [E+1] -> ``c`` [M_total, N]."""
    _need(q, "q", (torch.int8,), 2)
    _need(qw, "qw", (torch.int8,), 3)
    _need(row_token, "row_token", (torch.int32,), 1)
    _need(offsets, "offsets", (torch.int32,), 1)
    T, K = q.shape
    E, N, K2 = qw.shape
    M = row_token.numel()
    if K2 != K or offsets.numel() != E + 1:
        raise ValueError("inconsistent grouped GEMM operand shapes")
    _need_out(s, "s", torch.float32, T)
    _need_out(sw, "sw", torch.float32, E * N)
    code = _out_code(out_dtype)
    if c is None:
        c = _empty(stream, (M, N), dtype=out_dtype, device=qw.device)
    _need_out(c, "c", out_dtype, M * N)
    _check(load_library().fp8q_grouped_gemm_int8_gather(
        _ptr(q), _ptr(s), T, _ptr(row_token), _ptr(qw), _ptr(sw), _ptr(c), code, _ptr(offsets), E, M, N, K,
        _stream_ptr(stream)), "fp8q_grouped_gemm_int8_gather")
    return c
