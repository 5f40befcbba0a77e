"""Python binding of libqift.so -- the B200 (sm_100a) hot path of Qift W2A4 linear layers.

"Qift: Shift-Friendly No-Zero W2 Post-Training Quantization for Rotated W2A4/KV4 LLM
Inference" (Huang, Tsai), Abstract: Hadamard-rotated weights and activations, fixed no-zero
2-bit level sets with one scale per output channel, 4-bit activations.

The functions here carry the C ABI's names (``include/qift.h``) and only marshal arguments:
they check devices, dtypes and shapes, allocate outputs with torch, and pass raw device
pointers plus the current CUDA stream, or the one given as ``stream``, to the library.  With
``stream`` given, the caller orders that stream after what the call's inputs come from, and
its own use of the results after that stream, as with any work on two streams; the results
come from that stream's memory.  Every step of the path runs in the library's kernels.  There
is no CPU fallback: without the built library or a CUDA device these functions raise.
"""
from __future__ import annotations

import ctypes as C
import functools
import math
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# QIFT_LIB_PATH selects another build of the same library -- the bounds-checked test build
# (libqift_check.so, `python -m w2a4_gemm_b200.build --check`); by default the normal one.
LIB_PATH = os.environ.get("QIFT_LIB_PATH") or os.path.join(_HERE, "libqift.so")

QIFT_OK, QIFT_ERR_INVALID_ARG, QIFT_ERR_UNSUPPORTED, QIFT_ERR_CUDA, QIFT_ERR_TIMEOUT = range(5)
QIFT_SET_QIFT, QIFT_SET_POT, QIFT_SET_STD, QIFT_SET_INT4 = 0, 1, 2, 3
QIFT_F32, QIFT_F16 = 0, 1
LEVELSETS = {"qift": QIFT_SET_QIFT, "pot": QIFT_SET_POT, "std": QIFT_SET_STD, "int4": QIFT_SET_INT4}

_lib = None


class QiftError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {qift_status_string(status)}")


def lib() -> C.CDLL:
    """Load libqift.so from the package directory; raise if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m w2a4_gemm_b200.build`")
        L = C.CDLL(LIB_PATH)
        i64, i32, f64, vp = C.c_int64, C.c_int32, C.c_double, C.c_void_p
        L.qift_rotate.argtypes = [vp, vp, i32, i64, i64, i32, vp]
        L.qift_quantize_weights.argtypes = [vp, i64, i64, i32, i32, f64, f64, vp, vp, vp, vp]
        L.qift_rotate_quantize_weights.argtypes = [vp, i64, i64, i32, i32, i32, f64, f64, vp, vp, vp, vp]
        L.qift_quantize_weights_asym.argtypes = [vp, i64, i64, i32, f64, f64, vp, vp, vp, vp, vp]
        L.qift_quantize_acts.argtypes = [vp, i64, i64, i32, vp, vp, vp]
        L.qift_quantize_kv.argtypes = [vp, i64, i64, i32, vp, vp, vp]
        L.qift_dequantize_kv.argtypes = [vp, vp, i64, i64, i32, vp, vp]
        L.qift_linear.argtypes = [vp, vp, vp, vp, i32, i64, i64, i64, vp, i32, vp]
        L.qift_decode_linear.argtypes = [vp, i64, i64, i32, vp, vp, i32, i64, vp, i32, vp, vp, vp]
        L.qift_append_kv.argtypes = [vp, i64, vp, i64, vp, i64, i64, i32, i32, i32, vp, i64, i32, i32, vp, vp, i32, vp,
                                     vp, vp, vp, vp, i64, i32, vp]
        L.qift_gather_kv.argtypes = [vp, vp, vp, vp, i64, i32, i32, i32, vp, i64, i32, vp, vp, vp]
        L.qift_paged_attention_workspace.argtypes = [i64] + [i32] * 11
        L.qift_paged_attention_workspace.restype = i64
        L.qift_paged_attention.argtypes = [vp, i64, i64, i32, i32, i32, vp, i32, i32, vp, vp, vp, vp, i64, i32, vp, i32,
                                           vp, i32, vp, i32, i32, i32, C.c_float, i32, vp, i32, vp, vp, i64, vp]
        L.qift_device_error.argtypes = [vp, C.POINTER(i32)]
        L.qift_debug_set_wait_limit.argtypes = [i64]
        L.qift_debug_stall_next_gemm.argtypes = []
        L.qift_debug_stall_next_one_token.argtypes = []
        L.qift_debug_stall_next_attention.argtypes = []
        L.qift_debug_set_attention_path.argtypes = [i32]
        L.qift_debug_set_linear_path.argtypes = [i32]
        L.qift_debug_set_pdl.argtypes = [i32]
        L.qift_debug_check_line.argtypes = [C.POINTER(i32)]
        L.qift_debug_checked_build.argtypes = []
        L.qift_debug_checked_build.restype = i32
        L.qift_status_string.argtypes = [i32]
        L.qift_status_string.restype = C.c_char_p
        for name in ("qift_rotate", "qift_quantize_weights", "qift_rotate_quantize_weights",
                     "qift_quantize_weights_asym", "qift_quantize_acts",
                     "qift_quantize_kv", "qift_dequantize_kv",
                     "qift_linear", "qift_decode_linear",
                     "qift_append_kv", "qift_gather_kv", "qift_paged_attention",
                     "qift_device_error", "qift_debug_set_wait_limit", "qift_debug_stall_next_gemm",
                     "qift_debug_stall_next_one_token", "qift_debug_stall_next_attention",
                     "qift_debug_set_attention_path",
                     "qift_debug_set_linear_path", "qift_debug_set_pdl", "qift_debug_check_line"):
            getattr(L, name).restype = C.c_int
        _lib = L
    return _lib


def qift_status_string(status: int) -> str:
    return lib().qift_status_string(int(status)).decode()


def _stream(stream, device=None):
    """The stream to launch on: `stream`, else the current stream of `device` (the device the
    call's tensors live on)."""
    if stream is None:
        stream = torch.cuda.current_stream(device)
    elif device is not None and stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
    return C.c_void_p(stream.cuda_stream)


def _made(stream, make, *args, **kw):
    """What make(...) allocates for a call on `stream` to write.  With a stream given, the memory is that stream's: memory
    of the current one may still be read by work queued there, which the call would not wait for.  The current stream,
    where the caller goes on (ordered after `stream` by the caller), is recorded, so that a result dropped there is not
    reused before what is queued there by then is done."""
    if stream is None:
        return make(*args, **kw)
    with torch.cuda.stream(stream):
        t = make(*args, **kw)
    current = torch.cuda.current_stream(t.device)
    if current != stream:
        t.record_stream(current)
    return t


def _ptr(t):
    return C.c_void_p(t.data_ptr()) if t is not None else None


def _cuda(t: torch.Tensor, name: str, dtype=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _same_device(*named):
    """All given (name, tensor) pairs (None tensors skipped) on one CUDA device; returns it."""
    dev = None
    for name, t in named:
        if t is None:
            continue
        if dev is None:
            dev, first = t.device, name
        elif t.device != dev:
            raise ValueError(f"{name} is on {t.device}, {first} on {dev}: every tensor of a call must be on one device")
    return dev


def _shape(t: torch.Tensor, name: str, shape: tuple):
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


def _at_least(t: torch.Tensor, name: str, n: int):
    if t.numel() < n:
        raise ValueError(f"{name} must hold at least {n} elements, got {t.numel()}")
    return t


def _2d(t: torch.Tensor, name: str):
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D, got shape {tuple(t.shape)}")
    return t


def _check(status: int, what: str):
    if status != QIFT_OK:
        raise QiftError(status, what)


def _set(levelset) -> int:
    return LEVELSETS[levelset] if isinstance(levelset, str) else int(levelset)


def _codes_per_word(levelset) -> int:
    """Codes per 32-bit word: 16 two-bit codes, or 8 four-bit codes for the INT4 set."""
    return 8 if _set(levelset) == QIFT_SET_INT4 else 16


def qift_rotate(x: torch.Tensor, block: int, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Block-diagonal normalised Walsh-Hadamard rotation along the last axis (fp32 or fp16)."""
    _cuda(x, "x")
    if x.dtype not in (torch.float32, torch.float16):
        raise ValueError("x must be float32 or float16")
    if x.dim() == 0:
        raise ValueError("x must have at least one dimension")
    if out is not None:
        _shape(_cuda(out, "out", x.dtype), "out", x.shape)
    dev = _same_device(("x", x), ("out", out))
    y = _made(stream, torch.empty_like, x) if out is None else out
    n = x.shape[-1]
    rows = x.numel() // n if n else 0
    dt = QIFT_F32 if x.dtype == torch.float32 else QIFT_F16
    with torch.cuda.device(dev):
        _check(lib().qift_rotate(_ptr(x), _ptr(y), dt, rows, n, block, _stream(stream, dev)), "qift_rotate")
    return y


def qift_quantize_weights(w_rot: torch.Tensor, levelset="qift", grid_points: int = 100, lo: float = 0.2,
                          hi: float = 1.0, with_mse: bool = True, stream=None):
    """Per-row scale search + nearest-level encode + 2-bit pack (4-bit for ``"int4"``).

    Returns ``(codes int32-viewed-as-u32 [N, K/16] ([N, K/8] for "int4"), scales f32 [N],
    row_mse f64 [N] or None)``.
    """
    _2d(_cuda(w_rot, "w_rot", torch.float32), "w_rot")
    n_out, n_in = w_rot.shape
    dev = w_rot.device
    codes = _made(stream, torch.empty, (n_out, n_in // _codes_per_word(levelset)), dtype=torch.int32, device=dev)
    scales = _made(stream, torch.empty, n_out, dtype=torch.float32, device=dev)
    mse = _made(stream, torch.empty, n_out, dtype=torch.float64, device=dev) if with_mse else None
    with torch.cuda.device(dev):
        _check(lib().qift_quantize_weights(_ptr(w_rot), n_out, n_in, _set(levelset), grid_points, lo, hi,
                                           _ptr(codes), _ptr(scales), _ptr(mse), _stream(stream, dev)),
               "qift_quantize_weights")
    return codes, scales, mse


def qift_quantize_weights_asym(w_rot: torch.Tensor, grid_points: int = 100, lo: float = 0.2, hi: float = 1.0,
                               with_mse: bool = True, stream=None):
    """Conventional asymmetric W2 baseline: per-row scale and integer zero point, weight (c - z) * s.

    Returns ``(codes int32-viewed-as-u32 [N, K/16], scales f32 [N], zeros int32 [N],
    row_mse f64 [N] or None)``.
    """
    _2d(_cuda(w_rot, "w_rot", torch.float32), "w_rot")
    n_out, n_in = w_rot.shape
    dev = w_rot.device
    codes = _made(stream, torch.empty, (n_out, n_in // 16), dtype=torch.int32, device=dev)
    scales = _made(stream, torch.empty, n_out, dtype=torch.float32, device=dev)
    zeros = _made(stream, torch.empty, n_out, dtype=torch.int32, device=dev)
    mse = _made(stream, torch.empty, n_out, dtype=torch.float64, device=dev) if with_mse else None
    with torch.cuda.device(dev):
        _check(lib().qift_quantize_weights_asym(_ptr(w_rot), n_out, n_in, grid_points, lo, hi, _ptr(codes),
                                                _ptr(scales), _ptr(zeros), _ptr(mse), _stream(stream, dev)),
               "qift_quantize_weights_asym")
    return codes, scales, zeros, mse


def qift_rotate_quantize_weights(w: torch.Tensor, block: int, levelset="qift", grid_points: int = 100,
                                 lo: float = 0.2, hi: float = 1.0, with_mse: bool = True, stream=None):
    """Rotation (block b; 0 = none) + scale search + encode + pack in one pass over the raw
    weights.  Same outputs, bit for bit, as ``qift_quantize_weights(qift_rotate(w, b))``."""
    _2d(_cuda(w, "w", torch.float32), "w")
    n_out, n_in = w.shape
    dev = w.device
    codes = _made(stream, torch.empty, (n_out, n_in // _codes_per_word(levelset)), dtype=torch.int32, device=dev)
    scales = _made(stream, torch.empty, n_out, dtype=torch.float32, device=dev)
    mse = _made(stream, torch.empty, n_out, dtype=torch.float64, device=dev) if with_mse else None
    with torch.cuda.device(dev):
        _check(lib().qift_rotate_quantize_weights(_ptr(w), n_out, n_in, block, _set(levelset), grid_points, lo,
                                                  hi, _ptr(codes), _ptr(scales), _ptr(mse), _stream(stream, dev)),
               "qift_rotate_quantize_weights")
    return codes, scales, mse


def qift_quantize_acts(x: torch.Tensor, block: int = 0, out_q: torch.Tensor | None = None,
                       out_scales: torch.Tensor | None = None, stream=None):
    """Optional rotation + symmetric per-token INT4.  Returns ``(q int8 [T, K], s_a f32 [T])``."""
    _2d(_cuda(x, "x", torch.float16), "x")
    T, K = x.shape
    if out_q is not None:
        _shape(_cuda(out_q, "out_q", torch.int8), "out_q", (T, K))
    if out_scales is not None:
        _at_least(_cuda(out_scales, "out_scales", torch.float32), "out_scales", T)
    dev = _same_device(("x", x), ("out_q", out_q), ("out_scales", out_scales))
    q = _made(stream, torch.empty, (T, K), dtype=torch.int8, device=dev) if out_q is None else out_q
    s = _made(stream, torch.empty, T, dtype=torch.float32, device=dev) if out_scales is None else out_scales
    with torch.cuda.device(dev):
        _check(lib().qift_quantize_acts(_ptr(x), T, K, block, _ptr(q), _ptr(s), _stream(stream, dev)),
               "qift_quantize_acts")
    return q, s


def qift_quantize_kv(x: torch.Tensor, block: int, stream=None):
    """KV4: rotation by ``block`` + per-token INT4, two codes per byte.
    Returns ``(packed uint8 [T, n/2], scales f32 [T])``."""
    _2d(_cuda(x, "x", torch.float16), "x")
    T, n = x.shape
    dev = x.device
    packed = _made(stream, torch.empty, (T, n // 2), dtype=torch.uint8, device=dev)
    scales = _made(stream, torch.empty, T, dtype=torch.float32, device=dev)
    with torch.cuda.device(dev):
        _check(lib().qift_quantize_kv(_ptr(x), T, n, block, _ptr(packed), _ptr(scales), _stream(stream, dev)),
               "qift_quantize_kv")
    return packed, scales


def qift_dequantize_kv(packed: torch.Tensor, scales: torch.Tensor, block: int, stream=None) -> torch.Tensor:
    """Inverse of ``qift_quantize_kv`` up to the quantization error: fp16 [T, n]."""
    _2d(_cuda(packed, "packed", torch.uint8), "packed")
    _cuda(scales, "scales", torch.float32)
    T, n2 = packed.shape
    _at_least(scales, "scales", T)
    dev = _same_device(("packed", packed), ("scales", scales))
    out = _made(stream, torch.empty, (T, 2 * n2), dtype=torch.float16, device=dev)
    with torch.cuda.device(dev):
        _check(lib().qift_dequantize_kv(_ptr(packed), _ptr(scales), T, 2 * n2, block, _ptr(out),
                                        _stream(stream, dev)), "qift_dequantize_kv")
    return out


def qift_linear(q: torch.Tensor, act_scale: torch.Tensor, codes: torch.Tensor, w_scale: torch.Tensor,
                levelset="qift", out_dtype=torch.float16, out: torch.Tensor | None = None, stream=None):
    """Fused W2A4 linear (W4A4 for ``"int4"``, 1..16 tokens):
    ``y[t, n] = ((float)acc * w_scale[n]) * act_scale[t]``."""
    _cuda(q, "q", torch.int8)
    _cuda(act_scale, "act_scale", torch.float32)
    _cuda(codes, "codes")
    _cuda(w_scale, "w_scale", torch.float32)
    if codes.dtype not in (torch.int32, torch.uint32):
        raise ValueError("codes must be 32-bit words")
    if out_dtype not in (torch.float16, torch.float32):
        raise ValueError("out_dtype must be torch.float16 or torch.float32")
    _2d(q, "q")
    _2d(codes, "codes")
    T, K = q.shape
    N = codes.shape[0]
    cpw = _codes_per_word(levelset)
    if codes.shape[1] * cpw != K:
        raise ValueError(f"codes must be [n_out, n_in/{cpw}]")
    _at_least(act_scale, "act_scale", T)
    _at_least(w_scale, "w_scale", N)
    if out is not None:
        _shape(_cuda(out, "out", out_dtype), "out", (T, N))
    dev = _same_device(("q", q), ("act_scale", act_scale), ("codes", codes), ("w_scale", w_scale), ("out", out))
    y = _made(stream, torch.empty, (T, N), dtype=out_dtype, device=dev) if out is None else out
    dt = QIFT_F16 if out_dtype == torch.float16 else QIFT_F32
    with torch.cuda.device(dev):
        _check(lib().qift_linear(_ptr(q), _ptr(act_scale), _ptr(codes), _ptr(w_scale), _set(levelset), T, N, K,
                                 _ptr(y), dt, _stream(stream, dev)), "qift_linear")
    return y


def qift_decode_linear(x: torch.Tensor, block: int, codes: torch.Tensor, w_scale: torch.Tensor, levelset="qift",
                       out_dtype=torch.float16, out: torch.Tensor | None = None, q_out: torch.Tensor | None = None,
                       act_scale_out: torch.Tensor | None = None, stream=None):
    """One-launch decode step (1..4 tokens): rotation + INT4 + W2A4 linear.  Returns y."""
    _cuda(x, "x", torch.float16)
    _cuda(codes, "codes")
    _cuda(w_scale, "w_scale", torch.float32)
    if codes.dtype not in (torch.int32, torch.uint32):
        raise ValueError("codes must be 32-bit words")
    if out_dtype not in (torch.float16, torch.float32):
        raise ValueError("out_dtype must be torch.float16 or torch.float32")
    _2d(x, "x")
    _2d(codes, "codes")
    T, K = x.shape
    N = codes.shape[0]
    cpw = _codes_per_word(levelset)
    if codes.shape[1] * cpw != K:
        raise ValueError(f"codes must be [n_out, n_in/{cpw}]")
    _at_least(w_scale, "w_scale", N)
    if out is not None:
        _shape(_cuda(out, "out", out_dtype), "out", (T, N))
    if q_out is not None:
        _shape(_cuda(q_out, "q_out", torch.int8), "q_out", (T, K))
    if act_scale_out is not None:
        _at_least(_cuda(act_scale_out, "act_scale_out", torch.float32), "act_scale_out", T)
    dev = _same_device(("x", x), ("codes", codes), ("w_scale", w_scale), ("out", out), ("q_out", q_out),
                       ("act_scale_out", act_scale_out))
    y = _made(stream, torch.empty, (T, N), dtype=out_dtype, device=dev) if out is None else out
    dt = QIFT_F16 if out_dtype == torch.float16 else QIFT_F32
    with torch.cuda.device(dev):
        _check(lib().qift_decode_linear(_ptr(x), T, K, block, _ptr(codes), _ptr(w_scale), _set(levelset), N, _ptr(y),
                                        dt, _ptr(q_out), _ptr(act_scale_out), _stream(stream, dev)),
               "qift_decode_linear")
    return y


# The paged cache's calls are made once a layer and token, so their checks are kept lean: one quick test a
# tensor, and the checks above only to say what is wrong.
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device  # tensors exist: CUDA is up
_U8, _F16, _F32, _I32, _I64 = torch.uint8, torch.float16, torch.float32, torch.int32, torch.int64


def _is(t, name: str, dtype, shape: tuple, index: int) -> int:
    """Address of `t`, which must be a contiguous tensor of this dtype and shape on CUDA device `index`."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == index and \
            t.is_contiguous():
        return t.data_ptr()
    _shape(_cuda(t, name, dtype), name, shape)
    raise ValueError(f"{name} is on {t.device}, other tensors of the call on cuda:{index}")


def _heads(t, name: str, shape: tuple, index: int) -> tuple[int, int]:
    """Address and elements between tokens of a [tokens, heads, head_dim] fp16 tensor whose heads lie one behind
    the other (a slice of a projection's output is one)."""
    n, h, d = shape
    if isinstance(t, torch.Tensor) and t.dtype is _F16 and t.shape == shape and t.get_device() == index:
        row, head, one = t.stride()
        if n <= 1:
            row = h * d
        if (one == 1 or d <= 1) and (head == d or h <= 1) and row >= h * d:
            return t.data_ptr(), row
        raise ValueError(f"{name} must hold each token's heads one behind the other, got strides {t.stride()}")
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    if t.dtype is not _F16:
        raise ValueError(f"{name} must be torch.float16, got {t.dtype}")
    _shape(t, name, shape)
    raise ValueError(f"{name} is on {t.device}, other tensors of the call on cuda:{index}")


def _cache(k_cache, k_scales, v_cache, v_scales):
    """Checks a paged cache; returns its addresses, pages, kv_heads, page_size, head_dim and its device's index."""
    try:
        pages, kv_heads, size, half = shape = k_cache.shape
        rows, index = (pages, kv_heads, size), k_cache.get_device()
        if index >= 0 and k_cache.dtype is _U8 and v_cache.dtype is _U8 and k_scales.dtype is _F32 and \
                v_scales.dtype is _F32 and v_cache.shape == shape and k_scales.shape == rows and v_scales.shape == rows and \
                v_cache.get_device() == k_scales.get_device() == v_scales.get_device() == index and \
                k_cache.is_contiguous() and v_cache.is_contiguous() and k_scales.is_contiguous() and v_scales.is_contiguous():
            return (k_cache.data_ptr(), k_scales.data_ptr(), v_cache.data_ptr(), v_scales.data_ptr(), pages, kv_heads, size,
                    2 * half, index)
    except (AttributeError, TypeError, ValueError):
        pass
    _cuda(k_cache, "k_cache", _U8)  # which of it
    shape = k_cache.shape
    if len(shape) != 4:
        raise ValueError(f"k_cache must be [pages, kv_heads, page_size, head_dim / 2], got shape {tuple(shape)}")
    pages, kv_heads, size, half = shape
    rows, index = (pages, kv_heads, size), k_cache.get_device()
    return (k_cache.data_ptr(), _is(k_scales, "k_scales", _F32, rows, index), _is(v_cache, "v_cache", _U8, shape, index),
            _is(v_scales, "v_scales", _F32, rows, index), pages, kv_heads, size, 2 * half, index)


def _on(stream, index: int):
    """The stream to launch on: `stream`, or the current one of device `index`."""
    if stream is None:
        return _current_stream(index)
    if stream.device.index != index:
        raise ValueError(f"stream is on {stream.device}, the tensors on cuda:{index}")
    return stream.cuda_stream


def _launch(index: int, fn, args: tuple) -> int:
    """Calls the library's `fn` with device `index` current."""
    if _current_device() == index:
        return fn(*args)
    with torch.cuda.device(index):
        return fn(*args)


def _int32(**values):
    """Refuses what the library's 32-bit arguments would cut to another value."""
    for name, x in values.items():
        if not -2 ** 31 <= x < 2 ** 31:
            raise ValueError(f"{name} must fit 32 bits, got {x}")


def qift_append_kv(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, block: int, k_cache: torch.Tensor,
                   k_scales: torch.Tensor, v_cache: torch.Tensor, v_scales: torch.Tensor,
                   q: torch.Tensor | None = None, positions: torch.Tensor | None = None,
                   rope: torch.Tensor | None = None, interleaved: bool = False, q_out: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor | None:
    """New tokens into a paged KV4 cache: position rotation, Hadamard rotation by ``block``, INT4 rows.

    ``k``, ``v`` (and ``q``) are fp16 ``[tokens, heads, head_dim]``, slices of one projection's output as they
    are.  ``k_cache``/``v_cache`` uint8 ``[pages, kv_heads, page_size, head_dim / 2]`` and ``k_scales``/``v_scales``
    fp32 ``[pages, kv_heads, page_size]`` are written at ``slots`` (int64, ``page * page_size + offset``; -1 =
    padding).  ``rope`` fp32 ``[positions, rope_dim]`` holds cosines, then sines, and ``positions`` (int64) its row
    for each token; a token whose position is outside it is left out, its row of a new result not initialised.
    Returns the rotated queries ``[tokens, q_heads, head_dim]`` (None without ``q``)."""
    if not 0 <= block < 2 ** 31:
        _int32(block=block)
    kc, ks, vc, vs, pages, kv_heads, size, d, index = _cache(k_cache, k_scales, v_cache, v_scales)
    T = k.shape[0] if isinstance(k, torch.Tensor) and k.dim() else 0
    rows = (T, kv_heads, d)
    k_at, k_row = _heads(k, "k", rows, index)
    v_at, v_row = _heads(v, "v", rows, index)
    slots_at = _is(slots, "slots", _I64, (T,), index)
    q_at = out_at = rope_at = positions_at = None
    q_row = hq = rope_len = rope_dim = 0
    if rope is not None:
        if positions is None:
            raise ValueError("rope needs positions")
        if not isinstance(rope, torch.Tensor) or rope.dim() != 2:
            _2d(_cuda(rope, "rope", _F32), "rope")
        rope_len, rope_dim = shape = rope.shape
        rope_at = _is(rope, "rope", _F32, shape, index)
        if T and not (rope_len and rope_dim):  # without an address it would pass for no rotation at all
            raise ValueError(f"rope must hold at least one position and one pair, got shape {tuple(shape)}")
        positions_at = _is(positions, "positions", _I64, (T,), index)
    if q is not None:
        hq = q.shape[1] if isinstance(q, torch.Tensor) and q.dim() == 3 else 0
        q_at, q_row = _heads(q, "q", (T, hq, d), index)
        if hq == 0:
            raise ValueError("q must have at least one head")
        if q_out is None:
            if stream is not None:
                q_out = _made(stream, q.new_empty, (T, hq, d))
            else:
                q_out = torch.empty_like(q) if T <= 1 or q_row == hq * d else q.new_empty((T, hq, d))
            out_at = q_out.data_ptr()
        else:
            out_at = _is(q_out, "q_out", _F16, (T, hq, d), index)
    elif q_out is not None:
        raise ValueError("q_out without q")
    if T:  # an empty tensor has no address
        status = _launch(index, (_lib or lib()).qift_append_kv, (
            q_at, q_row, k_at, k_row, v_at, v_row, T, hq, kv_heads, d, rope_at, rope_len, rope_dim, 1 if interleaved else 0,
            positions_at, slots_at, block, out_at, kc, ks, vc, vs, pages, size, _on(stream, index)))
        if status:
            _check(status, "qift_append_kv")
    return q_out


def qift_gather_kv(k_cache: torch.Tensor, k_scales: torch.Tensor, v_cache: torch.Tensor, v_scales: torch.Tensor,
                   slots: torch.Tensor, block: int, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Rows of a paged KV4 cache read back, rotated back by ``block`` (0: in the cache's domain): fp16
    ``(k, v)``, each ``[tokens, kv_heads, head_dim]``; zeros for slots outside the cache."""
    if not 0 <= block < 2 ** 31:
        _int32(block=block)
    kc, ks, vc, vs, pages, kv_heads, size, d, index = _cache(k_cache, k_scales, v_cache, v_scales)
    T = slots.shape[0] if isinstance(slots, torch.Tensor) and slots.dim() else 0
    slots_at = _is(slots, "slots", _I64, (T,), index)
    if stream is None:
        k = k_scales.new_empty((T, kv_heads, d), dtype=_F16)
        v = torch.empty_like(k)
    else:
        k, v = (_made(stream, k_scales.new_empty, (T, kv_heads, d), dtype=_F16) for _ in range(2))
    status = _launch(index, (_lib or lib()).qift_gather_kv, (
        kc, ks, vc, vs, pages, size, kv_heads, d, slots_at, T, block, k.data_ptr(), v.data_ptr(), _on(stream, index)))
    if status:
        _check(status, "qift_gather_kv")
    return k, v


def qift_paged_attention(q: torch.Tensor, cu_q: torch.Tensor | None, max_q: int, k_cache: torch.Tensor,
                         k_scales: torch.Tensor, v_cache: torch.Tensor, v_scales: torch.Tensor,
                         page_table: torch.Tensor, kv_lens: torch.Tensor, window: int = 0, sinks: int = 0,
                         prefix_table: torch.Tensor | None = None, prefix_len: int = 0, max_kv: int = 0,
                         scale: float | None = None, block: int = 0, out_dtype=torch.float16,
                         out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                         workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Causal attention of a ragged batch over a paged KV4 cache.

    ``q`` fp16 ``[tokens, q_heads, head_dim]`` holds rotated queries (what ``qift_append_kv`` returns); sequence
    ``b`` has rows ``cu_q[b] .. cu_q[b + 1] - 1`` (int32; None: ``max_q`` rows each), at most ``max_q``, and
    ``kv_lens[b]`` keys (int32, the new tokens and the prefix included) in the pages ``page_table[b]`` (int32
    ``[batch, max_pages]``).  ``window``: keys a row sees up to its own (0: all), besides the first ``sinks``.
    ``prefix_table`` (int32): pages of the ``prefix_len`` first keys that all sequences share.  ``block``: the
    result is rotated back by Hadamard blocks of this size (0: left rotated, as ``qift_quantize_acts`` with block
    0 takes it).  ``lse`` (fp32 ``[tokens, q_heads]``), if given, receives the log-sum-exp.  ``workspace`` (uint8,
    ``qift_paged_attention_workspace`` bytes) is allocated on the call's stream if not given.  The softmax's
    weights are rounded to binary16 whatever ``out_dtype`` is.  Rows of a new result that belong to no sequence are
    not initialised."""
    if not 0 <= (max_q | window | sinks | prefix_len | max_kv | block) < 2 ** 31:
        _int32(max_q=max_q, window=window, sinks=sinks, prefix_len=prefix_len, max_kv=max_kv, block=block)
    kc, ks, vc, vs, pages, kv_heads, size, d, index = _cache(k_cache, k_scales, v_cache, v_scales)
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be a [tokens, q_heads, head_dim] tensor")
    shape = q.shape
    T, hq = shape[0], shape[1]
    q_at, q_row = _heads(q, "q", (T, hq, d), index)
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
        raise ValueError("page_table must be a [batch, max_pages] tensor")
    B, max_pages = table_shape = page_table.shape
    table_at = _is(page_table, "page_table", _I32, table_shape, index)
    lens_at = _is(kv_lens, "kv_lens", _I32, (B,), index)
    cu_at = prefix_at = lse_at = None
    if cu_q is not None:
        cu_at = _is(cu_q, "cu_q", _I32, (B + 1,), index)
    elif T != B * max_q:
        raise ValueError(f"without cu_q, q must have batch * max_q = {B * max_q} rows, got {T}")
    if prefix_table is not None:
        _at_least(_cuda(prefix_table, "prefix_table", _I32), "prefix_table", -(-prefix_len // size))
        prefix_at = _is(prefix_table, "prefix_table", _I32, prefix_table.shape, index)
    elif prefix_len != 0:
        raise ValueError("prefix_len needs prefix_table")
    if out_dtype is not _F16 and out_dtype is not _F32:
        raise ValueError("out_dtype must be torch.float16 or torch.float32")
    if lse is not None:
        lse_at = _is(lse, "lse", torch.float32, (T, hq), index)
    need = _workspace_bytes(T, hq, kv_heads, d, B, max_q, size, max_pages, max_kv, prefix_len, window, sinks)
    ws_at, ws_bytes = None, 0
    if workspace is not None:
        _at_least(_cuda(workspace, "workspace", _U8), "workspace", need)
        ws_at, ws_bytes = _is(workspace, "workspace", _U8, workspace.shape, index), workspace.numel()
    elif need > 0:
        if stream is None:
            workspace = k_cache.new_empty(need)
        else:  # freed, and used again, in the order of the stream that runs the kernels
            with torch.cuda.stream(stream):
                workspace = k_cache.new_empty(need)
        ws_at, ws_bytes = workspace.data_ptr(), need
    if out is None:
        if stream is not None:
            out = _made(stream, q.new_empty, shape, dtype=out_dtype)
        else:
            plain = out_dtype is _F16 and (T <= 1 or q_row == hq * d)
            out = torch.empty_like(q) if plain else q.new_empty(shape, dtype=out_dtype)
        out_at = out.data_ptr()
    else:
        out_at = _is(out, "out", out_dtype, shape, index)
    status = _launch(index, (_lib or lib()).qift_paged_attention, (
        q_at, q_row, T, hq, kv_heads, d, cu_at, B, max_q, kc, ks, vc, vs, pages, size, table_at, max_pages, lens_at, max_kv,
        prefix_at, prefix_len, window, sinks, 1.0 / math.sqrt(d) if scale is None else scale, block, out_at,
        QIFT_F16 if out_dtype is _F16 else QIFT_F32, lse_at, ws_at, ws_bytes, _on(stream, index)))
    if status:
        _check(status, "qift_paged_attention")
    return out


_kernel_pin = threading.local()  # the answer is the pinned kernel's, and a pin is a thread's


def _workspace_bytes(*sizes: int) -> int:
    return _workspace_bytes_of(getattr(_kernel_pin, "path", 0), *sizes)


@functools.lru_cache(maxsize=1024)
def _workspace_bytes_of(path: int, *sizes: int) -> int:
    return lib().qift_paged_attention_workspace(*sizes)


def qift_paged_attention_workspace(tokens: int, q_heads: int, kv_heads: int, head_dim: int, batch: int, max_q: int,
                                   page_size: int, max_pages: int, max_kv: int = 0, prefix_len: int = 0,
                                   window: int = 0, sinks: int = 0) -> int:
    """Bytes of workspace that ``qift_paged_attention`` needs for these sizes; raises if it would refuse them."""
    _int32(q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim, batch=batch, max_q=max_q, page_size=page_size,
           max_pages=max_pages, max_kv=max_kv, prefix_len=prefix_len, window=window, sinks=sinks)
    n = _workspace_bytes(tokens, q_heads, kv_heads, head_dim, batch, max_q, page_size, max_pages, max_kv, prefix_len,
                         window, sinks)
    if n < 0:
        raise ValueError("qift_paged_attention would refuse these sizes")
    return n


def qift_device_error(stream=None) -> tuple[int, int]:
    """Synchronise the stream, read and clear the device error word: ``(status, raw word)``."""
    detail = C.c_int32(0)
    st = lib().qift_device_error(_stream(stream), C.byref(detail))
    return st, detail.value


def qift_debug_checked_build() -> bool:
    """True when the loaded library is the bounds-checked test build."""
    return bool(lib().qift_debug_checked_build())


def qift_debug_check_line() -> int:
    """Source line of the first failed bounds check since the last call (0: none; always 0 in
    the normal build).  Read after qift_device_error(), which synchronises."""
    line = C.c_int32(0)
    _check(lib().qift_debug_check_line(C.byref(line)), "qift_debug_check_line")
    return line.value


def qift_debug_set_wait_limit(cycles: int) -> None:
    """Test hook: SM-cycle limit of every on-chip wait in later tensor-core GEMM and one-token
    launches (<= 0: default)."""
    _check(lib().qift_debug_set_wait_limit(int(cycles)), "qift_debug_set_wait_limit")


def qift_debug_stall_next_gemm() -> None:
    """Test hook: the next tensor-core GEMM waits on a barrier nothing arrives on and times out."""
    _check(lib().qift_debug_stall_next_gemm(), "qift_debug_stall_next_gemm")


def qift_debug_stall_next_one_token() -> None:
    """Test hook: the next one-token launch waits on a barrier nothing arrives on and times out."""
    _check(lib().qift_debug_stall_next_one_token(), "qift_debug_stall_next_one_token")


def qift_debug_stall_next_attention() -> None:
    """Test hook: the next attention launch for many rows waits on a barrier nothing arrives on and times out."""
    _check(lib().qift_debug_stall_next_attention(), "qift_debug_stall_next_attention")


LINEAR_PATHS = {"auto": 0, "gemv": 1, "skinny": 2, "gemm_pair": 6, "one_token": 7}


def qift_debug_set_linear_path(path) -> None:
    """Test hook: pin qift_linear's kernel family in this thread ("auto", "gemv", "skinny",
    "gemm_pair", "one_token")."""
    p = LINEAR_PATHS[path] if isinstance(path, str) else int(path)
    _check(lib().qift_debug_set_linear_path(p), "qift_debug_set_linear_path")


ATTENTION_PATHS = {"auto": 0, "stream": 1, "wide": 2}


def qift_debug_set_attention_path(path) -> None:
    """Test hook: pin qift_paged_attention's kernel in this thread ("auto", "stream", "wide")."""
    p = ATTENTION_PATHS[path] if isinstance(path, str) else int(path)
    _check(lib().qift_debug_set_attention_path(p), "qift_debug_set_attention_path")
    _kernel_pin.path = p


def qift_debug_set_pdl(enable: bool) -> None:
    """Test hook: programmatic dependent launch of the decode kernels on (default) or off."""
    _check(lib().qift_debug_set_pdl(1 if enable else 0), "qift_debug_set_pdl")
