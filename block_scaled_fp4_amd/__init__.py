"""Python binding of libfp4mi.so, the gfx950 block-scaled FP4 codec.

Argument marshalling only: every step of the codec runs in the library's
HIP kernels.  Tensors are torch tensors on the GPU (PyTorch supplies device
memory and the current stream); outputs that are not passed in are
allocated with torch.empty.  A non-zero status from the library raises
Fp4Error.  If the shared library has not been built this module raises at
import: there is no CPU fallback.

Entry points (same names as the C ABI in include/fp4mi.h):
  fp4_quantize, fp4_dequantize, fp4quant_encode, fp4quant_decode,
  fp4_errfeedback_qdq, mxfp4_row_to_fp8_col, mxfp4_row_to_fp8_col_tokblk,
  mxfp4_row_to_fp8_row
and in include/fp4mi_ops.h:
  mxfp4_matmul, mxfp4_matmul_grouped, fp8_matmul_tokblk, rmsnorm_quantize,
  rmsnorm_backward
plus ErrorFeedback, a name-keyed holder of residual buffers in the style of
the fp4-train page's ErrorFeedback.qdq(name, x, step).
"""
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfp4mi.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with "
                      "`python __graft_entry__.py` or `python block_scaled_fp4_amd/build.py` (hipcc, gfx950)")

_lib = ctypes.CDLL(LIB_PATH)

# ---- constants (mirror include/fp4mi.h)
FP4_OK, FP4_EINVAL, FP4_ESHAPE, FP4_EALIGN, FP4_EDTYPE, FP4_EHIP, FP4_EOVERLAP = range(7)
DTYPE = {torch.float32: 0, torch.bfloat16: 1}
FMT = {"nvfp4": 0, "mxfp4": 1}
ROUND = {"rtn": 0, "sr": 1}
TSCALE = {"compute": 0, "given": 1}
ROWS = {"mxfp4": 0, "fp8": 1}

_p, _i, _i32, _i64, _u64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64
_f = ctypes.c_float
_SIGS = {
    "fp4_quantize": [_p, _i, _i64, _i64, _i, _i, _u64, _u64, _i, _p, _p, _p, _p],
    "fp4_dequantize": [_p, _p, _p, _i64, _i64, _i, _p, _i, _p],
    "fp4quant_encode": [_p, _i, _i64, _i64, _i32, _p, _p, _p, _p],
    "fp4quant_encode_ex": [_p, _i, _i64, _i64, _i32, _i, _u64, _u64, _p, _p, _p, _p],
    "fp4quant_decode": [_p, _p, _p, _i64, _i64, _i32, _p, _i, _p],
    "fp4_errfeedback_qdq": [_p, _i, _i64, _i64, _p, _p, _i, _i, _u64, _u64, _i, _p, _p, _p, _p],
    "mxfp4_row_to_fp8_col": [_p, _p, _p, _i32, _i64, _i64, _p, _p, _p],
    "mxfp4_row_to_fp8_col_tokblk": [_p, _p, _p, _i32, _i64, _i64, _p, _p, _p],
    "mxfp4_row_to_fp8_row": [_p, _p, _i64, _i64, _p, _p, _p],
    "mxfp4_matmul": [_p, _i, _p, _p, _p, _p, _i64, _i64, _i64, _p, _i, _p],
    "mxfp4_matmul_grouped": [_p, _i, _p, _p, _p, _p, _p, _i32, _i64, _i64, _i64, _p, _i, _p],
    "fp8_matmul_tokblk": [_p, _p, _p, _p, _p, _i32, _i64, _i64, _i64, _p, _i, _p],
    "rmsnorm_quantize": [_p, _p, _i, _p, _i, _i64, _i64, _f, _i, _p, _p, _p, _p, _p],
    "rmsnorm_backward": [_p, _p, _p, _i, _p, _i, _p, _i64, _i64, _p, _p, _p, _i64, _p],
}
for _name, _args in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.argtypes = _args
    _fn.restype = ctypes.c_int
_lib.rmsnorm_backward_workspace.argtypes = [_i64, _i64]
_lib.rmsnorm_backward_workspace.restype = ctypes.c_int64
_lib.fp4_status_string.argtypes = [ctypes.c_int]
_lib.fp4_status_string.restype = ctypes.c_char_p
_lib.fp4_abi_version.argtypes = []
_lib.fp4_abi_version.restype = ctypes.c_int


class Fp4Error(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn}: {_lib.fp4_status_string(status).decode()} (status {status})")


def raw():
    """The ctypes handle of the library (for ABI-level tests)."""
    return _lib


def status_string(status):
    return _lib.fp4_status_string(status).decode()


def abi_version():
    return _lib.fp4_abi_version()


def _check(fn, status):
    if status != FP4_OK:
        raise Fp4Error(fn, status)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is None:   # torch.cuda.current_stream() without its Stream object, 0.3 us for 2.8
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def _on_stream(fn, args):
    """fn(**args), which has something to allocate, with args["stream"] (a Stream
    or a raw handle) as the current stream.  What fn allocates then comes from
    that stream's memory: a block from another stream's could still be in use
    there, and scratch would go back to it, for others to write, before the
    launches are done.  New outputs are recorded on the caller's stream as well,
    where they are read."""
    stream = args.pop("stream")
    if not isinstance(stream, torch.cuda.Stream):
        handle = getattr(stream, "cuda_stream", stream)
        handle = getattr(handle, "value", handle) or 0
        if handle == _stream(None):
            return fn(**args)
        stream = torch.cuda.ExternalStream(handle)
    elif stream.cuda_stream == _stream(None):
        return fn(**args)
    before = caller = torch.cuda.current_stream()
    if stream.device != before.device:   # a stream of another GPU: that one's current stream
        caller = torch.cuda.current_stream(stream.device)
    torch.cuda.set_stream(stream)
    try:
        out = fn(**args)
    finally:
        if caller is not before:
            torch.cuda.set_stream(caller)
        torch.cuda.set_stream(before)
    for t in out if isinstance(out, tuple) else (out,):
        if t is not None and not any(t is a for a in args.values()):
            t.record_stream(caller)
    return out


def _dtype_code(dt):
    return DTYPE.get(dt, 99)


def _dev(x):
    if not x.is_cuda:
        raise ValueError("tensors must be on the GPU")
    if not x.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return x


def _arg(t, name, dtype, numel, device, optional=False):
    """Checks a tensor argument the C ABI only sees as a pointer: same GPU as
    the main input, contiguous, of `dtype`, with at least `numel` elements
    (the library writes or reads exactly that many)."""
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name} is required")
    if not t.is_cuda or t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.numel() < numel:
        raise ValueError(f"{name} holds {t.numel()} elements, {numel} are needed")
    return t


def fp4_quantize(x, fmt="nvfp4", rounding="rtn", seed=0, step=0, tscale="compute",
                 tensor_scale=None, packed=None, scales=None, stream=None):
    """Quantize x [.., cols] -> (packed uint8 [rows, cols/2], scales uint8, tensor_scale).
    tensor_scale is a 1-element fp32 device tensor (NVFP4; None for MXFP4)."""
    if stream is not None and (packed is None or scales is None or (tensor_scale is None and fmt == "nvfp4")):
        return _on_stream(fp4_quantize, locals())
    _dev(x)
    cols = x.shape[-1]
    rows = x.numel() // cols if cols else 0
    blk = 32 if fmt == "mxfp4" else 16
    if packed is None:
        packed = torch.empty((rows, cols // 2), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((rows, cols // blk), dtype=torch.uint8, device=x.device)
    if fmt == "nvfp4" and tensor_scale is None:
        tensor_scale = torch.empty(1, dtype=torch.float32, device=x.device)
    _arg(packed, "packed", torch.uint8, rows * cols // 2, x.device)
    _arg(scales, "scales", torch.uint8, rows * cols // blk, x.device)
    _arg(tensor_scale, "tensor_scale", torch.float32, 1, x.device, optional=fmt == "mxfp4")
    _check("fp4_quantize", _lib.fp4_quantize(
        _ptr(x), _dtype_code(x.dtype), rows, cols, FMT[fmt], ROUND[rounding], seed, step,
        TSCALE[tscale], _ptr(tensor_scale), _ptr(packed), _ptr(scales), _stream(stream)))
    return packed, scales, tensor_scale


def fp4_dequantize(packed, scales, rows, cols, fmt="nvfp4", tensor_scale=None,
                   out_dtype=torch.bfloat16, y=None, stream=None):
    """Receiver: (packed, scales[, tensor_scale]) -> y [rows, cols] in out_dtype."""
    if stream is not None and y is None:
        return _on_stream(fp4_dequantize, locals())
    _dev(packed)
    if y is None:
        y = torch.empty((rows, cols), dtype=out_dtype, device=packed.device)
    blk = 32 if fmt == "mxfp4" else 16
    _arg(packed, "packed", torch.uint8, rows * cols // 2, packed.device)
    _arg(scales, "scales", torch.uint8, rows * cols // blk, packed.device)
    _arg(tensor_scale, "tensor_scale", torch.float32, 1, packed.device, optional=fmt == "mxfp4")
    _arg(y, "y", y.dtype, rows * cols, packed.device)
    _check("fp4_dequantize", _lib.fp4_dequantize(
        _ptr(packed), _ptr(scales), _ptr(tensor_scale), rows, cols, FMT[fmt], _ptr(y),
        _dtype_code(y.dtype), _stream(stream)))
    return y


def fp4quant_encode(x, group, packed=None, s_rms=None, s_abs=None, stream=None):
    """FP4Quant encode -> (packed [rows, cols/2], s_rms [rows, cols/G], s_abs [rows, cols/G])."""
    if stream is not None and (packed is None or s_rms is None or s_abs is None):
        return _on_stream(fp4quant_encode, locals())
    return _fq_encode("fp4quant_encode", x, group, None, 0, 0, packed, s_rms, s_abs, stream)


def fp4quant_encode_ex(x, group, rounding="sr", seed=0, step=0, packed=None, s_rms=None, s_abs=None,
                       stream=None):
    """FP4Quant encode with RTN or stochastic rounding keyed by (seed, step,
    element index) -> (packed, s_rms, s_abs) as fp4quant_encode."""
    if stream is not None and (packed is None or s_rms is None or s_abs is None):
        return _on_stream(fp4quant_encode_ex, locals())
    return _fq_encode("fp4quant_encode_ex", x, group, rounding, seed, step, packed, s_rms, s_abs,
                      stream)


def _fq_encode(fn, x, group, rounding, seed, step, packed, s_rms, s_abs, stream):
    _dev(x)
    cols = x.shape[-1]
    rows = x.numel() // cols if cols else 0
    if packed is None:
        packed = torch.empty((rows, cols // 2), dtype=torch.uint8, device=x.device)
    ng = cols // group if group > 0 else 0
    if s_rms is None:
        s_rms = torch.empty((rows, ng), dtype=torch.float32, device=x.device)
    if s_abs is None:
        s_abs = torch.empty((rows, ng), dtype=torch.float32, device=x.device)
    _arg(packed, "packed", torch.uint8, rows * cols // 2, x.device)
    _arg(s_rms, "s_rms", torch.float32, rows * ng, x.device)
    _arg(s_abs, "s_abs", torch.float32, rows * ng, x.device)
    if rounding is None:
        status = _lib.fp4quant_encode(_ptr(x), _dtype_code(x.dtype), rows, cols, group, _ptr(packed),
                                      _ptr(s_rms), _ptr(s_abs), _stream(stream))
    else:
        status = _lib.fp4quant_encode_ex(_ptr(x), _dtype_code(x.dtype), rows, cols, group,
                                         ROUND.get(rounding, 99), seed, step, _ptr(packed), _ptr(s_rms),
                                         _ptr(s_abs), _stream(stream))
    _check(fn, status)
    return packed, s_rms, s_abs


def fp4quant_decode(packed, s_rms, s_abs, rows, cols, group, out_dtype=torch.bfloat16, y=None,
                    stream=None):
    """FP4Quant receiver -> y [rows, cols]."""
    if stream is not None and y is None:
        return _on_stream(fp4quant_decode, locals())
    _dev(packed)
    if y is None:
        y = torch.empty((rows, cols), dtype=out_dtype, device=packed.device)
    ng = cols // group if group > 0 else 0
    _arg(packed, "packed", torch.uint8, rows * cols // 2, packed.device)
    _arg(s_rms, "s_rms", torch.float32, rows * ng, packed.device)
    _arg(s_abs, "s_abs", torch.float32, rows * ng, packed.device)
    _arg(y, "y", y.dtype, rows * cols, packed.device)
    _check("fp4quant_decode", _lib.fp4quant_decode(
        _ptr(packed), _ptr(s_rms), _ptr(s_abs), rows, cols, group, _ptr(y), _dtype_code(y.dtype),
        _stream(stream)))
    return y


def fp4_errfeedback_qdq(x, residual=None, y=None, out_dtype=None, rounding="sr", seed=0, step=0,
                        tscale="compute", tensor_scale=None, packed=None, scales=None,
                        stream=None):
    """NVFP4 qdq with an fp32 error-feedback residual (updated in place).
    Returns (y, tensor_scale).  y may be x for an in-place update."""
    if stream is not None and (y is None or tensor_scale is None):
        return _on_stream(fp4_errfeedback_qdq, locals())
    _dev(x)
    cols = x.shape[-1]
    rows = x.numel() // cols if cols else 0
    if y is None:
        y = torch.empty(x.shape, dtype=out_dtype or x.dtype, device=x.device)
    if tensor_scale is None:
        tensor_scale = torch.empty(1, dtype=torch.float32, device=x.device)
    n = rows * cols
    _arg(residual, "residual", torch.float32, n, x.device, optional=True)
    _arg(y, "y", y.dtype, n, x.device)
    _arg(tensor_scale, "tensor_scale", torch.float32, 1, x.device)
    _arg(packed, "packed", torch.uint8, n // 2, x.device, optional=True)
    _arg(scales, "scales", torch.uint8, n // 16, x.device, optional=True)
    _check("fp4_errfeedback_qdq", _lib.fp4_errfeedback_qdq(
        _ptr(x), _dtype_code(x.dtype), rows, cols, _ptr(residual), _ptr(y), _dtype_code(y.dtype),
        ROUND[rounding], seed, step, TSCALE[tscale], _ptr(tensor_scale), _ptr(packed),
        _ptr(scales), _stream(stream)))
    return y, tensor_scale


def mxfp4_row_to_fp8_col(packed, scales_e8m0, token_offsets, hidden, fp8_out=None,
                         fp8_scales=None, stream=None):
    """Ragged MXFP4 rows [T, H/2] (+ UE8M0 [T, H/32]) -> per-expert FP8 E4M3
    columns (flat uint8 [T*H]) and fp32 block scales (flat [T*H/128])."""
    if stream is not None and (fp8_out is None or fp8_scales is None):
        return _on_stream(mxfp4_row_to_fp8_col, locals())
    _dev(packed)
    T = packed.shape[0]
    E = token_offsets.numel() - 1
    if fp8_out is None:
        fp8_out = torch.empty(T * hidden, dtype=torch.uint8, device=packed.device)
    if fp8_scales is None:
        fp8_scales = torch.empty(T * hidden // 128, dtype=torch.float32, device=packed.device)
    _arg(packed, "packed", torch.uint8, T * hidden // 2, packed.device)
    _arg(scales_e8m0, "scales_e8m0", torch.uint8, T * hidden // 32, packed.device)
    _arg(token_offsets, "token_offsets", torch.int64, 1, packed.device)
    _arg(fp8_out, "fp8_out", torch.uint8, T * hidden, packed.device)
    _arg(fp8_scales, "fp8_scales", torch.float32, T * hidden // 128, packed.device)
    _check("mxfp4_row_to_fp8_col", _lib.mxfp4_row_to_fp8_col(
        _ptr(packed), _ptr(scales_e8m0), _ptr(token_offsets), E, T, hidden, _ptr(fp8_out),
        _ptr(fp8_scales), _stream(stream)))
    return fp8_out, fp8_scales


def tokblk_scale_count(total_tokens, num_experts, hidden):
    """fp32 elements of the token-block scale buffer: H (ceil(T / 128) + E)."""
    return hidden * ((total_tokens + 127) // 128 + num_experts)


def mxfp4_row_to_fp8_col_tokblk(packed, scales_e8m0, token_offsets, hidden, fp8_out=None,
                                fp8_scales=None, stream=None):
    """Ragged MXFP4 rows [T, H/2] (+ UE8M0 [T, H/32]) -> per-expert FP8 E4M3
    columns (flat uint8 [T*H]) with FP8 blocks of 128 tokens per channel, and
    fp32 scales (flat [H (ceil(T/128) + E)]; expert e's [H, ceil(n_e/128)]
    matrix at element H (ceil(off_e/128) + e))."""
    if stream is not None and (fp8_out is None or fp8_scales is None):
        return _on_stream(mxfp4_row_to_fp8_col_tokblk, locals())
    _dev(packed)
    T = packed.shape[0]
    E = token_offsets.numel() - 1
    nsc = tokblk_scale_count(T, E, hidden)
    if fp8_out is None:
        fp8_out = torch.empty(T * hidden, dtype=torch.uint8, device=packed.device)
    if fp8_scales is None:
        fp8_scales = torch.empty(nsc, dtype=torch.float32, device=packed.device)
    _arg(packed, "packed", torch.uint8, T * hidden // 2, packed.device)
    _arg(scales_e8m0, "scales_e8m0", torch.uint8, T * hidden // 32, packed.device)
    _arg(token_offsets, "token_offsets", torch.int64, 1, packed.device)
    _arg(fp8_out, "fp8_out", torch.uint8, T * hidden, packed.device)
    _arg(fp8_scales, "fp8_scales", torch.float32, nsc, packed.device)
    _check("mxfp4_row_to_fp8_col_tokblk", _lib.mxfp4_row_to_fp8_col_tokblk(
        _ptr(packed), _ptr(scales_e8m0), _ptr(token_offsets), E, T, hidden, _ptr(fp8_out),
        _ptr(fp8_scales), _stream(stream)))
    return fp8_out, fp8_scales


def mxfp4_row_to_fp8_row(packed, scales_e8m0, hidden, fp8_out=None, fp8_scales=None,
                         stream=None):
    """MXFP4 rows [T, H/2] (+ UE8M0 [T, H/32]) -> FP8 E4M3 rows [T, H] and
    fp32 block scales [T, H/128] (no transpose)."""
    if stream is not None and (fp8_out is None or fp8_scales is None):
        return _on_stream(mxfp4_row_to_fp8_row, locals())
    _dev(packed)
    T = packed.shape[0]
    if fp8_out is None:
        fp8_out = torch.empty((T, hidden), dtype=torch.uint8, device=packed.device)
    if fp8_scales is None:
        fp8_scales = torch.empty((T, hidden // 128), dtype=torch.float32, device=packed.device)
    _arg(packed, "packed", torch.uint8, T * hidden // 2, packed.device)
    _arg(scales_e8m0, "scales_e8m0", torch.uint8, T * hidden // 32, packed.device)
    _arg(fp8_out, "fp8_out", torch.uint8, T * hidden, packed.device)
    _arg(fp8_scales, "fp8_scales", torch.float32, T * hidden // 128, packed.device)
    _check("mxfp4_row_to_fp8_row", _lib.mxfp4_row_to_fp8_row(
        _ptr(packed), _ptr(scales_e8m0), T, hidden, _ptr(fp8_out), _ptr(fp8_scales),
        _stream(stream)))
    return fp8_out, fp8_scales


def _fits(t, dtype, numel, gpu):
    """_arg's conditions for a tensor on GPU number `gpu`, without its messages."""
    return t.dtype is dtype and t.get_device() == gpu and t.is_contiguous() and t.numel() >= numel


def _codes(t):
    """E4M3 codes as bytes, whichever dtype they came in."""
    return t.view(torch.uint8) if t.dtype is torch.float8_e4m3fn else t


def _product(name, a, a_scales, a_row_scale, w, w_scales, offsets, out_dtype, out, stream):
    """Checks and launches either product (small sizes are over in the time
    that a call takes here, so the common case is one run of plain tests)."""
    a = _codes(a)
    shape, gpu = a.shape, a.get_device()
    fp8 = a_scales.dtype is torch.float32
    width, N, kb = shape[-1], w.shape[-2], w.shape[-1]
    M = a.numel() // width if width else 0
    K = 2 * kb
    E = 1 if offsets is None else w.shape[0]
    if (width if fp8 else 2 * width) != K:
        raise ValueError(f"a has {width if fp8 else 2 * width} columns, the weights have {K}")
    if out is None:
        out = a.new_empty((M, N) if len(shape) == 2 else (*shape[:-1], N), dtype=out_dtype)
    sdt, sn = (torch.float32, M * (K // 128)) if fp8 else (torch.uint8, M * (K // 32))
    if not (gpu >= 0 and _fits(a, torch.uint8, M * width, gpu) and _fits(a_scales, sdt, sn, gpu)
            and _fits(w, torch.uint8, E * N * kb, gpu) and _fits(w_scales, torch.uint8, E * N * (K // 32), gpu)
            and _fits(out, out.dtype, M * N, gpu)
            and (a_row_scale is None or _fits(a_row_scale, torch.float32, M, gpu))
            and (offsets is None or _fits(offsets, torch.int64, E + 1, gpu))):
        _dev(a)
        _arg(a, "a", torch.uint8, M * width, a.device)
        _arg(a_scales, "a_scales", sdt, sn, a.device)
        _arg(w, "w", torch.uint8, E * N * kb, a.device)
        _arg(w_scales, "w_scales", torch.uint8, E * N * (K // 32), a.device)
        _arg(out, "out", out.dtype, M * N, a.device)
        _arg(a_row_scale, "a_row_scale", torch.float32, M, a.device, optional=True)
        _arg(offsets, "token_offsets", torch.int64, E + 1, a.device, optional=True)
    row = None if a_row_scale is None else a_row_scale.data_ptr()
    if offsets is None:
        status = _lib.mxfp4_matmul(a.data_ptr(), fp8, a_scales.data_ptr(), row, w.data_ptr(),
                                   w_scales.data_ptr(), M, N, K, out.data_ptr(),
                                   _dtype_code(out.dtype), _stream(stream))
    else:
        status = _lib.mxfp4_matmul_grouped(a.data_ptr(), fp8, a_scales.data_ptr(), row, w.data_ptr(),
                                           w_scales.data_ptr(), offsets.data_ptr(), E, M, N, K,
                                           out.data_ptr(), _dtype_code(out.dtype), _stream(stream))
    _check(name, status)
    return out


def mxfp4_matmul(a, a_scales, b, b_scales, a_row_scale=None, out_dtype=torch.bfloat16, out=None,
                 stream=None):
    """a [.., K] . b [N, K]^T -> [.., N] in out_dtype (or out's dtype).

    a is MXFP4 (uint8 [.., K/2] with UE8M0 uint8 scales) or FP8 rows (E4M3
    [.., K], uint8 or float8_e4m3fn, with power-of-two fp32 scales [.., K/128]):
    the scales' dtype tells.  b is MXFP4 [N, K/2].  a_row_scale: fp32 factor
    per row of a, such as rmsnorm_quantize's row_scale."""
    if stream is not None and out is None:
        return _on_stream(mxfp4_matmul, locals())
    if b.dim() != 2:
        raise ValueError("b must be [N, K/2]")
    return _product("mxfp4_matmul", a, a_scales, a_row_scale, b, b_scales, None, out_dtype, out, stream)


def mxfp4_matmul_grouped(a, a_scales, w, w_scales, token_offsets, a_row_scale=None,
                         out_dtype=torch.bfloat16, out=None, stream=None):
    """Rows token_offsets[e] .. token_offsets[e+1]-1 of a [T, K] times w[e]^T,
    w MXFP4 [E, N, K/2] -> [T, N].  Operands as mxfp4_matmul."""
    if stream is not None and out is None:
        return _on_stream(mxfp4_matmul_grouped, locals())
    if w.dim() != 3:
        raise ValueError("w must be [E, N, K/2]")
    if token_offsets is None:
        raise ValueError("token_offsets is required")
    return _product("mxfp4_matmul_grouped", a, a_scales, a_row_scale, w, w_scales, token_offsets,
                    out_dtype, out, stream)


def fp8_matmul_tokblk(a, a_scales, b, b_scales, token_offsets, m, n, out_dtype=torch.bfloat16,
                      out=None, stream=None):
    """Per-expert weight gradient A_e [m, n_e] . B_e [n, n_e]^T -> [E, m, n].

    Operands as mxfp4_row_to_fp8_col_tokblk returns them (flat E4M3 columns and
    flat fp32 scales) for hidden sizes m and n and the same token_offsets.  A
    factor that the rows of b were used with (a_row_scale) has to be in a."""
    if stream is not None and out is None:
        return _on_stream(fp8_matmul_tokblk, locals())
    a, b = _codes(a), _codes(b)
    gpu, T, E = a.get_device(), a.numel() // m if m else 0, token_offsets.numel() - 1
    na, nb = tokblk_scale_count(T, E, m), tokblk_scale_count(T, E, n)
    if out is None:
        out = a.new_empty((E, m, n), dtype=out_dtype)
    if not (gpu >= 0 and _fits(a, torch.uint8, T * m, gpu) and _fits(b, torch.uint8, T * n, gpu)
            and _fits(a_scales, torch.float32, na, gpu) and _fits(b_scales, torch.float32, nb, gpu)
            and _fits(token_offsets, torch.int64, 1, gpu) and _fits(out, out.dtype, E * m * n, gpu)):
        _dev(a)
        _arg(a, "a", torch.uint8, T * m, a.device)
        _arg(b, "b", torch.uint8, T * n, a.device)
        _arg(a_scales, "a_scales", torch.float32, na, a.device)
        _arg(b_scales, "b_scales", torch.float32, nb, a.device)
        _arg(token_offsets, "token_offsets", torch.int64, 1, a.device)
        _arg(out, "out", out.dtype, E * m * n, a.device)
    _check("fp8_matmul_tokblk", _lib.fp8_matmul_tokblk(
        a.data_ptr(), a_scales.data_ptr(), b.data_ptr(), b_scales.data_ptr(),
        token_offsets.data_ptr(), E, T, m, n, out.data_ptr(), _dtype_code(out.dtype),
        _stream(stream)))
    return out


def rmsnorm_quantize(x, weight, residual=None, eps=1e-6, fmt="fp8", q=None, scales=None,
                     row_scale=None, h=None, stream=None):
    """RMS norm of h = x + residual over the last axis, as quantized rows
    -> (q, scales, row_scale, h).

    fmt "mxfp4": q uint8 [.., cols/2], scales UE8M0 uint8 [.., cols/32]; "fp8":
    q E4M3 uint8 [.., cols], scales fp32 [.., cols/128].  The rows hold
    h * weight; row_scale (fp32, one per row) is 1 / rms, the a_row_scale of
    the products, and a factor of dY's rows in the weight gradient.  Without a
    residual, and without an h to fill, h is x."""
    if stream is not None and (q is None or scales is None or row_scale is None or
                               (h is None and residual is not None)):
        return _on_stream(rmsnorm_quantize, locals())
    shape, gpu, dt = x.shape, x.get_device(), x.dtype
    cols = shape[-1]
    rows = x.numel() // cols if cols else 0
    lead, fp8 = shape[:-1], fmt == "fp8"
    per, block, sdt = (1, 128, torch.float32) if fp8 else (2, 32, torch.uint8)
    if q is None:
        q = (torch.empty_like(x, dtype=torch.uint8) if fp8 else
             x.new_empty((*lead, cols // 2), dtype=torch.uint8))
    if scales is None:
        scales = x.new_empty((*lead, cols // block), dtype=sdt)
    if row_scale is None:
        row_scale = x.new_empty(lead, dtype=torch.float32)
    if h is None and residual is not None:
        h = torch.empty_like(x)
    n = rows * cols
    if not (gpu >= 0 and _fits(x, dt, n, gpu) and _fits(q, torch.uint8, n // per, gpu)
            and _fits(scales, sdt, rows * (cols // block), gpu) and _fits(row_scale, torch.float32, rows, gpu)
            and (residual is None or _fits(residual, dt, n, gpu)) and (h is None or _fits(h, dt, n, gpu))
            and _fits(weight, weight.dtype, cols, gpu)):
        _dev(x)
        _arg(q, "q", torch.uint8, n // per, x.device)
        _arg(scales, "scales", sdt, rows * (cols // block), x.device)
        _arg(row_scale, "row_scale", torch.float32, rows, x.device)
        _arg(residual, "residual", dt, n, x.device, optional=True)
        _arg(h, "h", dt, n, x.device, optional=True)
        _arg(weight, "weight", weight.dtype, cols, x.device)
    _check("rmsnorm_quantize", _lib.rmsnorm_quantize(
        x.data_ptr(), _ptr(residual), _dtype_code(dt), weight.data_ptr(), _dtype_code(weight.dtype),
        rows, cols, eps, ROWS.get(fmt, 99), q.data_ptr(), scales.data_ptr(), row_scale.data_ptr(),
        _ptr(h), _stream(stream)))
    return q, scales, row_scale, x if h is None else h


def rmsnorm_backward(dy, h, weight, row_scale, dh=None, dx=None, dweight=None, workspace=None,
                     stream=None):
    """Gradient of row_scale * h * weight -> (dx, dweight fp32 [cols]); dh, if
    given, is added to dx.  workspace: uint8 of at least
    rmsnorm_backward_workspace(rows, cols) elements (allocated if None)."""
    if stream is not None and (dx is None or dweight is None or workspace is None):
        return _on_stream(rmsnorm_backward, locals())
    gpu, dt, cols = dy.get_device(), dy.dtype, dy.shape[-1]
    rows = dy.numel() // cols if cols else 0
    n, need = rows * cols, _lib.rmsnorm_backward_workspace(rows, cols)
    if dx is None:
        dx = torch.empty_like(dy)
    if dweight is None:
        dweight = dy.new_empty(cols, dtype=torch.float32)
    if workspace is None:
        workspace = dy.new_empty(need, dtype=torch.uint8)
    if not (gpu >= 0 and _fits(dy, dt, n, gpu) and _fits(h, dt, n, gpu) and _fits(dx, dt, n, gpu)
            and (dh is None or _fits(dh, dt, n, gpu)) and _fits(weight, weight.dtype, cols, gpu)
            and _fits(row_scale, torch.float32, rows, gpu) and _fits(dweight, torch.float32, cols, gpu)
            and _fits(workspace, torch.uint8, need, gpu)):
        _dev(dy)
        _arg(h, "h", dt, n, dy.device)
        _arg(dh, "dh", dt, n, dy.device, optional=True)
        _arg(dx, "dx", dt, n, dy.device)
        _arg(weight, "weight", weight.dtype, cols, dy.device)
        _arg(row_scale, "row_scale", torch.float32, rows, dy.device)
        _arg(dweight, "dweight", torch.float32, cols, dy.device)
        _arg(workspace, "workspace", torch.uint8, need, dy.device)
    _check("rmsnorm_backward", _lib.rmsnorm_backward(
        dy.data_ptr(), h.data_ptr(), _ptr(dh), _dtype_code(dt), weight.data_ptr(),
        _dtype_code(weight.dtype), row_scale.data_ptr(), rows, cols, dx.data_ptr(),
        dweight.data_ptr(), workspace.data_ptr(), workspace.numel(), _stream(stream)))
    return dx, dweight


def rmsnorm_backward_workspace(rows, cols):
    """Bytes of rmsnorm_backward's workspace."""
    return _lib.rmsnorm_backward_workspace(rows, cols)


class ErrorFeedback:
    """Residual holder keyed by tensor name (fp4-train, "Usage").

    qdq(name, x, step) runs fp4_errfeedback_qdq with the residual kept for
    `name` (created as zeros on first use) and returns the new bf16/fp32
    tensor in x's dtype."""

    def __init__(self, stochastic=False, seed=0):
        self.rounding = "sr" if stochastic else "rtn"
        self.seed = seed
        self.residuals = {}

    def qdq(self, name, x, step, out=None):
        r = self.residuals.get(name)
        if r is None or r.shape != x.shape:
            r = torch.zeros(x.shape, dtype=torch.float32, device=x.device)
            self.residuals[name] = r
        y, _ = fp4_errfeedback_qdq(x, residual=r, y=out, rounding=self.rounding, seed=self.seed,
                                   step=step)
        return y
