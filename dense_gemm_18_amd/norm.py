"""The root-mean-square norm with the residual's addition: tensors in, tensors out.

Over the C ABI of ``include/rms_norm.h``, which defines the formulas, the
rounding and the limits.  A call is enqueued on ``stream`` (default: the current
stream of the tensors' device); tensors that it makes are that stream's.
"""
from __future__ import annotations

from . import binding
from .w4 import check_out, dtype_code, launch, new_rows, on_stream, row_stride, stream_of

_FORMATS = None


def _format(dtype) -> int:
    """GEMM_FP8_* of a torch dtype; TypeError for any other than the two."""
    global _FORMATS
    if _FORMATS is None:
        import torch
        _FORMATS = {torch.float8_e4m3fn: binding.GEMM_FP8_E4M3,
                    torch.float8_e5m2: binding.GEMM_FP8_E5M2}
    try:
        return _FORMATS[dtype]
    except KeyError:
        raise TypeError(f"unsupported dtype {dtype}: float8_e4m3fn or float8_e5m2") from None


def _rows(x, weight, residual, residual_out, stream):
    """Checked operands: (type code, device, T, H, ldx, residual address, its stride, weight
    address, the tensor for s or None, its address, its stride)."""
    dtype, shape, device = x.dtype, x.shape, x.device
    code = dtype_code(dtype)
    if len(shape) != 2 or not shape[1]:
        raise ValueError(f"shape {tuple(shape)} is not [T, H]")
    if not x.is_cuda:
        raise ValueError("x must be on a GPU")
    T, H = shape
    w = r = s = None
    if weight is not None:
        if weight.dtype != dtype:
            raise TypeError(f"x is {dtype}, the weight {weight.dtype}")
        if weight.shape != (H,) or not weight.is_contiguous() or weight.device != device:
            raise ValueError(f"the weight must be a contiguous tensor of {H} elements on x's GPU")
        w = weight.data_ptr()
    ldx = ldr = lds = H
    if not x.is_contiguous():
        ldx = row_stride(x, "x")
    if residual is not None:
        if residual.dtype != dtype:
            raise TypeError(f"x is {dtype}, the residual {residual.dtype}")
        if residual.shape != shape or residual.device != device:
            raise ValueError(f"the residual must be of shape {tuple(shape)}, on x's GPU")
        r = residual.data_ptr()
        if not residual.is_contiguous():
            ldr = row_stride(residual, "residual")
        if residual_out is None:
            residual_out = new_rows(x, T, H, stream)
        else:
            check_out(residual_out, shape, dtype, device)
            lds = row_stride(residual_out, "residual_out")
        s = residual_out.data_ptr()
    elif residual_out is not None:
        raise ValueError("residual_out without a residual")
    return code, device, T, H, ldx, r, ldr, w, residual_out, s, lds


def rms_norm(x, weight=None, eps: float = 1e-6, residual=None, out=None, residual_out=None,
             stream=None):
    """y = s / sqrt(mean(s^2) + eps) * weight for each row of ``x`` [T, H] (float16 or
    bfloat16), where s = x + ``residual`` (optional, like x) and ``weight`` [H] is of x's
    type or None (ones).  Returns y, or with a residual (y, s), both in x's type.

    All may have a row stride.  ``out`` and ``residual_out`` (optional) take the results;
    each may be x or the residual itself."""
    code, device, T, H, ldx, r, ldr, w, total, s, lds = _rows(x, weight, residual, residual_out,
                                                              stream)
    if out is None:
        out, ldy = new_rows(x, T, H, stream), H
    else:
        check_out(out, (T, H), x.dtype, device)
        ldy = row_stride(out, "out")
    launch("rms_norm", device, (x.data_ptr(), r, w, out.data_ptr(), s, T, H, ldx, ldr, ldy, lds,
                                eps, code, stream_of(device, stream)))
    return out if s is None else (out, total)


def rms_norm_fp8(x, weight=None, eps: float = 1e-6, residual=None, dtype=None, scale=None,
                 out=None, residual_out=None, stream=None):
    """`rms_norm` into 8 bits: (q, scales), or with a residual (q, scales, s).  q [T, H] is
    of ``dtype`` (float8_e4m3fn, the default, or float8_e5m2) and scales [T] (float32) hold
    max|y| / largest number of each row, so that y is q * scales[:, None]: what
    ``gemm_nt`` takes as A and ``a_scale``.  With a number as ``scale`` all rows go by it
    and scales is that number: ``gemm_nt``'s ``scale``."""
    import torch
    if dtype is None:
        dtype = torch.float8_e4m3fn
    fmt = _format(dtype)
    code, device, T, H, ldx, r, ldr, w, total, s, lds = _rows(x, weight, residual, residual_out,
                                                              stream)
    with on_stream(stream):
        if out is None:
            out, ldq = torch.empty(T, H, dtype=dtype, device=device), H
        else:
            check_out(out, (T, H), dtype, device)
            ldq = row_stride(out, "out")
        scales = torch.empty(T, dtype=torch.float32, device=device) if scale is None else None
    launch("rms_norm_fp8", device,
           (x.data_ptr(), r, w, out.data_ptr(), None if scales is None else scales.data_ptr(), s,
            T, H, ldx, ldr, ldq, lds, eps, 0.0 if scale is None else scale, fmt, code,
            stream_of(device, stream)))
    held = scale if scales is None else scales
    return (out, held) if s is None else (out, held, total)
