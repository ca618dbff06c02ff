"""4-bit weights with group scales: tensors in, tensors out.

Over the C ABI of ``include/gemm_nt_w4.h``, which defines the packed layout,
the rounding and the limits.  A call is enqueued on ``stream`` (default: the
current stream of the tensors' device); tensors that it makes are that stream's.
"""
from __future__ import annotations

import math
from contextlib import nullcontext

from . import binding
from .binding import GEMM_OK, GemmError

_DTYPES = None
_HERE = nullcontext()


def dtype_code(dtype) -> int:
    """GEMM_T_* of a torch dtype; TypeError for any other than the two."""
    global _DTYPES
    if _DTYPES is None:
        import torch
        _DTYPES = {torch.float16: binding.GEMM_T_F16, torch.bfloat16: binding.GEMM_T_BF16}
    try:
        return _DTYPES[dtype]
    except KeyError:
        raise TypeError(f"unsupported dtype {dtype}: float16 or bfloat16") from None


def stream_of(device, stream) -> int:
    """The raw handle of ``stream``, or of the device's current stream."""
    import torch
    if stream is not None:
        return stream.cuda_stream
    # torch.cuda.current_stream would build an object around it: 2 us
    return torch._C._cuda_getCurrentRawStream(device.index)


def on_stream(stream):
    """Allocations inside are ``stream``'s: the memory of a tensor made for another
    stream may still be in use on this one."""
    if stream is None:
        return _HERE
    import torch
    return torch.cuda.stream(stream)


def on_device(device):
    """``device`` is the current one inside."""
    import torch
    return _HERE if device.index == torch.cuda.current_device() else torch.cuda.device(device)


def launch(name: str, device, args) -> None:
    """The raw entry point ``name`` with ``args`` on ``device``."""
    fn = getattr(binding.lib(), name)
    # the library launches on the current device: make it the operands' one
    with on_device(device):
        rc = fn(*args)
    if rc != GEMM_OK:
        raise GemmError(rc, name)


def row_stride(x, what: str) -> int:
    """Elements between the rows of a 2-D tensor whose rows are dense."""
    rows, cols = x.shape
    if x.is_contiguous():
        return cols
    if cols > 1 and x.stride(1) != 1:
        raise ValueError(f"{what} must have dense rows")
    ld = x.stride(0) if rows > 1 else cols
    if ld < cols:
        raise ValueError(f"the rows of {what} overlap")
    return ld


def check_out(out, shape, dtype, device) -> None:
    if out.dtype != dtype or tuple(out.shape) != tuple(shape) or out.device != device:
        raise ValueError(f"out must be a {dtype} tensor of shape {tuple(shape)} on {device}")


class W4Weight:
    """A packed weight [..., N, K]: ``q`` (int32 words [..., N, ceil(K / 128) * 16]),
    ``scales`` [..., N, ceil(K / group)] in float16 or bfloat16 and ``zeros`` of that
    shape (uint8), or None for zero points of 8; all contiguous, on one GPU."""

    __slots__ = ("q", "scales", "zeros", "shape", "group", "dtype", "device", "N", "K", "code",
                 "pointers")

    def __init__(self, q, scales, zeros=None, *, shape, group):
        import torch
        shape = tuple(int(n) for n in shape)
        if group not in (32, 64, 128):
            raise ValueError(f"group {group} is not 32, 64 or 128")
        if len(shape) < 2:
            raise ValueError(f"shape {shape} is not [..., N, K]")
        K = shape[-1]
        dtype_code(scales.dtype)
        want = {"q": (q, torch.int32, -(-K // 128) * 16),
                "scales": (scales, scales.dtype, -(-K // group))}
        if zeros is not None:
            want["zeros"] = (zeros, torch.uint8, -(-K // group))
        for name, (x, dtype, last) in want.items():
            if x.dtype != dtype or tuple(x.shape) != shape[:-1] + (last,):
                raise ValueError(f"{name} must be a {dtype} tensor of shape "
                                 f"{shape[:-1] + (last,)}, not {x.dtype} {tuple(x.shape)}")
            if not x.is_contiguous() or not x.is_cuda or x.device != q.device:
                raise ValueError(f"{name} must be contiguous, on the GPU of q")
        self._hold(q, scales, zeros, shape, group)

    def _hold(self, q, scales, zeros, shape, group):
        self.q, self.scales, self.zeros = q, scales, zeros
        self.shape, self.group = shape, group
        self.dtype, self.device = scales.dtype, q.device
        self.code = dtype_code(scales.dtype)
        self.N, self.K = math.prod(shape[:-1]), shape[-1]
        self.pointers = (q.data_ptr(), scales.data_ptr(),
                         zeros.data_ptr() if zeros is not None else None)


def quantize_w4(W, group: int = 128, zeros: bool = False, stream=None) -> W4Weight:
    """``W`` [..., N, K] (float16 or bfloat16) in 4 bits with a scale per ``group``
    elements of a row, and with ``zeros`` a zero point (otherwise symmetric).  A 2-D
    W may have a row stride; with more dimensions it is contiguous."""
    import torch
    code = dtype_code(W.dtype)
    if W.dim() < 2:
        raise ValueError(f"shape {tuple(W.shape)} is not [..., N, K]")
    if not W.is_cuda:
        raise ValueError("W must be on a GPU")
    if W.dim() > 2 and not W.is_contiguous():
        raise ValueError("W must be contiguous")
    if group not in (32, 64, 128):
        raise ValueError(f"group {group} is not 32, 64 or 128")
    shape = tuple(W.shape)
    K, lead, device = shape[-1], shape[:-1], W.device
    ldw = row_stride(W, "W") if len(shape) == 2 else K
    groups = lead + (-(-K // group),)
    w = W4Weight.__new__(W4Weight)
    with on_stream(stream):
        w._hold(torch.empty(lead + (-(-K // 128) * 16,), dtype=torch.int32, device=device),
                W.new_empty(groups),
                torch.empty(groups, dtype=torch.uint8, device=device) if zeros else None,
                shape, group)
    q, s, z = w.pointers
    launch("gemm_w4_quantize", device, (W.data_ptr(), q, s, z, w.N, K, ldw, group, code,
                                        stream_of(device, stream)))
    return w


def dequantize_w4(w: W4Weight, out=None, stream=None):
    """The values of ``w``, rounded to its 16-bit type, in its shape.  ``out``
    (optional): 2-D with a row stride, or contiguous."""
    if out is None:
        with on_stream(stream):
            out = w.scales.new_empty(w.shape)
    else:
        check_out(out, w.shape, w.dtype, w.device)
        if out.dim() > 2 and not out.is_contiguous():
            raise ValueError("out must be contiguous")
    ldw = row_stride(out, "out") if out.dim() == 2 else w.K
    launch("gemm_w4_dequantize", w.device, (*w.pointers, out.data_ptr(), w.N, w.K, ldw, w.group,
                                            w.code, stream_of(w.device, stream)))
    return out


def gemm_nt_w4(A, w: W4Weight, out=None, stream=None, workspace=None):
    """D = A @ W.T for ``A`` [M, K] in the weight's 16-bit type and a 2-D ``w`` [N, K].

    A and ``out`` (optional, [M, N]) may have a row stride.  ``workspace`` (optional):
    a contiguous uint8 tensor for the unpacked weight of large M, allocated here where
    it is needed and none is given."""
    import torch
    N, K, device = w.N, w.K, w.device
    if len(w.shape) != 2 or A.dim() != 2 or A.shape[1] != K:
        raise ValueError(f"shapes {tuple(A.shape)} and {w.shape} are not [M, K] and [N, K]")
    if A.dtype != w.dtype:
        raise TypeError(f"A is {A.dtype}, the weight's scales are {w.dtype}")
    if A.device != device:
        raise ValueError("A and the weight must be on the same GPU")
    M = A.shape[0]
    lda = row_stride(A, "A")
    if out is None:
        with on_stream(stream):
            out, ldd = A.new_empty((M, N)), N
    else:
        check_out(out, (M, N), A.dtype, device)
        ldd = row_stride(out, "out")
    ws = ws_bytes = 0
    if workspace is None:
        need = binding.lib().gemm_nt_w4_ws_size(M, N, K) if lda == K and ldd == N else 0
        if need:
            with on_stream(stream):
                workspace = torch.empty(need, dtype=torch.uint8, device=device)
    elif workspace.device != device or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous, on A's device")
    if workspace is not None:
        ws, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    launch("gemm_nt_w4", device, (A.data_ptr(), *w.pointers, out.data_ptr(), M, N, K, lda, ldd,
                                  w.group, w.code, ws, ws_bytes, stream_of(device, stream)))
    return out
