"""Low-rank adapters beside a shared projection: tensors in, tensors out.

Over the C ABI of ``include/lora_nt.h``, which defines the product, its rounding
and its limits.  A call is enqueued on ``stream`` (default: the current stream of
the tensors' device); tensors that it makes are that stream's.
"""
from __future__ import annotations

import ctypes
import functools

from . import binding
from .w4 import (W4Weight, check_out, dtype_code, launch, new_rows, on_stream, row_stride,
                 stream_of)


class LoraAdapters:
    """``A`` [count, rank, K] and ``B`` [count, N, rank] in float16 or bfloat16 and
    ``scales`` [count] (float32), or None for 1: adapter a adds
    scales[a] * (x @ A[a].T) @ B[a].T.  All contiguous, on one GPU; kept, not copied.  An
    adapter of a smaller rank is one whose last rows of A and columns of B are 0."""

    __slots__ = ("A", "B", "scales", "count", "rank", "N", "K", "dtype", "device", "code", "_held",
                 "_ref")

    def __init__(self, A, B, scales=None):
        import torch
        self.code = dtype_code(A.dtype)
        if A.dim() != 3 or B.dim() != 3 or B.shape[0] != A.shape[0] or B.shape[2] != A.shape[1]:
            raise ValueError(f"shapes {tuple(A.shape)} and {tuple(B.shape)} are not "
                             "[count, rank, K] and [count, N, rank]")
        if B.dtype != A.dtype:
            raise TypeError(f"A is {A.dtype}, B {B.dtype}")
        self.count, self.rank, self.K = A.shape
        self.N = B.shape[1]
        if not 1 <= self.rank <= 256:
            raise ValueError(f"rank {self.rank} is not in 1 .. 256")
        if scales is not None:
            if scales.dtype != torch.float32:
                raise TypeError(f"scales are {scales.dtype}, not float32")
            if tuple(scales.shape) != (self.count,):
                raise ValueError(f"scales must be of shape ({self.count},)")
        for x in (A, B) if scales is None else (A, B, scales):
            if not x.is_cuda or not x.is_contiguous() or x.device != A.device:
                raise ValueError("A, B and scales must be contiguous, on one GPU")
        self.A, self.B, self.scales = A, B, scales
        self.dtype, self.device = A.dtype, A.device
        self._held = binding.lora_nt_adapters(A.data_ptr(), B.data_ptr(),
                                              None if scales is None else scales.data_ptr(),
                                              self.count, self.rank)
        self._ref = ctypes.byref(self._held)


@functools.lru_cache(maxsize=4096)
def _ws_size(M, N, K, rank, group):
    return binding.lib().gemm_nt_lora_ws_size(M, N, K, rank, group)


def gemm_nt_lora(X, w, adapters: LoraAdapters, ids, out=None, stream=None, workspace=None):
    """D = X @ w.T and, in each row, the part of its own adapter: row m has the adapter
    ids[m] (int32, [M]), or none where that is outside [0, count), -1 say.

    ``w``: a contiguous [N, K] tensor of X's type or a 2-D W4Weight.  X [M, K] and ``out``
    (optional, [M, N]) may have a row stride.  ``workspace`` (optional): a contiguous uint8
    tensor of ``binding.gemm_nt_lora_ws_size`` bytes, allocated here if none is given."""
    import torch
    packed = isinstance(w, W4Weight)
    device, K, N, dtype = adapters.device, adapters.K, adapters.N, adapters.dtype
    shape = X.shape
    if w.shape != (N, K) or len(shape) != 2 or shape[1] != K:
        raise ValueError(f"shapes {tuple(shape)}, {tuple(w.shape)} and adapters of {N} x {K} are "
                         "not [M, K], [N, K] and N x K")
    if X.dtype != dtype or w.dtype != dtype:
        raise TypeError(f"X is {X.dtype}, the weight {w.dtype}, the adapters {dtype}")
    if X.device != device or w.device != device or ids.device != device:
        raise ValueError("X, the weight, the ids and the adapters must be on the same GPU")
    if packed:
        pointers, group = w.pointers, w.group
    elif w.is_contiguous():
        pointers, group = (w.data_ptr(), None, None), 0
    else:
        raise ValueError("the weight must be contiguous")
    M = shape[0]
    if ids.dtype != torch.int32 or ids.shape != (M,) or not ids.is_contiguous():
        raise ValueError(f"ids must be a contiguous int32 tensor of {M} values")
    ldx = K if X.is_contiguous() else row_stride(X, "X")
    if out is None:
        out, ldd = new_rows(X, M, N, stream), N
    else:
        check_out(out, (M, N), dtype, device)
        ldd = row_stride(out, "out")
    if workspace is None:
        need = _ws_size(M, N, K, adapters.rank, group)
        with on_stream(stream):
            workspace = torch.empty(need, dtype=torch.uint8, device=device)
    else:
        if workspace.device != device or not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous, on X's device")
        need = workspace.numel() * workspace.element_size()
    launch("gemm_nt_lora", device,
           (X.data_ptr(), *pointers, adapters._ref, ids.data_ptr(), out.data_ptr(), M, N, K, ldx,
            ldd, group, adapters.code, workspace.data_ptr(), need, stream_of(device, stream)))
    return out
