"""A mixture-of-experts layer for a few tokens: tensors in, tensors out.

Over the C ABI of ``include/moe_nt.h``, which defines the layer, its
rounding and its limits.
"""
from __future__ import annotations

import ctypes
import math

from . import binding
from .w4 import W4Weight, check_out, dtype_code, launch, on_device, on_stream, row_stride, stream_of


_SCORING = {"softmax": binding.MOE_SOFTMAX, "sigmoid": binding.MOE_SIGMOID}
_LOGITS = {}


def _gate(E, device, topk, scoring, bias, groups, topk_groups, group_top, scale):
    """The gate's C structure; ValueError or TypeError where it is out of range."""
    import torch
    if scoring not in _SCORING:
        raise ValueError(f"scoring {scoring!r} is not 'softmax' or 'sigmoid'")
    if not 1 <= topk <= min(E, 16):
        raise ValueError(f"topk {topk} is not in 1 .. min({E}, 16)")
    if not 1 <= groups <= 64 or E % groups:
        raise ValueError(f"{groups} groups: not 1 .. 64 that divide {E} experts")
    kept, each = groups if topk_groups is None else topk_groups, E // groups
    if not 1 <= kept <= groups or topk > kept * each:
        raise ValueError(f"{kept} of {groups} groups of {each} experts do not hold {topk}")
    if group_top not in (1, 2) or group_top > each:
        raise ValueError(f"group_top {group_top} is not 1 or 2, and at most {each}")
    if not math.isfinite(scale):
        raise ValueError(f"scale {scale} is not finite")
    if bias is not None:
        if bias.dtype != torch.float32:
            raise TypeError(f"the bias is {bias.dtype}, not float32")
        if tuple(bias.shape) != (E,) or not bias.is_contiguous() or bias.device != device:
            raise ValueError(f"the bias must be a contiguous tensor of {E} values on {device}")
    return binding.moe_nt_gate(None if bias is None else bias.data_ptr(), _SCORING[scoring],
                               groups, kept, group_top, scale)


def choose_experts(logits, topk: int, scoring: str = "softmax", bias=None, groups: int = 1,
                   topk_groups=None, group_top: int = 1, renormalize: bool = True,
                   scale: float = 1.0, stream=None):
    """(ids, weights) of ``logits`` [T, E] (float32, float16 or bfloat16), both [T, topk],
    int32 and float32: what ``MoeLayer.experts`` takes.

    The scores are the logits' softmax or sigmoid; the topk experts with the largest score
    + ``bias`` ([E], float32) are chosen, in falling order, equal ones by rising index.
    With ``groups``, only ``topk_groups`` of them (default: all) are chosen from, those whose
    ``group_top`` (1 or 2) largest score + bias have the largest sums.  The weights are the
    chosen scores, without the bias, divided by their sum if ``renormalize``, times
    ``scale``.  ``logits`` may have a row stride; the rows may be any number."""
    import torch
    if not _LOGITS:
        _LOGITS.update({torch.float32: binding.GEMM_T_F32, torch.float16: binding.GEMM_T_F16,
                        torch.bfloat16: binding.GEMM_T_BF16})
    code = _LOGITS.get(logits.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {logits.dtype}: float32, float16 or bfloat16")
    if logits.dim() != 2 or not 1 <= logits.shape[1] <= 1024:
        raise ValueError(f"shape {tuple(logits.shape)} is not [T, E] with E in 1 .. 1024")
    if not logits.is_cuda:
        raise ValueError("the logits must be on a GPU")
    T, E = logits.shape
    device = logits.device
    g = _gate(E, device, topk, scoring, bias, groups, topk_groups, group_top, scale)
    ldl = E if logits.is_contiguous() else row_stride(logits, "logits")
    with on_stream(stream):
        ids = torch.empty(T, topk, dtype=torch.int32, device=device)
        weights = torch.empty(T, topk, dtype=torch.float32, device=device)
    launch("moe_nt_choose", device,
           (ctypes.byref(g), logits.data_ptr(), ids.data_ptr(), weights.data_ptr(), T, E, ldl,
            topk, binding.MOE_RENORMALIZE if renormalize else 0, code,
            stream_of(device, stream)))
    return ids, weights


class MoeLayer:
    """router [E, H] and the experts' weights w13 [E, 2 I, H] (gate rows, then up
    rows) and w2 [E, H, I], both as contiguous tensors in the router's 16-bit type or
    both as W4Weight of one group size.  The tensors are kept, not copied.

    Without ``scoring`` and the arguments after it the experts are the topk of a softmax
    over all; with any of them ``choose_experts`` says what they are and how they weigh
    (``scoring`` is then "softmax" unless given).

    Calls are enqueued on ``stream`` (default: the current stream of the weights'
    device).  The layer keeps one workspace for each stream it has been called on, so
    calls on different streams may overlap; host threads may call it on one stream or
    on several.  A call that is being captured takes a workspace of its own from the
    graph's memory, and its zero fill becomes a part of the graph: replays may run beside
    eager calls and other graphs."""

    def __init__(self, router, w13, w2, topk: int, renormalize: bool = True, scoring=None,
                 bias=None, groups: int = 1, topk_groups=None, group_top: int = 1,
                 scale: float = 1.0):
        packed = isinstance(w13, W4Weight)
        if packed != isinstance(w2, W4Weight):
            raise TypeError("w13 and w2 must both be tensors or both W4Weight")
        if packed and (w13.group != w2.group or (w13.zeros is None) != (w2.zeros is None)):
            raise ValueError("w13 and w2 must have one group size, and both zeros or neither")
        E, H = router.shape if router.dim() == 2 else (0, 0)
        if len(w13.shape) != 3 or len(w2.shape) != 3 or w13.shape[1] % 2:
            raise ValueError(f"shapes {tuple(w13.shape)} and {tuple(w2.shape)} are not "
                             "[E, 2 I, H] and [E, H, I]")
        inner = w13.shape[1] // 2
        if tuple(w13.shape) != (E, 2 * inner, H) or tuple(w2.shape) != (E, H, inner):
            raise ValueError(f"shapes {tuple(router.shape)}, {tuple(w13.shape)} and "
                             f"{tuple(w2.shape)} are not [E, H], [E, 2 I, H] and [E, H, I]")
        for x in (w13, w2):
            if x.dtype != router.dtype:
                raise TypeError(f"weights of {x.dtype} and a router of {router.dtype}")
            if x.device != router.device:
                raise ValueError("the router and the weights must be on one GPU")
        code = dtype_code(router.dtype)
        for x in (router,) if packed else (router, w13, w2):
            if not x.is_cuda or not x.is_contiguous():
                raise ValueError("the router and the weights must be contiguous, on a GPU")
        if not 1 <= topk <= min(E, 16):
            raise ValueError(f"topk {topk} is not in 1 .. min({E}, 16)")
        self.router, self.w13, self.w2 = router, w13, w2
        self.topk, self.renormalize = int(topk), bool(renormalize)
        self.hidden, self.dtype, self.device = H, router.dtype, router.device
        p13 = w13.pointers if packed else (w13.data_ptr(), None, None)
        p2 = w2.pointers if packed else (w2.data_ptr(), None, None)
        self._weights = binding.moe_nt_weights(router.data_ptr(), *p13, *p2, E, H, inner,
                                               w13.group if packed else 0, code)
        self._ref = ctypes.byref(self._weights)
        self._flags = binding.MOE_RENORMALIZE if renormalize else 0
        # a call runs at most 64 tokens at a time, so this serves every one
        self._ws_bytes = binding.moe_nt_ws_size(64, self._weights, self.topk)
        if not self._ws_bytes:
            raise ValueError(f"sizes E = {E}, H = {H}, I = {inner} are out of range")
        self._workspaces = {}
        self.bias, self._gate = bias, None
        if bias is not None or (scoring, groups, topk_groups, group_top,
                                scale) != (None, 1, None, 1, 1.0):
            gate = _gate(E, router.device, self.topk, scoring or "softmax", bias, groups,
                         topk_groups, group_top, scale)
            self._gate = ctypes.byref(gate)

    def _workspace(self, T, stream):
        """(a zero-filled workspace for T tokens on ``stream``, its bytes, the stream).
        The caller keeps the tensor until it has launched."""
        import torch
        handle = stream_of(self.device, stream)
        # the current stream, of which torch knows whether it captures, is the device's
        with on_stream(stream), on_device(self.device):
            if torch.cuda.is_current_stream_capturing():
                need = binding.moe_nt_ws_size(T, self._weights, self.topk)
                return torch.zeros(need, dtype=torch.uint8, device=self.device), need, handle
            ws = self._workspaces.get(handle)
            if ws is None:
                ws = torch.zeros(self._ws_bytes, dtype=torch.uint8, device=self.device)
                # another thread may have been here: one of the two for both
                ws = self._workspaces.setdefault(handle, ws)
        return ws, self._ws_bytes, handle

    def _check(self, X):
        if X.dim() != 2 or X.shape[1] != self.hidden:
            raise ValueError(f"shape {tuple(X.shape)} is not [T, {self.hidden}]")
        if X.dtype != self.dtype:
            raise TypeError(f"X is {X.dtype}, the layer {self.dtype}")
        if X.device != self.device:
            raise ValueError("X must be on the layer's GPU")
        return row_stride(X, "X")

    def _out(self, X, out, stream):
        if out is None:
            with on_stream(stream):
                return X.new_empty(X.shape), self.hidden
        check_out(out, X.shape, X.dtype, X.device)
        return out, row_stride(out, "out")

    def _slots(self, X, stream):
        import torch
        shape = (X.shape[0], self.topk)
        with on_stream(stream):
            return (torch.empty(shape, dtype=torch.int32, device=X.device),
                    torch.empty(shape, dtype=torch.float32, device=X.device))

    def __call__(self, X, out=None, stream=None):
        """(y, ids, weights) for the tokens X [T, H]: y [T, H] in X's type, the chosen
        experts ids [T, topk] (int32) and their weights [T, topk] (float32).  X and
        ``out`` may have a row stride."""
        ldx = self._check(X)
        out, ldd = self._out(X, out, stream)
        ids, weights = self._slots(X, stream)
        ws, ws_bytes, handle = self._workspace(X.shape[0], stream)
        gate = () if self._gate is None else (self._gate,)
        launch("moe_nt_layer_gated" if gate else "moe_nt_layer", self.device,
               (self._ref, *gate, X.data_ptr(), out.data_ptr(), ids.data_ptr(),
                weights.data_ptr(), X.shape[0], ldx, ldd, self.topk, self._flags, ws.data_ptr(),
                ws_bytes, handle))
        return out, ids, weights

    def route(self, X, stream=None):
        """(ids, weights) of the tokens X, as the layer's call returns them."""
        ldx = self._check(X)
        ids, weights = self._slots(X, stream)
        ws, ws_bytes, handle = self._workspace(X.shape[0], stream)
        gate = () if self._gate is None else (self._gate,)
        launch("moe_nt_route_gated" if gate else "moe_nt_route", self.device,
               (self._ref, *gate, X.data_ptr(), ids.data_ptr(), weights.data_ptr(), X.shape[0],
                ldx, self.topk, self._flags, ws.data_ptr(), ws_bytes, handle))
        return ids, weights

    def experts(self, X, ids, weights, out=None, stream=None):
        """y of the tokens X for given ids [T, topk] (int32) and weights [T, topk]
        (float32).  Slots whose id is not an expert's are left out."""
        import torch
        ldx = self._check(X)
        for x, dtype, what in ((ids, torch.int32, "ids"), (weights, torch.float32, "weights")):
            if x.dtype != dtype or tuple(x.shape) != (X.shape[0], self.topk) \
                    or not x.is_contiguous() or x.device != X.device:
                raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape "
                                 f"{(X.shape[0], self.topk)} on X's device")
        out, ldd = self._out(X, out, stream)
        ws, ws_bytes, handle = self._workspace(X.shape[0], stream)
        launch("moe_nt_experts", self.device,
               (self._ref, X.data_ptr(), ids.data_ptr(), weights.data_ptr(), out.data_ptr(),
                X.shape[0], ldx, ldd, self.topk, ws.data_ptr(), ws_bytes, handle))
        return out
