"""CPU checks of the 4-bit weight and mixture-of-experts operators: refusals
before any HIP call, sizes, and the packed layout."""
from __future__ import annotations

import pytest
import torch

from dense_gemm_18_amd import MoeLayer, W4Weight, binding, dequantize_w4, gemm_nt_w4, quantize_w4
from tests import w4_ref

OK, BAD = binding.GEMM_OK, binding.GEMM_EINVAL
# host-side integers used as addresses; never dereferenced
A, Q, S, Z, D, WS = (0x10000000 * i for i in range(1, 7))
F16 = binding.GEMM_T_F16


def w4(**kw):
    a = dict(A=A, Q=Q, S=S, Z=Z, D=D, M=4, N=64, K=256, lda=256, ldd=64, group=128, dtype=F16,
             workspace=0, ws_bytes=0, stream=0)
    a.update(kw)
    return binding.gemm_nt_w4(**a)


@pytest.mark.parametrize("kw", [
    dict(M=-1), dict(N=-1), dict(K=-1), dict(M=2 ** 31), dict(N=2 ** 31),
    dict(K=binding.GEMM_MAX_K + 1, lda=2 ** 30), dict(lda=255), dict(ldd=63),
    dict(lda=2 ** 41), dict(ldd=2 ** 41),
    dict(group=0), dict(group=16), dict(group=256), dict(dtype=2), dict(dtype=-1),
    dict(A=0), dict(Q=0), dict(S=0), dict(D=0), dict(A=A + 1), dict(D=D + 1), dict(S=S + 1),
    dict(Q=Q + 8),
    dict(D=A + 2), dict(D=Q + 64 * 128 - 2), dict(D=S + 2), dict(D=Z + 2),
    dict(ws_bytes=-1), dict(ws_bytes=256), dict(workspace=WS + 128, ws_bytes=256),
    dict(workspace=A, ws_bytes=256), dict(workspace=D, ws_bytes=256),
    dict(workspace=Q, ws_bytes=256),
])
def test_product_refuses_before_any_hip_call(kw):
    assert w4(**kw) == BAD


def test_product_of_nothing_is_a_no_op():
    assert w4(M=0, A=0, D=0) == OK
    assert w4(N=0, Q=0, S=0, Z=0, D=0, ldd=0) == OK


@pytest.mark.parametrize("fn", ["quantize", "dequantize"])
@pytest.mark.parametrize("kw", [
    dict(N=-1), dict(K=-1), dict(N=2 ** 31), dict(K=binding.GEMM_MAX_K + 1, ldw=2 ** 30),
    dict(ldw=255), dict(ldw=2 ** 41), dict(group=1), dict(dtype=7), dict(W=0), dict(Q=0),
    dict(S=0), dict(W=A + 1), dict(Q=Q + 4), dict(S=S + 1), dict(Q=A), dict(S=A + 2),
    dict(Z=A + 3),
])
def test_conversion_refuses_before_any_hip_call(fn, kw):
    a = dict(W=A, Q=Q, S=S, Z=Z, N=64, K=256, ldw=256, group=64, dtype=F16)
    a.update(kw)
    assert getattr(binding, "gemm_w4_" + fn)(**a) == BAD


def test_outputs_of_the_quantisation_may_not_overlap():
    a = dict(W=A, Q=Q, S=Q + 32, Z=0, N=64, K=256, ldw=256, group=64, dtype=F16)
    assert binding.gemm_w4_quantize(**a) == BAD
    a = dict(W=A, Q=Q, S=S, Z=S + 1, N=64, K=256, ldw=256, group=64, dtype=F16)
    assert binding.gemm_w4_quantize(**a) == BAD
    for n, k in ((0, 256), (64, 0)):
        assert binding.gemm_w4_quantize(0, 0, 0, 0, n, k, k, 64, F16) == OK
        assert binding.gemm_w4_dequantize(0, 0, 0, 0, n, k, k, 64, F16) == OK


def test_sizes():
    assert binding.gemm_w4_packed_bytes(3, 1) == 3 * 64
    assert binding.gemm_w4_packed_bytes(3, 128) == 3 * 64
    assert binding.gemm_w4_packed_bytes(2 ** 31 - 1, 129) == (2 ** 31 - 1) * 128
    assert binding.gemm_w4_packed_bytes(-1, 5) == 0
    assert binding.gemm_nt_w4_ws_size(1, 4096, 4096) == 0
    assert binding.gemm_nt_w4_ws_size(4096, 4096, 4097) == -(-4096 * 4097 * 2 // 256) * 256
    assert binding.gemm_nt_w4_ws_size(4096, 0, 4096) == 0
    assert binding.gemm_nt_w4_ws_size(4096, 4096, binding.GEMM_MAX_K + 1) == 0


def weights(**kw):
    a = dict(router=0x100000000, w13=0x200000000, w13_scales=0x300000000, w13_zeros=0,
             w2=0x400000000, w2_scales=0x500000000, w2_zeros=0, experts=8, hidden=256, inner=64,
             group=128, dtype=F16)
    a.update(kw)
    return binding.moe_nt_weights(**{k: v or (None if k.startswith(("w", "router")) else 0)
                                     for k, v in a.items()})


X, IDS, WTS, OUT, MWS = (0x1000000000 * i for i in range(1, 6))


def layer(w=None, topk=2, flags=0, T=4, ldx=256, ldd=256, x=X, ids=IDS, wts=WTS, d=OUT, ws=MWS,
          short=0, only=None):
    w = weights() if w is None else w
    need = max(0, binding.moe_nt_ws_size(max(T, 0), w, topk) - short) or 1 << 20
    if only == "route":
        return binding.moe_nt_route(w, x, ids, wts, T, ldx, topk, flags, ws, need)
    if only == "experts":
        return binding.moe_nt_experts(w, x, ids, wts, d, T, ldx, ldd, topk, ws, need)
    return binding.moe_nt_layer(w, x, d, ids, wts, T, ldx, ldd, topk, flags, ws, need)


@pytest.mark.parametrize("kw", [
    dict(w=weights(experts=0)), dict(w=weights(experts=1025)), dict(w=weights(hidden=0)),
    dict(w=weights(hidden=binding.GEMM_MAX_K + 1), ldx=2 ** 30, ldd=2 ** 30),
    dict(w=weights(inner=0)), dict(w=weights(inner=binding.GEMM_MAX_K + 1)),
    dict(w=weights(group=16)), dict(w=weights(dtype=3)), dict(w=weights(router=0)),
    dict(w=weights(router=0x100000001)), dict(w=weights(w13=0)), dict(w=weights(w2=0)),
    dict(w=weights(w13_scales=0)), dict(w=weights(w2_scales=0)),
    dict(w=weights(w13=0x200000008)), dict(w=weights(w2=0x400000002)),
    dict(w=weights(w13_zeros=0x600000000)), dict(w=weights(w2_scales=0x500000001)),
    dict(topk=0), dict(topk=9), dict(topk=17), dict(flags=2), dict(T=-1), dict(T=2 ** 31),
    dict(ldx=255), dict(ldd=255), dict(x=0), dict(ids=0), dict(wts=0), dict(d=0), dict(ws=0),
    dict(x=X + 1), dict(ids=IDS + 2), dict(wts=WTS + 1), dict(d=OUT + 1), dict(ws=MWS + 64),
    dict(short=256), dict(d=X), dict(d=IDS), dict(ids=X), dict(wts=IDS + 4), dict(ws=X),
    dict(d=0x200000000), dict(d=0x400000000), dict(d=0x300000000), dict(d=MWS),
])
def test_layer_refuses_before_any_hip_call(kw):
    assert layer(**kw) == BAD


def test_halves_refuse_too():
    assert layer(only="route", topk=9) == BAD
    assert layer(only="route", wts=IDS) == BAD
    assert layer(only="experts", ldd=10) == BAD
    assert layer(only="experts", topk=17) == BAD
    assert layer(only="experts", d=WTS) == BAD
    assert layer(T=0) == OK
    assert layer(only="route", T=0, x=0, ids=0, wts=0) == OK
    assert layer(only="experts", T=0, x=0, ids=0, wts=0, d=0) == OK
    assert binding.lib().moe_nt_layer(None, X, OUT, IDS, WTS, 1, 256, 256, 1, 0, MWS, 1 << 20,
                                      None) == BAD


def test_layer_workspace_does_not_grow_past_a_chunk():
    w = weights()
    one = binding.moe_nt_ws_size(1, w, 2)
    assert 0 < one < binding.moe_nt_ws_size(64, w, 2) == binding.moe_nt_ws_size(10 ** 6, w, 2)
    assert binding.moe_nt_ws_size(0, w, 2) == 0
    assert binding.moe_nt_ws_size(4, weights(experts=2000), 2) == 0


def test_layout_is_a_bijection_and_packs_back():
    K = 300
    word, bit = w4_ref.word_and_bit(384)
    assert len({(int(a), int(b)) for a, b in zip(word, bit)}) == 384
    assert int(word.max()) == 47 and set(bit.tolist()) == set(range(0, 32, 4))
    q = torch.randint(0, 16, (5, K), generator=torch.Generator().manual_seed(1))
    assert torch.equal(w4_ref.unpack(w4_ref.pack(q), K), q)


def test_tensor_calls_refuse_before_any_gpu_use():
    h = torch.zeros((4, 256), dtype=torch.float16)
    with pytest.raises(TypeError):
        quantize_w4(h.float())
    with pytest.raises(ValueError):
        quantize_w4(h)                                      # CPU tensor
    with pytest.raises(ValueError):
        quantize_w4(h[0])
    q = torch.zeros((4, 32), dtype=torch.int32)
    s = torch.zeros((4, 2), dtype=torch.float16)
    with pytest.raises(ValueError):
        W4Weight(q, s, shape=(4, 256), group=128)           # CPU tensors
    with pytest.raises(ValueError):
        W4Weight(q, s, shape=(4, 256), group=100)
    with pytest.raises(ValueError):
        W4Weight(q, s, shape=(256,), group=128)
    with pytest.raises(ValueError):
        W4Weight(q, s, shape=(4, 257), group=128)           # 3 blocks wanted
    with pytest.raises(TypeError):
        W4Weight(q, s.float(), shape=(4, 256), group=128)
    router = torch.zeros((4, 256), dtype=torch.float16)
    w13 = torch.zeros((4, 128, 256), dtype=torch.float16)
    w2 = torch.zeros((4, 256, 64), dtype=torch.float16)
    with pytest.raises(ValueError):
        MoeLayer(router, w13, w2, topk=2)                   # CPU tensors
    with pytest.raises(ValueError):
        MoeLayer(router, w13, w2[:, :, :63], topk=2)
    with pytest.raises(ValueError):
        MoeLayer(router, w13[:, :127], w2, topk=2)
    with pytest.raises(TypeError):
        MoeLayer(router, w13.float(), w2, topk=2)
    assert callable(gemm_nt_w4) and callable(dequantize_w4)


def test_limits_shared_with_the_headers():
    root = binding.library_path().parents[1] / "include"
    text = (root / "gemm_nt_w4.h").read_text() + (root / "moe_nt.h").read_text()
    for name in ("GEMM_T_F16", "GEMM_T_BF16", "MOE_RENORMALIZE"):
        assert f"#define {name} {getattr(binding, name)}" in text


def test_row_lengths_past_the_limits_are_refused():
    assert w4(M=0, A=0, D=0, lda=16777215) == OK
    assert w4(M=0, A=0, D=0, lda=16777216) == BAD
    assert w4(M=2, lda=16777216) == BAD
    assert layer(T=0, ldx=16777215) == OK
    assert layer(T=0, ldx=16777216) == BAD
    assert layer(ldx=16777216) == BAD
    assert layer(w=weights(inner=1048577)) == BAD
    # (of 8 experts, the operands would overlap at these addresses)
    assert layer(T=0, topk=1, w=weights(inner=1048576, experts=1)) == OK


def test_workspace_of_the_product_starts_past_the_direct_rows():
    assert binding.gemm_nt_w4_ws_size(384, 4096, 4096) == 0
    assert binding.gemm_nt_w4_ws_size(385, 4096, 4096) == 4096 * 4096 * 2
