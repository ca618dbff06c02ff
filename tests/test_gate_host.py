"""CPU checks of the choice of experts: refusals before any HIP call."""
from __future__ import annotations

import ctypes

import pytest
import torch

from dense_gemm_18_amd import binding, choose_experts

OK, BAD = binding.GEMM_OK, binding.GEMM_EINVAL
# host-side integers used as addresses; never dereferenced
L, IDS, WEIGHTS, BIAS, X, WS, D = (0x10000000 * i for i in range(1, 8))
GATE = dict(bias=BIAS, scoring=binding.MOE_SIGMOID, groups=8, topk_groups=4, group_top=2,
            scale=1.0)


def gate(**kw):
    return ctypes.byref(binding.moe_nt_gate(*{**GATE, **kw}.values()))


def choose(g=None, **kw):
    a = dict(logits=L, ids=IDS, weights=WEIGHTS, T=5, experts=64, ldl=64, topk=6,
             flags=binding.MOE_RENORMALIZE, dtype=binding.GEMM_T_F32)
    a.update(kw)
    return binding.moe_nt_choose(gate(**(g or {})), **a)


BAD_GATES = [dict(scoring=2), dict(scoring=-1), dict(groups=0), dict(groups=7), dict(groups=65),
             dict(groups=-8), dict(topk_groups=0), dict(topk_groups=9), dict(group_top=0),
             dict(group_top=3), dict(groups=64), dict(groups=32, topk_groups=2, group_top=1),
             dict(scale=float("inf")), dict(scale=float("nan")), dict(bias=BIAS + 2),
             dict(bias=IDS), dict(bias=WEIGHTS + 4)]


@pytest.mark.parametrize("g", BAD_GATES)
def test_gate_is_refused_before_any_hip_call(g):
    assert choose(g) == BAD


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(T=2 ** 31), dict(experts=0), dict(experts=1032, ldl=2000), dict(ldl=63),
    dict(ldl=2 ** 41), dict(topk=0), dict(topk=17), dict(flags=2), dict(dtype=3), dict(dtype=-1),
    dict(logits=0), dict(ids=0), dict(weights=0), dict(logits=L + 2), dict(ids=IDS + 2),
    dict(weights=WEIGHTS + 1), dict(ids=L + 4 * 319), dict(weights=L), dict(weights=IDS + 116)])
def test_choice_refuses_before_any_hip_call(kw):
    assert choose(**kw) == BAD
    assert binding.moe_nt_choose(None, L, IDS, WEIGHTS, 5, 64, 64, 6, 0, 2) == BAD


def test_no_rows_are_a_no_op():
    assert choose(T=0, logits=0, ids=0, weights=0) == OK


def layer(g, route=False, **kw):
    w = binding.moe_nt_weights(0x100000000, 0x200000000, None, None, 0x300000000, None, None, 64,
                               128, 64, 0, binding.GEMM_T_F16)
    a = dict(X=X, D=D, ids=IDS, weights=WEIGHTS, T=5, ldx=128, ldd=128, topk=6, flags=0,
             workspace=WS, ws_bytes=binding.moe_nt_ws_size(5, w, 6))
    a.update(kw)
    if route:
        del a["D"], a["ldd"]
        return binding.moe_nt_route_gated(w, g, **a)
    return binding.moe_nt_layer_gated(w, g, **a)


@pytest.mark.parametrize("route", [False, True])
def test_gated_layer_refuses_before_any_hip_call(route):
    for g in BAD_GATES:
        assert layer(gate(**g), route) == BAD
    assert layer(None, route) == BAD
    assert layer(gate(bias=WS + 256), route) == BAD
    if not route:
        assert layer(gate(bias=D + 8)) == BAD
        assert layer(gate(), D=X) == BAD
    for kw in (dict(T=-1), dict(topk=17), dict(flags=2), dict(ids=0), dict(ws_bytes=10),
               dict(ids=X)):
        assert layer(gate(), route, **kw) == BAD
    assert layer(gate(), route, T=0) == OK


def test_python_refuses():
    logits = torch.zeros((4, 64))
    for kw in (dict(), dict(topk=0)):
        with pytest.raises(ValueError):
            choose_experts(logits, **{"topk": 2, **kw})        # not on a GPU
    with pytest.raises(TypeError):
        choose_experts(logits.double(), 2)
    with pytest.raises(ValueError):
        choose_experts(torch.zeros((4, 1025)), 2)
    from dense_gemm_18_amd.moe import _gate
    good = dict(E=64, device=logits.device, topk=6, scoring="sigmoid", bias=None, groups=8,
                topk_groups=4, group_top=2, scale=1.0)
    _gate(**good)
    for kw in (dict(scoring="tanh"), dict(topk=0), dict(topk=17), dict(groups=7), dict(groups=0),
               dict(topk_groups=9), dict(topk_groups=0), dict(topk=16, topk_groups=1),
               dict(group_top=3), dict(groups=64, topk_groups=8), dict(scale=float("inf")),
               dict(bias=torch.zeros(63))):
        with pytest.raises(ValueError):
            _gate(**{**good, **kw})
    with pytest.raises(TypeError):
        _gate(**{**good, "bias": torch.zeros(64, dtype=torch.float16)})
