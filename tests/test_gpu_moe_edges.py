"""GPU checks of the mixture of experts at the edges of its variants: a router
in several pieces of odd rows, one token's workgroups of 32 inner rows, gated
rows past fp16's range.  Tolerances: those of the layer's own tests."""
from __future__ import annotations

import math

import pytest
import torch

from dense_gemm_18_amd import MoeLayer
from tests.gpu_util import device, note
from tests.test_gpu_moe import Case
from tests.test_gpu_w4 import bits
from tests.w4_ref import TYPES, half_step

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,E,topk,H", [(5, 65, 4, 2051), (17, 16, 3, 3001), (1, 64, 8, 4097),
                                        (1, 300, 8, 2049), (3, 300, 5, 1535), (64, 16, 2, 5003),
                                        (2, 1, 1, 1025)])
def test_router_in_pieces_of_odd_rows(T, E, topk, H, dtype):
    # rows of an odd number of elements start at every second one in the middle of a
    # 4-byte word, and a piece ends there too
    note(f"moe odd router T{T} E{E} k{topk} H{H} {dtype}")
    c = Case(T + E + H, E, topk, H, 24, dtype)
    X = c.tokens(T)
    y, ids, weights = c.layer(X)
    ids2, weights2 = c.layer.route(X)
    assert torch.equal(ids, ids2) and torch.equal(weights, weights2)
    c.check_route(X, ids, weights)
    c.check_y(X, ids, weights, y)
    # the elements around the pieces' ends alone: every one counts
    X.zero_()
    ends = [0, H - 1] + [k + d for k in range(128, H - 1, 128) for d in (-1, 0)]
    X[:, ends] = torch.randn((T, len(ends)), generator=c.gen, device=device()).to(dtype)
    c.check_route(X, *c.layer.route(X))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("group", [32, 64, 128])
def test_one_token_of_long_packed_rows(group, dtype):
    # 8 slots of 129 blocks of 32 inner rows: the wider workgroups, and the choice
    # of the experts inside them
    note(f"moe one token, wide workgroups, group {group} {dtype}")
    c = Case(group, 16, 8, 4100, 4100, dtype, group, zeros=True)
    X = c.tokens(1)
    y, ids, weights = c.layer(X)
    c.check_route(X, ids, weights)
    c.check_y(X, ids, weights, y)
    assert torch.equal(bits(c.layer.experts(X, ids, weights)), bits(y))
    ids[0, 3] = ids[0, 0]                     # an expert twice, one slot left out
    ids[0, 5] = 16
    c.check_y(X, ids, weights, c.layer.experts(X, ids, weights))


@pytest.mark.parametrize("T", [1, 4, 40])
@pytest.mark.parametrize("dtype", TYPES)
def test_gated_rows_past_the_range_of_fp16(T, dtype):
    """silu(gate) * up = 90000: infinite where it is held in fp16, a number in
    bfloat16, and nothing of it in another token."""
    note(f"moe gated rows out of range T{T} {dtype}")
    E, H, I = 3, 64, 40
    X = torch.zeros((T, H), device=device(), dtype=dtype)
    X[:, 1] = 1
    X[T // 2, 0] = 1
    w13 = torch.zeros((E, 2 * I, H), device=device(), dtype=dtype)
    w13[:, [0, I], 0] = 300                   # gate and up of inner row 0
    w13[:, [1, I + 1], 1] = 2
    w2 = torch.zeros((E, H, I), device=device(), dtype=dtype)
    w2[:, 0, 0] = 0.25
    w2[:, 1, 0] = -0.25
    w2[:, 2, 1] = 1
    layer = MoeLayer(torch.zeros((E, H), device=device(), dtype=dtype), w13, w2, topk=2)
    ids = torch.tensor([[0, 2]], dtype=torch.int32, device=device()).expand(T, 2).contiguous()
    weights = torch.full((T, 2), 0.5, device=device())
    y = layer.experts(X, ids, weights).double()
    other = torch.arange(T, device=device()) != T // 2
    small = 4 / (1 + math.exp(-2))            # silu(2) * 2
    u = half_step(dtype)
    assert bool((y[other, 2] - small).abs().le(2.1 * u * small).all())
    assert not bool(y[other][:, :2].any()) and not bool(y[other][:, 3:].any())
    got = y[T // 2]
    if dtype == torch.float16:
        assert got[0] == math.inf and got[1] == -math.inf
        assert bool(torch.isnan(got[2:]).all())           # 0 times infinity
    else:
        assert abs(got[0] - 22500) <= 2.1 * u * 22500 and got[1] == -got[0]
        assert abs(got[2] - small) <= 2.1 * u * small and not bool(got[3:].any())
