"""GPU checks of activations far larger than the others.

Where such an activation meets a weight of exactly 0 (q == z), it adds exactly
0 to the sum, whatever its size: the result has the bits that it has with a 0
in the activation's place.  Elsewhere the tolerance goes by the terms that the
sum has: u |ref| + 2^-23 (group + G + 12) sum |A| |q - z| s, one rounding of
the result and the fp32 sums of a group, over G groups and of 8 waves, with u
the 16-bit type's half step.
"""
from __future__ import annotations

import math

import pytest
import torch

from dense_gemm_18_amd import MoeLayer, W4Weight
from tests import w4_ref
from tests.gpu_util import device, note
from tests.test_gpu_w4 import bits, gen, product
from tests.w4_ref import TYPES, half_step

pytestmark = pytest.mark.gpu

LARGE = {torch.float16: [3.0e3, 6.0e4], torch.bfloat16: [4.0e3, 3.0e4, -1.0e6, 1.0e30]}

# every tile of the product, by the rows and columns that choose it
SHAPES = [(3, 16390, 300), (2, 8200, 333), (1, 50, 1000), (16, 16390, 2184), (13, 8200, 2700),
          (16, 400, 4100), (260, 1000, 515), (500, 1030, 387), (1030, 1000, 300)]


def without_weight_at(Q, Z, K, columns):
    """Q with q = z in `columns`."""
    q = w4_ref.unpack(Q, K)
    for k, group in columns:
        q[..., k] = 8 if Z is None else (Z.to(torch.int64) & 15)[..., k // group]
    return w4_ref.pack(q)


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", TYPES)
def test_an_outlier_meets_weights_of_zero(M, N, K, group, dtype):
    note(f"w4 outlier {M}x{N}x{K} group {group} {dtype}")
    for zeros in (False, True):
        g = gen(M + N + K + group + zeros)
        A = torch.randn((M, K), generator=g, device=device(), dtype=dtype)
        Q, S, Z = w4_ref.random_weight(g, N, K, group, zeros, dtype)
        Q = without_weight_at(Q, Z, K, [(17, group), (K - 2, group)])
        A[:, 17] = A[:, K - 2] = 0
        # rows of D apart: many rows too are unpacked on the way
        want = product(A, Q, S, Z, group, ldd_pad=2)
        for value in LARGE[dtype]:
            A[:, 17] = value
            A[0, K - 2] = -value
            assert torch.equal(bits(product(A, Q, S, Z, group, ldd_pad=2)), bits(want)), value


@pytest.mark.parametrize("M,N,K", [(1, 300, 1024), (7, 200, 500), (40, 130, 2050)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", TYPES)
def test_an_outlier_among_all_weights(M, N, K, group, dtype):
    note(f"w4 outlier among weights {M}x{N}x{K} group {group} {dtype}")
    g = gen(M + N + K)
    A = torch.randn((M, K), generator=g, device=device(), dtype=dtype)
    Q, S, Z = w4_ref.random_weight(g, N, K, group, True, dtype)
    w = w4_ref.values(Q, S, Z, K, group)
    for value in LARGE[dtype][:3]:
        A[:, 100] = value / 8
        D = product(A, Q, S, Z, group)
        ref = A.double() @ w.T
        C = A.double().abs() @ w.abs().T
        u = half_step(dtype)
        bound = (u * ref.abs() + 2.0 ** -23 * (group + S.shape[1] + 12) * C
                 + torch.finfo(dtype).smallest_normal * u)
        assert bool(((D.double() - ref).abs() <= bound).all()), value


@pytest.mark.parametrize("T", [1, 5, 40])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", TYPES)
def test_an_outlier_in_the_layer(T, group, dtype):
    """Of the tokens against gate and up rows, and of the gated rows against W2."""
    note(f"moe outlier T{T} group {group} {dtype}")
    E, topk, H, I = 6, 3, 390, 260
    g = gen(T + group)
    raw = []
    for n, k in ((2 * I, H), (H, I)):
        Q, S, Z = w4_ref.random_weight(g, n, k, group, True, dtype, scale=0.25 / math.sqrt(k),
                                       lead=(E,))
        raw.append((without_weight_at(Q, Z, k, [(33, group)]), S, Z))
    router = torch.zeros((E, H), device=device(), dtype=dtype)
    ids = (torch.arange(T * topk, device=device()).view(T, topk) % E).to(torch.int32)
    weights = torch.rand((T, topk), generator=g, device=device())
    X = torch.randn((T, H), generator=g, device=device()).to(dtype)

    def run(w13, X):
        layer = MoeLayer(router, W4Weight(*w13, shape=(E, 2 * I, H), group=group),
                         W4Weight(*raw[1], shape=(E, H, I), group=group), topk=topk)
        return layer.experts(X, ids, weights)

    X[:, 33] = 0
    want = run(raw[0], X)
    X[:, 33] = LARGE[dtype][-1]
    assert torch.equal(bits(run(raw[0], X)), bits(want))
    X[:, 33] = 0
    # h[33] large by its gate and up rows' scales (in fp16 within its range), or 0
    outs = []
    for scale in (0.0, 8.0 if dtype == torch.float16 else 1.0e8):
        S = raw[0][1].clone()
        S[:, [33, I + 33]] = (0.25 / math.sqrt(H)) * scale
        outs.append(run((raw[0][0], S, raw[0][2]), X))
    assert bool(torch.isfinite(outs[1]).all())
    assert torch.equal(bits(outs[0]), bits(outs[1]))


@pytest.mark.parametrize("M,N,K", [(1, 300, 1024), (20, 130, 500), (40, 130, 2050)])
@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("power", [-126, -120, -100, 100, 120, 126])
def test_the_whole_range_of_bfloat16(M, N, K, group, power):
    """Integers times a power of two, and scales that bring the sums back: as exact
    as for small numbers, and no sum of a group leaves fp32's range."""
    note(f"w4 range {M}x{N}x{K} group {group} 2^{power}")
    dtype = torch.bfloat16
    g = gen(M + N + K)
    A = torch.randint(-2, 3, (M, K), generator=g, device=device()).to(dtype)
    Q, S, Z = w4_ref.random_weight(g, N, K, group, True, dtype)
    S = torch.exp2(torch.randint(-2, 2, S.shape, generator=g, device=device()).float()).to(dtype)
    ref = A.double() @ w4_ref.values(Q, S, Z, K, group).T
    back = 2.0 ** -(power // 2)
    D = product((A.double() * 2.0 ** power).to(dtype), Q, (S.double() * back).to(dtype), Z, group)
    assert torch.equal(D, (ref * 2.0 ** power * back).to(dtype))
