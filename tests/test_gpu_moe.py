"""GPU checks of the mixture-of-experts layer against plain 64-bit forms.

Tolerances, with u the 16-bit type's half step: y is rounded once (u |y|),
the gated rows h once (u times W = sum_j w_j sum_i |W2 h|); what fp32 sums
and silu add is below 2^-23 times the number of terms and is given by
2^-23 (H + I + 64) times the largest sums of magnitudes, 16 sqrt(H) times W
for inputs of unit size, times 64 more where bfloat16 multiplies packed
weights as 128 + q.  In the 2-norm the two roundings give 2 u.  Router
weights: fp32 logits of unit size to 2^-23 sqrt(H) and an exponential, 1e-5.
"""
from __future__ import annotations

import math

import pytest
import torch

from dense_gemm_18_amd import MoeLayer, W4Weight, quantize_w4
from tests import w4_ref
from tests.gpu_util import device, note
from tests.test_gpu_w4 import bits, check_guard, gen, strided
from tests.w4_ref import TYPES, half_step

pytestmark = pytest.mark.gpu


class Case:
    """A layer with random weights, and its weights in 64 bits."""

    def __init__(self, seed, E, topk, H, I, dtype, group=0, zeros=False, renorm=True):
        g = gen(seed)
        self.gen, self.group, self.topk, self.renorm = g, group, topk, renorm
        self.E, self.H, self.I, self.dtype = E, H, I, dtype

        def normal(scale, *shape):
            return (torch.randn(shape, generator=g, device=device()) * scale).to(dtype)
        self.router = normal(2 / math.sqrt(H), E, H)
        if group:
            raw = [w4_ref.random_weight(g, n, k, group, zeros, dtype, scale=0.25 / math.sqrt(k),
                                        lead=(E,)) for n, k in ((2 * I, H), (H, I))]
            w13, w2 = (W4Weight(*r, shape=(E, n, k), group=group)
                       for r, (n, k) in zip(raw, ((2 * I, H), (H, I))))
            self.w13, self.w2 = (w4_ref.values(*r, k, group) for r, k in zip(raw, (H, I)))
        else:
            w13, w2 = normal(1 / math.sqrt(H), E, 2 * I, H), normal(1 / math.sqrt(I), E, H, I)
            self.w13, self.w2 = w13.double(), w2.double()
        self.layer = MoeLayer(self.router, w13, w2, topk=topk, renormalize=renorm)

    def tokens(self, T):
        return torch.randn((T, self.H), generator=self.gen, device=device()).to(self.dtype)

    def check_route(self, X, ids, weights):
        """ids: a falling order of the exact logits up to fp32's error, equal ones by
        rising index; weights by the definition for those ids."""
        logits = X.double() @ self.router.double().T
        assert ids.dtype == torch.int32 and weights.dtype == torch.float32
        at = ids.long()
        assert bool(((at >= 0) & (at < self.E)).all())
        chosen = logits.gather(1, at)
        slack = 2.0 ** -22 * math.sqrt(self.H) * 8
        assert bool((chosen[:, :-1] >= chosen[:, 1:] - slack).all())
        rest = logits.scatter(1, at, -math.inf)
        assert bool((rest.amax(-1) <= chosen[:, -1] + slack).all())
        over = chosen if self.renorm else logits
        want = torch.exp(chosen - torch.logsumexp(over, -1, keepdim=True))
        assert bool(((weights.double() - want).abs() <= 1e-5 * want + 1e-30).all())

    def check_y(self, X, ids, weights, y):
        u = half_step(self.dtype)
        ids, weights = ids.cpu(), weights
        ids = ids.to(device())
        ref = w4_ref.moe(X, ids, weights, self.w13, self.w2)
        size = torch.zeros_like(ref)
        for e in range(self.E):
            t, j = torch.nonzero(ids == e, as_tuple=True)
            if len(t):
                gu = X[t].double() @ self.w13[e].T
                h = (torch.sigmoid(gu[:, :self.I]) * gu[:, :self.I] * gu[:, self.I:]).abs()
                size.index_add_(0, t, h @ self.w2[e].abs().T
                                * weights[t, j].double().abs().unsqueeze(-1))
        extra = 64 if self.group and self.dtype == torch.bfloat16 else 1
        fp32 = 2.0 ** -23 * (self.H + self.I + 64) * 16 * extra
        # below the smallest normal number h's step no longer shrinks
        tiny = torch.finfo(self.dtype).smallest_normal * u * (1 + self.I)
        bound = u * ref.abs() + (u + min(fp32, u) / 4) * (1 + u) * size + tiny + fp32 * size / 64
        bad = (y.double() - ref).abs() > bound
        assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} outside"
        if ref.numel() >= 64 and float(ref.norm()) > 0:
            assert w4_ref.rel(y, ref) <= 2 * u


#        T   E  topk  H     I   group zeros renorm
CASES = [(1, 1, 1, 1, 1, 0, False, True),
         (1, 8, 2, 128, 64, 0, False, True),
         (1, 16, 8, 300, 130, 0, False, False),
         (2, 3, 3, 129, 33, 0, False, True),
         (5, 12, 3, 1000, 700, 0, False, False),
         (16, 64, 6, 512, 256, 0, False, True),
         (17, 65, 16, 200, 100, 0, False, False),
         (33, 5, 2, 257, 127, 0, False, True),
         (64, 16, 2, 384, 200, 0, False, True),
         (64, 2, 1, 130, 70, 0, False, True),
         (65, 4, 4, 96, 48, 0, False, False),
         (130, 9, 16 - 7, 64, 40, 0, False, True),
         (3, 257, 5, 100, 20, 0, False, False),
         (2, 1024, 16, 64, 16, 0, False, True),
         (1, 8, 2, 1, 1, 32, True, True),
         (1, 8, 2, 128, 64, 128, False, True),
         (1, 20, 8, 1024, 512, 128, True, True),
         (5, 12, 3, 1000, 700, 32, False, False),
         (7, 6, 2, 390, 129, 64, True, False),
         (16, 32, 4, 512, 256, 64, False, True),
         (31, 4, 2, 260, 100, 32, True, True),
         (64, 8, 2, 384, 200, 128, True, True),
         (70, 3, 3, 130, 66, 64, False, False)]


@pytest.mark.parametrize("T,E,topk,H,I,group,zeros,renorm", CASES)
@pytest.mark.parametrize("dtype", TYPES)
def test_layer_against_64_bits(T, E, topk, H, I, group, zeros, renorm, dtype):
    note(f"moe T{T} E{E} k{topk} H{H} I{I} group {group} {dtype}")
    c = Case(T + E + H, E, topk, H, I, dtype, group, zeros, renorm)
    X = c.tokens(T)
    y, ids, weights = c.layer(X)
    torch.cuda.synchronize()
    c.check_route(X, ids, weights)
    c.check_y(X, ids, weights, y)
    # the halves, and again: the same bits
    ids2, weights2 = c.layer.route(X)
    assert torch.equal(ids, ids2) and torch.equal(weights, weights2)
    assert torch.equal(bits(c.layer.experts(X, ids, weights)), bits(y))
    assert torch.equal(bits(c.layer(X)[0]), bits(y))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("group", [0, 64])
def test_left_out_repeated_and_uneven_slots(group, dtype):
    note(f"moe slots group {group} {dtype}")
    c = Case(3, 6, 4, 260, 140, dtype, group)
    T = 40
    X = c.tokens(T)
    g = gen(4)
    ids = torch.randint(-2, 9, (T, 4), generator=g, device=device()).to(torch.int32)
    ids[0] = -1                               # nothing left
    ids[1] = 6
    ids[2] = 2                                # one expert four times
    ids[3:30, 0] = 5                          # an expert with more than 16 rows
    ids[7] = torch.tensor([2 ** 31 - 1, -2 ** 31, 3, 1])
    weights = torch.randn((T, 4), generator=g, device=device())
    y = c.layer.experts(X, ids, weights)
    assert bool((bits(y[:2]) == 0).all())
    c.check_y(X, ids, weights, y)
    # what a left-out slot's weight holds does not matter
    odd = weights.clone()
    odd[(ids < 0) | (ids >= 6)] = float("nan")
    assert torch.equal(bits(c.layer.experts(X, ids, odd)), bits(y))
    # all rows to one expert, all four slots: 160 rows, more than one pass of 64
    ids = torch.full((T, 4), 4, dtype=torch.int32, device=device())
    y = c.layer.experts(X, ids, weights)
    c.check_y(X, ids, weights, y)
    # all left out
    y = c.layer.experts(X, ids + 100, weights)
    assert bool((bits(y) == 0).all())


def test_equal_logits_go_to_the_lowest_index():
    for E, topk in ((7, 3), (64, 8), (300, 16), (1024, 5)):
        c = Case(E, E, topk, 96, 16, torch.bfloat16)
        note(f"moe ties E {E}")
        c.router[:] = c.router[0]             # all logits alike
        X = c.tokens(9)
        ids, weights = c.layer.route(X)
        assert torch.equal(ids.cpu(), torch.arange(topk, dtype=torch.int32).expand(9, topk))
        assert bool(((weights - 1 / topk).abs() <= 1e-6).all())
        X.zero_()                             # logits +0 and -0
        c.router[::2] *= -1
        assert torch.equal(c.layer.route(X)[0].cpu(),
                           torch.arange(topk, dtype=torch.int32).expand(9, topk))


@pytest.mark.parametrize("E", [5, 100, 700])
def test_odd_logits(E):
    note(f"moe odd logits E {E}")
    c = Case(E, E, 4, 64, 16, torch.float16, renorm=False)
    X = c.tokens(6)
    clean = c.layer(X)
    c.router[3, 0] = float("nan")
    ids, weights = c.layer.route(X)
    assert bool(torch.isnan(weights).all())
    for row in ids.tolist():
        assert len(set(row)) == 4 and all(0 <= e < E and e != 3 for e in row)
    c.router[3, 0] = 0.0
    X2 = X.clone()
    X2[2, 5] = float("nan")                   # one token's own affair
    y, ids, weights = c.layer(X2)
    keep = [0, 1, 3, 4, 5]
    c.router[3, 0] = 0.0
    again = c.layer(X)
    assert torch.equal(ids[keep], again[1][keep])
    assert torch.equal(bits(y[keep]), bits(again[0][keep]))
    assert bool(torch.isnan(weights[2]).all()) and bool(torch.isnan(y[2]).all())
    assert sorted(set(ids[2].tolist())) == sorted(ids[2].tolist())
    assert clean[0].shape == y.shape
    # large logits: a weight of 1 and no overflow
    X3 = torch.full((1, 64), 100.0, dtype=torch.float16, device=device())
    c.router.zero_()
    c.router[2] = 600.0                       # a logit of 3.84e6
    ids, weights = c.layer.route(X3)
    assert ids[0].tolist() == [2, 0, 1, 3] and weights[0].tolist() == [1.0, 0.0, 0.0, 0.0]


@pytest.mark.parametrize("dtype", TYPES)
def test_row_strides(dtype):
    note(f"moe strides {dtype}")
    c = Case(8, 4, 2, 130, 50, dtype)
    X = c.tokens(5)
    want = c.layer(X)
    _, xs = strided(5, 130, 137, dtype)
    xs.copy_(X)
    buf, out = strided(5, 130, 141, dtype)
    y, ids, weights = c.layer(xs, out=out)
    torch.cuda.synchronize()
    check_guard(buf, 5, 130, 141, dtype)
    assert torch.equal(bits(y), bits(want[0])) and torch.equal(ids, want[1])
    assert torch.equal(weights, want[2])
    assert c.layer(X[:0])[0].shape == (0, 130)


def test_packed_layer_is_the_layer_of_its_values():
    # quantise 16-bit weights, run both ways: the difference is the weights' alone
    c = Case(2, 4, 2, 256, 128, torch.bfloat16)
    packed = [quantize_w4(w.to(torch.bfloat16), group=32, zeros=True) for w in (c.w13, c.w2)]
    layer = MoeLayer(c.router, *packed, topk=2)
    X = c.tokens(6)
    note("moe packed")
    y, ids, weights = layer(X)
    ids0, weights0 = c.layer.route(X)
    assert torch.equal(ids, ids0) and torch.equal(weights, weights0)
    c.group = 32
    c.w13, c.w2 = (w4_ref.values(p.q, p.scales, p.zeros, p.K, 32) for p in packed)
    c.check_y(X, ids, weights, y)


def test_offsets_past_32_bits():
    # w13: 40 experts of 2 * 8192 x 4096: 5.4 GB; only the last experts run
    E, H, I = 40, 4096, 8192
    note("moe offsets past 2^32")
    g = gen(1)
    w13 = torch.empty((E, 2 * I, H), dtype=torch.bfloat16, device=device())
    w2 = torch.empty((E, H, I), dtype=torch.bfloat16, device=device())
    for w, k in ((w13, H), (w2, I)):
        for e in (0, E - 2, E - 1):
            w[e] = torch.randn(w.shape[1:], generator=g, device=device()) / math.sqrt(k)
    router = torch.randn((E, H), generator=g, device=device(), dtype=torch.bfloat16)
    layer = MoeLayer(router, w13, w2, topk=2)
    X = torch.randn((3, H), generator=g, device=device(), dtype=torch.bfloat16)
    ids = torch.tensor([[39, 38], [0, 39], [38, 0]], dtype=torch.int32, device=device())
    weights = torch.rand((3, 2), generator=g, device=device())
    y = layer.experts(X, ids, weights)
    want = torch.zeros((3, H), dtype=torch.float64, device=device())
    for t in range(3):
        for j in range(2):
            e = int(ids[t, j])
            gu = X[t].double() @ w13[e].double().T
            h = gu[:I] * torch.sigmoid(gu[:I]) * gu[I:]
            want[t] += float(weights[t, j]) * (w2[e].double() @ h)
    assert w4_ref.rel(y, want) <= 2 * half_step(torch.bfloat16)


@pytest.mark.parametrize("group", [0, 128])
def test_streams_and_graph_replays(group):
    note(f"moe streams and graph, group {group}")
    c = Case(13, 16, 4, 512, 256, torch.bfloat16, group)
    A, B = c.tokens(9), c.tokens(33)
    want = [c.layer(A), c.layer(B)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [(torch.empty_like(A)), (torch.empty_like(B))]
    for _ in range(20):                       # two streams at once, a workspace each
        for s, X, o in zip(streams, (A, B), outs):
            with torch.cuda.stream(s):
                c.layer(X, out=o)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(bits(o), bits(w[0]))
    graph = torch.cuda.CUDAGraph()
    out = torch.empty_like(B)
    with torch.cuda.graph(graph):
        y, ids, weights = c.layer(B, out=out)
    for i in range(5):
        B.copy_(c.tokens(33))
        out.zero_()
        graph.replay()
        eager = c.layer(B)
        torch.cuda.synchronize()
        assert torch.equal(bits(out), bits(eager[0])) and torch.equal(ids, eager[1]), i
        assert torch.equal(weights, eager[2]), i


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("group", [0, 64])
def test_one_token_with_left_out_and_repeated_slots(group, dtype):
    note(f"moe one token, slots, group {group} {dtype}")
    c = Case(5, 6, 4, 260, 140, dtype, group)
    X = c.tokens(1)
    weights = torch.randn((1, 4), generator=c.gen, device=device())
    for slots in ([0, -1, 5, 6], [3, 3, 3, 3], [2 ** 31 - 1, 1, 1, -2 ** 31], [-1, 6, 100, -5]):
        ids = torch.tensor([slots], dtype=torch.int32, device=device())
        y = c.layer.experts(X, ids, weights)
        c.check_y(X, ids, weights, y)
        left = (ids < 0) | (ids >= 6)
        odd = weights.masked_fill(left, float("nan"))
        assert torch.equal(bits(c.layer.experts(X, ids, odd)), bits(y))
        if bool(left.all()):
            assert bool((bits(y) == 0).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,E,topk,H,I,group", [
    (1, 16, 16, 70, 3100, 0), (1, 16, 16, 70, 3100, 128),       # rows of h past one LDS
    (64, 2, 1, 4200, 70, 0), (64, 2, 1, 4200, 70, 32),          # activations in chunks
    (40, 3, 2, 100, 2500, 0), (40, 3, 2, 100, 2500, 64),
    (9, 2, 2, 4500, 3000, 0), (9, 2, 2, 4500, 3000, 128),
    (12, 200, 7, 130, 40, 0), (12, 600, 12, 130, 40, 32)])
def test_long_rows_and_many_experts(T, E, topk, H, I, group, dtype):
    note(f"moe T{T} E{E} k{topk} H{H} I{I} group {group} {dtype}")
    c = Case(T + E + H, E, topk, H, I, dtype, group, zeros=True)
    X = c.tokens(T)
    y, ids, weights = c.layer(X)
    torch.cuda.synchronize()
    c.check_route(X, ids, weights)
    c.check_y(X, ids, weights, y)
    assert torch.equal(bits(c.layer(X)[0]), bits(y))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("group", [0, 32])
@pytest.mark.parametrize("T", [1, 4, 40])
def test_infinities_stay_in_their_token(T, group, dtype):
    note(f"moe infinities T{T} group {group} {dtype}")
    c = Case(7, 4, 2, 260, 140, dtype, group)
    X = c.tokens(T)
    ids = (torch.arange(2 * T, device=device()).view(T, 2) % 4).to(torch.int32)
    weights = torch.rand((T, 2), generator=c.gen, device=device())
    want = c.layer.experts(X, ids, weights)
    for value in (float("inf"), float("-inf"), float("nan")):
        B = X.clone()
        B[T // 2, 137] = value
        y = c.layer.experts(B, ids, weights)
        other = torch.arange(T, device=device()) != T // 2
        assert torch.equal(bits(y[other]), bits(want[other])), "another token changed"
        # gates of both signs: silu has infinities and 0 * inf among its values
        assert not bool(torch.isfinite(y[T // 2]).any())


@pytest.mark.parametrize("group", [0, 64])
def test_replays_beside_eager_calls_and_another_graph(group):
    # captured on a stream that the layer has run on, replayed on others: no
    # workspace is shared
    note(f"moe replays beside eager calls, group {group}")
    c = Case(17, 16, 4, 512, 256, torch.bfloat16, group)
    Xs = [c.tokens(t) for t in (9, 33, 20)]
    want = [c.layer(X)[0].clone() for X in Xs]
    home, away = torch.cuda.Stream(), torch.cuda.Stream()
    home.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(home):
        c.layer(Xs[0])
    torch.cuda.synchronize()
    graphs, outs = [], [torch.empty_like(X) for X in Xs]
    for X, out in zip(Xs[:2], outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=home):
            c.layer(X, out=out)
            c.layer(X, out=out)
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(20):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(away):
            graphs[0].replay()
        graphs[1].replay()
        c.layer(Xs[2], out=outs[2], stream=home)
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(bits(o), bits(w))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,E,topk,H", [(1, 16, 4, 2048), (16, 16, 16, 2048), (3, 1, 1, 2047),
                                        (16, 5, 2, 1500), (16, 16, 3, 2050), (17, 16, 3, 2048),
                                        (16, 17, 3, 2048), (2, 9, 9, 700)])
def test_router_around_one_workgroup(T, E, topk, H, dtype):
    note(f"moe router T{T} E{E} k{topk} H{H} {dtype}")
    c = Case(T + E + H, E, topk, H, 24, dtype, renorm=False)
    X = c.tokens(T)
    ids, weights = c.layer.route(X)
    c.check_route(X, ids, weights)
    y, ids2, weights2 = c.layer(X)
    assert torch.equal(ids, ids2)
    assert bool(((weights - weights2).abs() <= 1e-5 * weights).all())
    c.check_y(X, ids2, weights2, y)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("E,topk,H,group", [(64, 16, 1100, 0), (65, 8, 300, 0), (200, 7, 2100, 64),
                                            (256, 8, 4100, 128), (257, 8, 300, 0),
                                            (256, 16, 64, 32)])
def test_one_token_of_many_experts(E, topk, H, group, dtype):
    note(f"moe one token E{E} k{topk} H{H} group {group} {dtype}")
    c = Case(E + H, E, topk, H, 40, dtype, group, zeros=True)
    for round in range(2):
        X = c.tokens(1)
        if round:                             # equal logits, by rising index
            c.router[3:] = c.router[2]
        y, ids, weights = c.layer(X)
        ids2, weights2 = c.layer.route(X)
        assert torch.equal(ids, ids2) and torch.equal(weights, weights2)
        c.check_route(X, ids, weights)
        c.check_y(X, ids, weights, y)


@pytest.mark.parametrize("H,I", [(1, 140000), (270000, 3)])
def test_more_workgroups_than_one_dimension_of_a_grid(H, I):
    # 512 experts or slots times 8750 or 8438 blocks: the second dimension's last
    # row goes past the end
    E, T, topk = 512, 64, 8
    note(f"moe large grid H{H} I{I}")
    g = gen(H)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=device(), dtype=torch.float16)
    w13, w2 = normal(E, 2 * I, H), normal(E, H, I)
    w13 /= math.sqrt(H)
    w2 /= math.sqrt(I)
    layer = MoeLayer(normal(E, H), w13, w2, topk=topk)
    X = normal(T, H)
    ids = torch.randint(0, E, (T, topk), generator=g, device=device(), dtype=torch.int32)
    weights = torch.rand((T, topk), generator=g, device=device())
    y = layer.experts(X, ids, weights)
    assert torch.equal(bits(layer.experts(X, ids, weights)), bits(y))
    want = torch.zeros((T, H), dtype=torch.float64, device=device())
    for e in sorted(set(ids.flatten().tolist())):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        gu = X[t].double() @ w13[e].double().T
        h = torch.sigmoid(gu[:, :I]) * gu[:, :I] * gu[:, I:]
        want.index_add_(0, t, (h @ w2[e].double().T) * weights[t, j].double().unsqueeze(-1))
    assert w4_ref.rel(y, want) <= 2 * half_step(torch.float16)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,E,topk,H,group", [(2, 1, 1, 100, 0), (2, 2, 2, 300, 64), (8, 8, 8, 500, 0),
                                              (8, 16, 16, 2100, 32), (8, 256, 16, 1100, 0),
                                              (7, 65, 9, 4100, 128), (3, 256, 4, 260, 64),
                                              (9, 64, 6, 520, 0), (4, 257, 8, 520, 64),
                                              (72, 40, 2, 130, 0)])
def test_a_few_tokens_of_few_and_many_experts(T, E, topk, H, group, dtype):
    note(f"moe few tokens T{T} E{E} k{topk} H{H} group {group} {dtype}")
    c = Case(T * E + H, E, topk, H, 56, dtype, group, zeros=True)
    for alike in (False, True):
        X = c.tokens(T)
        if alike:                             # every token with the same experts
            X[:] = X[0] + X * 0.01
            if E > 2:
                c.router[2:] = c.router[1]    # and equal logits, by rising index
        y, ids, weights = c.layer(X)
        ids2, weights2 = c.layer.route(X)
        assert torch.equal(ids, ids2) and torch.equal(weights, weights2)
        c.check_route(X, ids, weights)
        c.check_y(X, ids, weights, y)
        assert torch.equal(bits(c.layer.experts(X, ids, weights)), bits(y))
        assert torch.equal(bits(c.layer(X)[0]), bits(y))


def test_a_nan_token_among_a_few():
    c = Case(6, 12, 3, 260, 40, torch.bfloat16)
    note("moe few tokens, NaN")
    X = c.tokens(5)
    want = c.layer(X)
    B = X.clone()
    B[2, 7] = float("nan")
    y, ids, weights = c.layer(B)
    keep = [0, 1, 3, 4]
    assert torch.equal(ids[keep], want[1][keep]) and torch.equal(weights[keep], want[2][keep])
    assert torch.equal(bits(y[keep]), bits(want[0][keep]))
    assert bool(torch.isnan(weights[2]).all()) and len(set(ids[2].tolist())) == 3


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,E,topk,H,I,group", [(8, 64, 8, 4100, 530, 128), (40, 8, 2, 4130, 4090, 64),
                                                (20, 33, 4, 4096, 1000, 32)])
def test_long_packed_rows(T, E, topk, H, I, group, dtype):
    note(f"moe long packed rows T{T} E{E} k{topk} H{H} I{I} group {group} {dtype}")
    c = Case(T + E + I, E, topk, H, I, dtype, group, zeros=True)
    X = c.tokens(T)
    y, ids, weights = c.layer(X)
    torch.cuda.synchronize()
    c.check_route(X, ids, weights)
    c.check_y(X, ids, weights, y)
    # an infinity stays in its token
    B = X.clone()
    B[T // 2, 137] = float("inf")
    z = c.layer.experts(B, ids, weights)
    other = torch.arange(T, device=device()) != T // 2
    assert torch.equal(bits(z[other]), bits(y[other]))
    assert not bool(torch.isfinite(z[T // 2]).any())
