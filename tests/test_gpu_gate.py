"""GPU checks of the choice of experts from logits against plain 64-bit forms.

Tolerances: ids are equal (logits are given, choices decided as in 64 bits).  Weights are formed
in fp32: a softmax's sum over all experts takes 16 terms and 6 joins, exponentials 2 each, the
chosen ones' sum 4 joins, quotients and products 4: 2^-24 * 32 in all.  In a layer the logits are fp32 sums: those
of the layer's own tests.
"""
from __future__ import annotations

import math

import pytest
import torch

from dense_gemm_18_amd import MoeLayer, choose_experts
from tests.gpu_util import device, note
from tests.test_gpu_moe import Case
from tests.test_gpu_w4 import bits, gen
from tests.w4_ref import TYPES

pytestmark = pytest.mark.gpu


def scores_of(logits, scoring):
    l = logits.double()
    if scoring == "sigmoid":
        return 1 / (1 + torch.exp(-l))
    return torch.exp(l - torch.logsumexp(l, -1, keepdim=True))


def reference(logits, topk, scoring="softmax", bias=None, groups=1, topk_groups=None,
              group_top=1, renormalize=True, scale=1.0):
    """Row by row, on the host, from the definition."""
    score = scores_of(logits, scoring).cpu()
    T, E = score.shape
    choice = score if bias is None else score + bias.double().cpu()
    kept, n = groups if topk_groups is None else topk_groups, E // groups
    ids = torch.empty((T, topk), dtype=torch.int32)
    weights = torch.empty((T, topk), dtype=torch.float64)
    for t, row in enumerate(choice.tolist()):
        value = [sum(sorted(row[g * n:(g + 1) * n], reverse=True)[:group_top])
                 for g in range(groups)]
        best = sorted(range(groups), key=lambda g: (-value[g], g))[:kept]
        among = [e for g in best for e in range(g * n, (g + 1) * n)]
        chosen = sorted(among, key=lambda e: (-row[e], e))[:topk]
        ids[t] = torch.tensor(chosen, dtype=torch.int32)
        w = score[t, chosen]
        weights[t] = (w / w.sum() if renormalize else w) * scale
    return ids.to(logits.device), weights.to(logits.device)


def check(logits, topk, **kw):
    ids, weights = choose_experts(logits, topk, **kw)
    want_ids, want = reference(logits, topk, **kw)
    assert ids.dtype == torch.int32 and weights.dtype == torch.float32
    assert torch.equal(ids, want_ids)
    bound = 2.0 ** -24 * 32 * want.abs() + 2.0 ** -149
    assert bool(((weights.double() - want).abs() <= bound).all())
    return ids, weights


#        T    E   topk groups kept group_top
CASES = [(1, 1, 1, 1, 1, 1), (1, 2, 2, 1, 1, 1), (3, 8, 2, 1, 1, 1), (1, 64, 8, 1, 1, 1),
         (5, 60, 4, 1, 1, 1), (70, 64, 6, 8, 3, 1), (9, 65, 16, 5, 2, 2), (33, 128, 8, 16, 4, 2),
         (130, 256, 8, 8, 4, 2), (2, 255, 8, 3, 1, 2), (7, 320, 8, 20, 7, 1), (4, 512, 16, 64, 9, 2),
         (3, 513, 5, 27, 2, 2), (6, 1024, 16, 2, 1, 1), (1, 1024, 16, 64, 64, 2),
         (11, 96, 3, 48, 3, 2), (12, 40, 10, 40, 10, 1)]


@pytest.mark.parametrize("T,E,topk,groups,kept,group_top", CASES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
def test_against_64_bits(T, E, topk, groups, kept, group_top, dtype):
    note(f"gate T{T} E{E} k{topk} groups {kept} of {groups} {dtype}")
    g = gen(T + E + topk)
    logits = (torch.randn((T, E), generator=g, device=device()) * 2).to(dtype)
    bias = torch.randn((E,), generator=g, device=device()) * 0.1
    for scoring in ("softmax", "sigmoid"):
        for b in (None, bias):
            for renorm, scale in ((True, 1.0), (False, 2.5)):
                check(logits, topk, scoring=scoring, bias=b, groups=groups, topk_groups=kept,
                      group_top=group_top, renormalize=renorm, scale=scale)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_equal_choices_go_by_index(scoring):
    note(f"gate ties {scoring}")
    for E, groups in ((16, 4), (100, 10), (256, 8), (300, 6)):
        logits = torch.randint(0, 2, (40, E), generator=gen(E), device=device()).float()
        logits[0] = 0
        for b in (None, torch.zeros(E, device=device())):
            for top in (1, 2):
                check(logits, 4, scoring=scoring, bias=b, groups=groups, topk_groups=2,
                      group_top=top)
    logits[:] = -0.0
    logits[:, 5] = 0.0                                  # both zeros are one logit
    assert choose_experts(logits, 3)[0].tolist() == [[0, 1, 2]] * 40


@pytest.mark.parametrize("bias", [False, True])
def test_infinities_and_nans(bias):
    note(f"gate infinities, bias {bias}")
    E = 72
    logits = torch.randn((8, E), generator=gen(4), device=device())
    b = torch.linspace(0.1, 0.2, E, device=device()) if bias else None
    logits[1, 10:] = -math.inf                          # masked experts
    logits[2] = -math.inf                               # all of them
    logits[3, 7] = math.nan
    logits[4, 9] = math.inf
    rows = [0, 1, 5, 6, 7]
    for scoring in ("softmax", "sigmoid"):
        for groups, kept in ((1, 1), (6, 3)):
            kw = dict(scoring=scoring, bias=b, groups=groups, topk_groups=kept, group_top=2)
            ids, weights = choose_experts(logits, 8, **kw)
            check(logits[rows], 8, **kw)
            assert all(len(set(r)) == 8 and min(r) >= 0 and max(r) < E for r in ids.tolist())
            assert bool(weights[3].isnan().all())
            if scoring == "softmax":
                assert bool(weights[2].isnan().all()) and bool(weights[4].isnan().all())
            else:
                assert bool((weights[2] == 0).all())
                assert bool(torch.isfinite(weights[4]).all()) and 9 in ids[4].tolist()


def test_bias_that_shuts_experts_out():
    note("gate bias -inf")
    logits = torch.randn((50, 64), generator=gen(5), device=device())
    bias = torch.zeros(64, device=device())
    bias[::2] = -math.inf
    for groups, kept in ((1, 1), (8, 4)):
        ids, _ = check(logits, 6, scoring="sigmoid", bias=bias, groups=groups, topk_groups=kept,
                       group_top=1)
        assert bool((ids % 2 == 1).all())
    bias[1] = math.inf
    assert bool((check(logits, 6, scoring="sigmoid", bias=bias)[0][:, 0] == 1).all())
    bias[:] = math.nan
    ids, weights = choose_experts(logits, 6, bias=bias)
    assert all(len(set(r)) == 6 for r in ids.tolist()) and bool(torch.isfinite(weights).all())


def test_values_next_to_a_border():
    """Choices one fp32 rounding apart: 64 bits tell them apart."""
    note("gate borders")
    E = 128
    base = torch.randn((200, 1), generator=gen(6), device=device())
    logits = base * torch.ones(E, device=device())
    step = torch.randint(-3, 4, (200, E), generator=gen(7), device=device()).float()
    logits = logits + step * logits.abs() * 2.0 ** -23
    bias = torch.full((E,), 0.3, device=device())
    check(logits, 8, scoring="sigmoid", bias=bias)
    check(logits, 8, scoring="sigmoid", bias=bias, groups=8, topk_groups=2, group_top=2)
    check(logits, 8, scoring="softmax", bias=bias)


def test_row_strides_many_rows_and_none():
    note("gate strides")
    wide = torch.randn((300, 100), generator=gen(8), device=device())
    view = wide[:, 3:67]
    ids, weights = check(view, 5)
    again = choose_experts(view.contiguous(), 5)
    assert torch.equal(ids, again[0]) and torch.equal(weights, again[1])
    ids, weights = choose_experts(wide[:0], 5)
    assert ids.shape == (0, 5) and weights.shape == (0, 5)
    logits = torch.randn((70001, 32), generator=gen(9), device=device())
    ids, _ = choose_experts(logits, 4, scoring="sigmoid")
    assert torch.equal(ids.long(), torch.sort(logits, -1, descending=True).indices[:, :4])


class GatedCase(Case):
    def __init__(self, *args, **kw):
        super().__init__(*args)
        self.kw = kw
        g = self.layer
        self.layer = MoeLayer(g.router, g.w13, g.w2, topk=self.topk, **kw)

    def check_gated(self, X, ids, weights):
        """The choice of the exact logits up to fp32's error in them."""
        kw = self.kw
        logits = X.double() @ self.router.double().T
        slack = 2.0 ** -22 * math.sqrt(self.H) * 8
        score = scores_of(logits, kw.get("scoring", "softmax"))
        choice = score if kw.get("bias") is None else score + kw["bias"].double()
        at = ids.long()
        assert bool(((at >= 0) & (at < self.E)).all())
        G = kw.get("groups", 1)
        kept, n = kw.get("topk_groups") or G, self.E // G
        value = torch.topk(choice.view(-1, G, n), kw.get("group_top", 1), dim=-1).values.sum(-1)
        used = torch.zeros_like(value).scatter_(1, at // n, 1.0) > 0
        assert int(used.sum(-1).max()) <= kept
        # every group used is among the largest, every expert left out of them smaller
        edge = torch.topk(value, kept, dim=-1).values[:, -1:]
        assert bool((value >= edge - slack)[used].all())
        chosen = choice.gather(1, at)
        assert bool((chosen[:, :-1] >= chosen[:, 1:] - slack).all())
        rest = choice.scatter(1, at, -math.inf).masked_fill(
            ~used.repeat_interleave(n, 1), -math.inf)
        assert bool((rest.amax(-1) <= chosen[:, -1] + slack).all())
        w = score.gather(1, at)
        if kw.get("renormalize", True):
            w = w / w.sum(-1, keepdim=True)
        w = w * kw.get("scale", 1.0)
        assert bool(((weights.double() - w).abs() <= 1e-5 * w + 1e-30).all())


#        T   E  topk  H    I  group  groups kept top
LAYERS = [(1, 8, 2, 128, 64, 0, 1, 1, 1), (1, 64, 8, 1000, 130, 64, 8, 3, 2),
          (1, 300, 8, 2049, 24, 0, 10, 4, 2), (5, 16, 3, 300, 70, 32, 4, 2, 1),
          (16, 64, 6, 2200, 40, 0, 8, 4, 2), (64, 32, 4, 260, 64, 0, 1, 1, 1),
          (130, 24, 5, 200, 48, 128, 6, 2, 2)]


@pytest.mark.parametrize("T,E,topk,H,I,group,groups,kept,top", LAYERS)
@pytest.mark.parametrize("dtype", TYPES)
def test_layer(T, E, topk, H, I, group, groups, kept, top, dtype):
    note(f"gated layer T{T} E{E} k{topk} H{H} I{I} group {group} {dtype}")
    bias = torch.randn((E,), generator=gen(E), device=device()) * 0.1
    for kw in (dict(scoring="sigmoid", bias=bias, groups=groups, topk_groups=kept, group_top=top,
                    scale=2.5), dict(scoring="sigmoid", renormalize=False),
               dict(groups=groups, topk_groups=kept)):
        c = GatedCase(T + E + H, E, topk, H, I, dtype, group, **kw)
        X = c.tokens(T)
        y, ids, weights = c.layer(X)
        c.check_gated(X, ids, weights)
        c.check_y(X, ids, weights, y)
        ids2, weights2 = c.layer.route(X)
        assert torch.equal(ids, ids2) and torch.equal(weights, weights2)
        assert torch.equal(bits(c.layer.experts(X, ids, weights)), bits(y))


@pytest.mark.parametrize("T", [1, 6])
def test_layer_replayed(T):
    note(f"gated layer graph T{T}")
    bias = torch.randn((32,), generator=gen(3), device=device()) * 0.1
    c = GatedCase(7, 32, 4, 512, 128, torch.bfloat16, scoring="sigmoid", bias=bias, groups=4,
                  topk_groups=2, group_top=2)
    X = c.tokens(T)
    c.layer(X)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = c.layer(X)
        logits = choose_experts(X[:, :32], 4)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        eager = c.layer(X)
        assert all(torch.equal(a, b) for a, b in zip(got, eager))
        assert all(torch.equal(a, b) for a, b in zip(logits, choose_experts(X[:, :32], 4)))
        X.mul_(-0.75)
        bias.mul_(0.5)


def vectorised(logits, topk, scoring="softmax", bias=None, groups=1, topk_groups=None,
               group_top=1, renormalize=True, scale=1.0):
    """The reference for many rows."""
    score = scores_of(logits, scoring)
    T, E = score.shape
    choice = score if bias is None else score + bias.double()
    kept, n = groups if topk_groups is None else topk_groups, E // groups
    value = torch.topk(choice.view(T, groups, n), group_top, dim=-1).values.sum(-1)
    best = torch.sort(value, dim=-1, descending=True, stable=True).indices[:, :kept]
    keep = torch.zeros((T, groups), dtype=torch.bool, device=device()).scatter_(1, best, True)
    choice = choice.masked_fill(~keep.repeat_interleave(n, 1), -math.inf)
    ids = torch.sort(choice, dim=-1, descending=True, stable=True).indices[:, :topk]
    w = score.gather(1, ids)
    if renormalize:
        w = w / w.sum(-1, keepdim=True)
    return ids.to(torch.int32), w * scale


def settled(logits, scoring, bias, groups, topk_groups, group_top, **_):
    """Rows whose groups 64 bits tell apart: of two sums of two choices that differ by less
    than 2^-50 of themselves, four roundings of 2^-53 and an exponential's two, which is
    larger hangs on those roundings (logits of a - d, a + d against a, a have sums that
    differ by d^2, here 2^-47 of a 64th part of them)."""
    score = scores_of(logits, scoring)
    choice = score if bias is None else score + bias.double()
    value = torch.topk(choice.view(len(choice), groups, -1), group_top, dim=-1).values.sum(-1)
    value = torch.sort(value, dim=-1, descending=True).values
    if topk_groups >= groups:
        return torch.ones(len(choice), dtype=torch.bool, device=device())
    a, b = value[:, topk_groups - 1], value[:, topk_groups]
    return a - b > 2.0 ** -50 * a.abs()


def check_many(logits, topk, **kw):
    ids, weights = choose_experts(logits, topk, **kw)
    want_ids, want = vectorised(logits, topk, **kw)
    same = (ids == want_ids).all(-1)
    if kw.get("group_top", 1) == 2:
        same |= ~settled(logits, **kw)
    assert bool(same.all())
    weights, want = weights[(ids == want_ids).all(-1)], want[(ids == want_ids).all(-1)]
    # below the smallest normal number an exponential, its correction, a quotient and a
    # product are off by up to 2, 1/2, 1/2 and 1/2 steps, and the quotient and the scale
    # make the ones before them up to 4 times larger here
    tiny = 16 * 2.0 ** -149
    assert bool(((weights.double() - want).abs() <= 2.0 ** -24 * 32 * want + tiny).all())
    return ids, weights


#       T    E   topk groups kept
MANY = [(1024, 64, 6, 1, 1), (1025, 64, 8, 8, 3), (2047, 128, 1, 1, 1), (3001, 128, 8, 16, 5),
        (1500, 256, 8, 8, 4), (4099, 256, 14, 1, 1), (1026, 256, 5, 2, 1), (1027, 256, 15, 4, 3),
        (2050, 256, 8, 8, 4), (2100, 256, 5, 2, 1), (2049, 256, 14, 16, 7), (1100, 256, 8, 32, 7), (1100, 200, 8, 8, 2), (2000, 64, 14, 4, 1), (1111, 128, 4, 4, 2)]


@pytest.mark.parametrize("T,E,topk,groups,kept", MANY)
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
def test_many_tokens(T, E, topk, groups, kept, dtype):
    note(f"gate many T{T} E{E} k{topk} groups {kept} of {groups} {dtype}")
    g = gen(T + E + topk)
    wide = (torch.randn((T, E + 3), generator=g, device=device()) * 2).to(dtype)
    bias = torch.randn((E,), generator=g, device=device()) * 0.1
    for logits in (wide[:, :E].contiguous(), wide[:, 1:E + 1]):
        for scoring in ("softmax", "sigmoid"):
            for b in (None, bias, bias * 30):
                for renorm, top in ((True, 1), (False, 2)):
                    check_many(logits, topk, scoring=scoring, bias=b, groups=groups,
                               topk_groups=kept, group_top=top, renormalize=renorm,
                               scale=2.5 if renorm else 1.0)


@pytest.mark.parametrize("E", [64, 128, 256])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_many_tokens_with_equal_and_close_choices(E, dtype):
    note(f"gate many ties E{E} {dtype}")
    g = gen(E)
    T = 2100 if E == 256 else 1200
    few = torch.randint(-2, 3, (T, E), generator=g, device=device()).to(dtype)
    close = torch.randn((T, 1), generator=g, device=device()) * torch.ones(E, device=device())
    step = torch.randint(-3, 4, (T, E), generator=g, device=device()).float()
    close = (close + step * close.abs() * 2.0 ** -23).to(dtype)
    flat = torch.full((T, E), -3.0, dtype=dtype, device=device())
    far = (torch.randn((T, E), generator=g, device=device()) * 40).to(dtype)
    for logits in (few, close, flat, far):
        for b in (None, torch.full((E,), 0.3, device=device())):
            for groups, kept, top in ((1, 1, 1), (8, 2, 2), (4, 2, 1)):
                kw = dict(bias=b, groups=groups, topk_groups=kept, group_top=top)
                # a sigmoid that rounds to 1 in 64 bits hides the order of its logits
                if logits is not far:
                    check_many(logits, 6, scoring="sigmoid", **kw)
                check_many(logits, 6, scoring="softmax", **kw)


def test_many_tokens_with_infinities_and_nans():
    note("gate many infinities")
    E = 128
    logits = torch.randn((1300, E), generator=gen(11), device=device())
    logits[::7, 40:90] = -math.inf
    logits[5] = math.nan
    logits[9, 3] = math.nan
    logits[11] = -math.inf
    rows = torch.ones(1300, dtype=torch.bool, device=device())
    rows[[5, 9, 11]] = False
    for b in (None, torch.linspace(0.1, 0.2, E, device=device())):
        for scoring in ("softmax", "sigmoid"):
            kw = dict(scoring=scoring, bias=b, groups=4, topk_groups=2, group_top=2)
            ids, weights = choose_experts(logits, 8, **kw)
            want_ids, want = vectorised(logits[rows], 8, **kw)
            assert torch.equal(ids[rows], want_ids)
            assert bool(((weights[rows].double() - want).abs() <= 2.0 ** -24 * 32 * want).all())
            assert bool(weights[5].isnan().all()) and bool(weights[9].isnan().all())
            for r in (5, 9, 11):
                assert len(set(ids[r].tolist())) == 8 and int(ids[r].min()) >= 0
                assert int(ids[r].max()) < E
