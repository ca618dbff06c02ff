"""GPU checks of the choice of experts from logits against plain 64-bit forms.

Tolerances: ids are equal (logits are given, choices are formed in 64 bits).  Weights are
formed in 64 bits and rounded to fp32, 2^-24; a softmax's sum over all experts, formed in
fp32 where there is neither a bias nor a sum of two, adds the roundings of 16 terms and 6
joins and an exponential's 2: 2^-24 * 32 in all.  In a layer the logits are fp32 sums: those
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
