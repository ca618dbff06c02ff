"""GPU checks of the low-rank adapters beside a projection against plain 64-bit forms.

Tolerances, with u the 16-bit type's half step: small integers and powers of two make every
sum exact (u too, which is then of few bits), so the result is the exact one rounded once, bit
for bit.  Otherwise, with C = sum |X| |W| + |s| sum_j (sum_k |X| |A|) |B| and E the second part
of C: fp32 sums of fewer than 2^8 roundings along any chain (K / 128 matrix instructions, 8
waves, 8 pieces of K, the rank), |D - ref| <= u |ref| + 2^-15 C, and in the 2-norm u |ref|.
Through the large tiles the adapters' part and its u are rounded to 16 bits too and a packed
weight is: 2 u E, u |the part|, u C more; in the 2-norm, where these average out, 2 u |ref|
with a packed weight and 1.5 u without.
"""
from __future__ import annotations

import math
import threading

import pytest
import torch

from dense_gemm_18_amd import LoraAdapters, W4Weight, binding, gemm_nt_lora, rms_norm
from tests import w4_ref
from tests.gpu_util import device, note
from tests.test_gpu_w4 import bits, check_guard, gen, strided
from tests.w4_ref import TYPES, half_step, rel

pytestmark = pytest.mark.gpu


def large(M, N, K, group):
    """Whether a dense call goes through the large tiles."""
    if group:
        return M > 384
    if M <= 16:
        return N > 4096 and M * (-(-K // 128) * 256 + 16) > 66 * 1024
    return (M > 32 or K > 2048) and (N > 2048 or -(-M // 32) * -(-N // 32) > 256)


class Case:
    def __init__(self, seed, M, N, K, rank, count, dtype, group=0, zeros=False, scales=True):
        g = self.gen = gen(seed)
        self.group, self.dtype, self.count, self.rank = group, dtype, count, rank

        def normal(scale, *shape):
            return (torch.randn(shape, generator=g, device=device()) * scale).to(dtype)
        self.X = normal(1.0, M, K)
        if group:
            raw = w4_ref.random_weight(g, N, K, group, zeros, dtype, scale=0.25 / math.sqrt(K))
            self.w = W4Weight(*raw, shape=(N, K), group=group)
            self.W = w4_ref.values(*raw, K, group)
        else:
            self.w = normal(1 / math.sqrt(K), N, K)
            self.W = self.w.double()
        self.A, self.B = normal(1 / math.sqrt(K), count, rank, K), normal(0.3, count, N, rank)
        self.s = torch.rand((count,), generator=g, device=device()) + 0.5 if scales else None
        self.adapters = LoraAdapters(self.A, self.B, self.s)
        self.ids = torch.randint(-1, count, (M,), generator=g, device=device()).to(torch.int32)

    def reference(self, X=None, ids=None):
        """(D, its sizes C, the adapters' part's E, that part) in 64 bits."""
        X = (self.X if X is None else X).double()
        ids = self.ids if ids is None else ids
        part = torch.zeros((X.shape[0], self.W.shape[0]), dtype=torch.float64, device=device())
        size = torch.zeros_like(part)
        for a in range(self.count):
            t = torch.nonzero(ids == a).squeeze(1)
            if len(t):
                s = 1.0 if self.s is None else float(self.s[a])
                A, B = self.A[a].double(), self.B[a].double()
                part[t] = X[t] @ A.T @ B.T * s
                size[t] = X[t].abs() @ A.abs().T @ B.abs().T * s
        return X @ self.W.T + part, X.abs() @ self.W.abs().T + size, size, part

    def check(self, D, X=None, ids=None, dense=True):
        ref, C, E, part = self.reference(X, ids)
        u, tiny = half_step(self.dtype), torch.finfo(self.dtype).smallest_normal
        bound = u * ref.abs() + 2.0 ** -15 * C + tiny
        most = u
        if dense and large(*ref.shape, self.X.shape[1], self.group):
            bound += 2 * u * E + u * part.abs() + (u * C if self.group else 0)
            most = (2 if self.group else 1.5) * u
        assert D.dtype == self.dtype and D.shape == ref.shape
        assert not bool(((D.double() - ref).abs() > bound).any())
        if ref.numel() >= 64:
            assert rel(D, ref) <= most

    def run(self, **kw):
        return gemm_nt_lora(self.X, self.w, self.adapters, self.ids, **kw)


#          M    N     K   rank count group zeros
CASES = [(1, 1, 1, 1, 1, 0, False), (1, 64, 128, 8, 1, 0, False), (1, 4100, 1000, 16, 3, 0, False),
         (2, 300, 2050, 12, 5, 0, False), (7, 130, 4099, 33, 2, 0, False),
         (16, 5000, 640, 64, 20, 0, False), (16, 4100, 2100, 16, 20, 0, False),
         (3, 9000, 11300, 16, 2, 0, False), (250, 1000, 1100, 30, 6, 0, False),
         (20, 9000, 1030, 16, 20, 0, False), (32, 4100, 2056, 24, 9, 0, False), (16, 100, 300, 256, 4, 0, False),
         (17, 64, 130, 100, 3, 0, False), (31, 2000, 1024, 16, 40, 0, False),
         (33, 777, 515, 5, 7, 0, False), (64, 1000, 2048, 16, 32, 0, False),
         (64, 5000, 512, 16, 70, 0, False), (65, 4096, 264, 64, 9, 0, False),
         (70, 3001, 1030, 20, 3, 0, False), (300, 1500, 520, 256, 6, 0, False),
         (500, 700, 2000, 129, 100, 0, False), (1025, 1030, 777, 17, 3, 0, False),
         (1500, 700, 1300, 64, 9, 0, False), (2100, 520, 520, 250, 5, 0, False),
         (600, 2501, 6, 8, 3, 0, False), (2000, 3001, 1100, 16, 5, 0, False),
         (2049, 4100, 520, 24, 4, 0, False), (2048, 4096, 512, 16, 4, 0, False),
         (1300, 2049, 600, 40, 4, 0, False), (700, 1030, 1024, 48, 3, 64, True),
         (1, 64, 128, 8, 1, 128, False), (1, 4100, 1000, 16, 3, 32, True),
         (5, 18500, 384, 16, 3, 64, True), (13, 5000, 2050, 12, 5, 32, True),
         (16, 300, 700, 256, 4, 64, False), (17, 8300, 260, 128, 3, 128, True),
         (40, 9000, 300, 64, 6, 32, False), (64, 16500, 256, 64, 5, 64, True),
         (64, 260, 1030, 200, 8, 128, False), (130, 5000, 390, 32, 9, 128, True),
         (384, 300, 520, 256, 20, 64, False), (385, 1000, 1032, 16, 9, 128, True),
         (600, 515, 999, 100, 3, 32, False)]


@pytest.mark.parametrize("M,N,K,rank,count,group,zeros", CASES)
@pytest.mark.parametrize("dtype", TYPES)
def test_against_64_bits(M, N, K, rank, count, group, zeros, dtype):
    note(f"lora {M}x{N}x{K} rank {rank} of {count} group {group} {dtype}")
    c = Case(M + N + K, M, N, K, rank, count, dtype, group, zeros, scales=count != 3)
    D = c.run()
    c.check(D)
    assert torch.equal(bits(c.run()), bits(D))
    for ids in (torch.full_like(c.ids, -1), torch.full_like(c.ids, count - 1),
                torch.sort(c.ids).values, torch.arange(M, device=device()).int() % count,
                torch.where(c.ids == 0, 2 ** 31 - 1, c.ids)):
        c.ids = ids.contiguous()
        c.check(c.run())


@pytest.mark.parametrize("M,N,K,rank,count,group", [
    (1, 300, 256, 8, 2, 0), (9, 4200, 130, 16, 4, 0), (30, 700, 515, 12, 9, 0),
    (64, 5000, 264, 16, 3, 0), (400, 1000, 136, 20, 5, 0), (5, 300, 256, 16, 3, 64),
    (100, 700, 390, 12, 9, 32), (400, 600, 256, 16, 3, 128)])
@pytest.mark.parametrize("dtype", TYPES)
def test_integers_are_exact(M, N, K, rank, count, group, dtype):
    note(f"lora integers {M}x{N}x{K} rank {rank} group {group} {dtype}")
    g = gen(M + K)

    def ints(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=g, device=device()).to(dtype)
    X = ints(-1, 2, M, K)
    A = torch.zeros((count, rank, K), dtype=dtype, device=device())
    A[:, :, :3] = ints(-1, 2, count, rank, 3)          # |s u| <= 6 in halves
    B = torch.zeros((count, N, rank), dtype=dtype, device=device())
    B[:, :, -4:] = ints(-1, 2, count, N, 4)            # the part: <= 24 in halves, 6 bits
    if group:
        Q, _, Z = w4_ref.random_weight(g, N, K, group, True, dtype)
        S = torch.full((N, -(-K // group)), 0.5, dtype=dtype, device=device())
        w, W = W4Weight(Q, S, Z, shape=(N, K), group=group), w4_ref.values(Q, S, Z, K, group)
    else:
        w = ints(-2, 3, N, K)
        W = w.double()
    s = 2.0 ** torch.randint(-1, 2, (count,), generator=g, device=device()).float()
    ids = torch.randint(-1, count, (M,), generator=g, device=device()).to(torch.int32)
    D = gemm_nt_lora(X, w, LoraAdapters(A, B, s), ids)
    at = ids.clamp(min=0).long()
    u = (X.double().unsqueeze(1) * A.double()[at]).sum(-1) * s.double()[at, None]
    part = (u.unsqueeze(1) * B.double()[at]).sum(-1) * (ids >= 0)[:, None]
    assert torch.equal(bits(D), bits((X.double() @ W.T + part).to(dtype) + 0.0))


@pytest.mark.parametrize("M,group", [(1, 0), (40, 0), (1, 32), (100, 64)])
@pytest.mark.parametrize("dtype", TYPES)
def test_rows_without_an_adapter(M, group, dtype):
    note(f"lora none M{M} group {group} {dtype}")
    c = Case(5, M, 200, 515, 16, 3, dtype, group)
    c.ids.fill_(-1)
    none = LoraAdapters(c.A[:0], c.B[:0])
    D = gemm_nt_lora(c.X, c.w, none, torch.zeros_like(c.ids))
    assert torch.equal(bits(D), bits(c.run()))
    c.check(D)


@pytest.mark.parametrize("M,N,K,rank", [(20, 300, 300, 16), (40, 5000, 300, 16),
                                        (500, 300, 300, 16), (600, 2300, 300, 64),
                                        (16, 4200, 2200, 16)])
@pytest.mark.parametrize("group", [0, 128])
def test_infinities_and_nans_stay_where_they_are(M, N, K, rank, group):
    note(f"lora NaN M{M} N{N} group {group}")
    c = Case(6, M, N, K, rank, 4, torch.bfloat16, group)
    c.ids[:8] = torch.tensor([0, 1, 2, 3, -1, 0, 1, 2], device=device())
    want = c.run()
    c.A[1, 3, 7] = math.nan
    c.B[2, 5, 2] = math.inf
    c.X[0, 9] = math.nan
    D = c.run()
    assert bool(D[c.ids == 1].isnan().all()) and bool(D[0].isnan().all())
    assert not bool(torch.isfinite(D[c.ids == 2][:, 5]).any())
    others = (c.ids != 1) & (c.ids != 2)
    others[0] = False
    assert torch.equal(bits(D[others]), bits(want[others]))
    two = c.ids == 2
    two[0] = False
    columns = torch.arange(N, device=device()) != 5
    assert torch.equal(bits(D[two][:, columns]), bits(want[two][:, columns]))


@pytest.mark.parametrize("M", [3, 33, 450])
@pytest.mark.parametrize("group", [0, 64])
@pytest.mark.parametrize("dtype", TYPES)
def test_strides_and_what_lies_around(M, group, dtype):
    note(f"lora strides M{M} group {group} {dtype}")
    N, K = 1500, 517
    c = Case(M, M, N, K, 12, 6, dtype, group)
    _, X = strided(M, K, K + 5, dtype)
    X.copy_(c.X)
    buf, out = strided(M, N, N + 3, dtype)
    ws = torch.full((binding.gemm_nt_lora_ws_size(M, N, K, 12, group),), 0xFF, dtype=torch.uint8,
                    device=device())
    got = gemm_nt_lora(X, c.w, c.adapters, c.ids, out=out, workspace=ws)
    assert got is out
    torch.cuda.synchronize()
    check_guard(buf, M, N, N + 3, dtype)
    c.check(out, dense=False)
    # dense, in a buffer of NaNs, with a workspace of NaNs
    buf, out = strided(M, N, N, dtype)
    ws.fill_(0xFF)
    gemm_nt_lora(c.X, c.w, c.adapters, c.ids, out=out, workspace=ws)
    torch.cuda.synchronize()
    check_guard(buf, M, N, N, dtype)
    c.check(out)
    # operands at odd elements
    if not group:
        held = []
        for t in (c.w, c.A, c.B):
            b = torch.empty(t.numel() + 1, dtype=dtype, device=device())
            b[1:].copy_(t.flatten())
            held.append(b[1:].view(t.shape))
        D = gemm_nt_lora(c.X, held[0], LoraAdapters(held[1], held[2], c.s), c.ids)
        c.check(D)


def test_no_rows():
    c = Case(1, 4, 50, 64, 8, 2, torch.float16)
    D = gemm_nt_lora(c.X[:0], c.w, c.adapters, c.ids[:0])
    assert D.shape == (0, 50)


@pytest.mark.parametrize("M,group", [(1, 0), (64, 0), (64, 64), (400, 128)])
def test_replayed_and_on_another_stream(M, group):
    note(f"lora graph M{M} group {group}")
    c = Case(8, M, 5000, 700, 16, 5, torch.bfloat16, group)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    D = c.run(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    want = c.run()
    assert torch.equal(bits(D), bits(want))
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = c.run()
        graphs.append((graph, got))
    for _ in range(3):
        for graph, got in graphs:
            graph.replay()
        torch.cuda.synchronize()
        eager = c.run()
        for _, got in graphs:
            assert torch.equal(bits(got), bits(eager))
        c.X.mul_(-0.5)
        c.ids.copy_(c.ids.roll(1))


@pytest.mark.parametrize("M,group", [(64, 0), (400, 64), (5, 32)])
def test_threads_that_share_a_stream_and_a_workspace(M, group):
    """Each call's launches are enqueued side by side, so another's u never comes between."""
    note(f"lora threads M{M} group {group}")
    cases = [Case(20 + k, M, 2500, 520, 16, 5, torch.bfloat16, group) for k in range(2)]
    want = [c.run() for c in cases]
    ws = torch.empty(binding.gemm_nt_lora_ws_size(M, 2500, 520, 16, group), dtype=torch.uint8,
                     device=device())
    got = [[torch.empty_like(want[k]) for _ in range(30)] for k in range(2)]
    stream = torch.cuda.current_stream()

    def calls(k):
        with torch.cuda.stream(stream):
            for out in got[k]:
                cases[k].run(out=out, workspace=ws)
    threads = [threading.Thread(target=calls, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for k in range(2):
        assert all(torch.equal(bits(out), bits(want[k])) for out in got[k])


@pytest.mark.parametrize("T", [1, 6, 70])
@pytest.mark.parametrize("dtype", TYPES)
def test_norm_projection_with_adapters_and_gated_experts(T, dtype):
    """The operators together as a step uses them: each against its own formula on what the
    one before left."""
    note(f"norm, adapters, gated experts T{T} {dtype}")
    from tests.test_gpu_gate import GatedCase
    from tests.test_gpu_norm import check_y, make, reference
    H, E = 512, 16
    x, w, r = make(gen(T), T, H, dtype)
    c = Case(T, T, H, H, 16, 3, dtype, 64, True)
    bias = torch.randn((E,), generator=gen(3), device=device()) * 0.1
    m = GatedCase(T, E, 4, H, 256, dtype, 64, True, scoring="sigmoid", bias=bias, groups=4,
                  topk_groups=2, group_top=2, scale=1.5)

    def step():
        h, s = rms_norm(x, w, residual=r)
        y = gemm_nt_lora(h, c.w, c.adapters, c.ids)
        h2, s2 = rms_norm(y, w, residual=s)
        z, ids, weights = m.layer(h2)
        return h, s, y, h2, s2, z, ids, weights
    h, s, y, h2, s2, z, ids, weights = step()
    check_y(h, reference(x, w, r), dtype)
    c.check(y, h)
    check_y(h2, reference(y, w, s), dtype)
    m.check_gated(h2, ids, weights)
    m.check_y(h2, ids, weights, z)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, step()))
        x.mul_(-0.5)


def test_refusals():
    c = Case(2, 4, 50, 64, 8, 2, torch.float16)
    for kw in (dict(X=c.X[:, :63]), dict(w=c.w[:49]), dict(ids=c.ids[:3]), dict(ids=c.ids.long()),
               dict(ids=c.ids.cpu()), dict(out=c.X)):
        a = dict(X=c.X, w=c.w, adapters=c.adapters, ids=c.ids)
        a.update(kw)
        with pytest.raises(ValueError):
            gemm_nt_lora(**a)
    with pytest.raises(TypeError):
        gemm_nt_lora(c.X.bfloat16(), c.w, c.adapters, c.ids)
    with pytest.raises(TypeError):
        gemm_nt_lora(c.X, c.w.bfloat16(), c.adapters, c.ids)
    with pytest.raises(binding.GemmError):
        c.run(workspace=torch.empty(8, dtype=torch.uint8, device=device()))
    with pytest.raises(ValueError):
        LoraAdapters(c.A, c.B[:1])
    with pytest.raises(ValueError):
        LoraAdapters(c.A.transpose(0, 1), c.B)
    with pytest.raises(TypeError):
        LoraAdapters(c.A, c.B.bfloat16())
    with pytest.raises(TypeError):
        LoraAdapters(c.A, c.B, c.s.double())
