"""GPU checks of the root-mean-square norm against plain 64-bit forms.

Tolerances.  y before its rounding: s is an fp32 sum (2^-24), the sum of squares a chain of
at most 32 terms in a lane (H / 1024 where rows are longer than registers) and 10 joins,
halved by the root; root, quotient and two products 4 more: f = 2^-24 (32 + H / 1024) |y|
covers them.  16-bit rows: one rounding, u |y| (u: the type's half step), or half the smallest
subnormal.  s: fp32, rounded once: bit for bit.  Scales: f of the largest |y| and 2^-24 for
the quotient.  8 bits: q * scale is within half a step of y, 2^-4 |y| (e4m3) or 2^-3 |y| (e5m2)
or half the smallest subnormal times the scale, and f for y and the scale each and 2 more
roundings of the quotient.
"""
from __future__ import annotations

import math

import pytest
import torch

from dense_gemm_18_amd import gemm_nt, rms_norm, rms_norm_fp8
from tests.gpu_util import device, note
from tests.test_gpu_w4 import bits, check_guard, gen, strided
from tests.w4_ref import TYPES, half_step

pytestmark = pytest.mark.gpu

FP8 = {torch.float8_e4m3fn: (448.0, 2.0 ** -4, 2.0 ** -10),
       torch.float8_e5m2: (57344.0, 2.0 ** -3, 2.0 ** -17)}
EPS = 1e-6


def fp32(H):
    return 2.0 ** -24 * (32 + H / 1024)


def reference(x, w, r, eps=EPS):
    s = x.double() + (0 if r is None else r.double())
    y = s / torch.sqrt(s.square().mean(-1, keepdim=True) + eps)
    return y if w is None else y * w.double()


def check_y(y, want, dtype):
    u, tiny = half_step(dtype), torch.finfo(dtype).smallest_normal * half_step(dtype)
    bound = (u + fp32(y.shape[1]) * (1 + u)) * want.abs() + tiny
    assert not bool(((y.double() - want).abs() > bound).any())


def check_q(q, scales, want, fmt):
    most, step, tiny = FP8[fmt]
    f = fp32(want.shape[1])
    top = want.abs().amax(-1)
    if torch.is_tensor(scales):
        assert scales.dtype == torch.float32
        assert bool(((scales.double() - top / most).abs() <= (f + 2 ** -23) * top / most).all())
        scales = scales.double()[:, None]
    value = q.double() * scales
    bound = (step + 2 * f + 2 ** -22) * want.abs() + tiny * scales
    clipped = want.abs() >= most * scales            # only with a given scale
    assert not bool((((value - want).abs() > bound) & ~clipped).any())
    assert bool((value.abs()[clipped] >= most * (scales + 0 * value)[clipped] * (1 - 2 * f
                                                                               - 2 ** -4)).all())


def make(g, T, H, dtype, residual=True, weight=True):
    def normal(scale, *shape):
        return (torch.randn(shape, generator=g, device=device()) * scale).to(dtype)
    return (normal(1.0, T, H), 1 + normal(0.2, H) if weight else None,
            normal(3.0, T, H) if residual else None)


SHAPES = [(1, 1), (1, 7), (3, 8), (2, 511), (1, 512), (300, 513), (5, 1024), (257, 1000),
          (400, 1537), (9, 2047), (600, 2048), (258, 2049), (1, 4096), (300, 4095), (270, 8191),
          (2, 8192), (1, 8193), (3, 16384), (259, 16385), (2, 32768), (3, 32769), (1, 50001),
          (2, 100000)]


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("dtype", TYPES)
def test_against_64_bits(T, H, dtype):
    note(f"norm T{T} H{H} {dtype}")
    g = gen(T + H)
    for residual, weight in ((True, True), (False, True), (True, False)):
        x, w, r = make(g, T, H, dtype, residual, weight)
        want = reference(x, w, r)
        got = rms_norm(x, w, EPS, residual=r)
        y = got[0] if residual else got
        check_y(y, want, dtype)
        if residual:
            assert torch.equal(bits(got[1]), bits((x.float() + r.float()).to(dtype)))
        for fmt in FP8:
            q, scales, *s = rms_norm_fp8(x, w, EPS, residual=r, dtype=fmt)
            assert q.dtype == fmt and q.shape == x.shape
            check_q(q, scales, want, fmt)
            assert len(s) == residual
            if residual:
                assert torch.equal(bits(s[0]), bits(got[1]))
            given, same, *_ = rms_norm_fp8(x, w, EPS, residual=r, dtype=fmt, scale=0.01)
            assert same == 0.01
            check_q(given, float(torch.tensor(0.01)), want, fmt)


@pytest.mark.parametrize("H", [300, 1111, 3000, 5001, 20001, 40001])
@pytest.mark.parametrize("dtype", TYPES)
def test_strides_and_what_lies_around(H, dtype):
    note(f"norm strides H{H} {dtype}")
    g, T = gen(H), 5
    x, w, r = make(g, T, H, dtype)
    want_y, want_s = rms_norm(x, w, EPS, residual=r)
    want_q, want_scales, _ = rms_norm_fp8(x, w, EPS, residual=r)
    views = []
    for t, pad in ((x, 3), (r, 8)):
        _, v = strided(T, H, H + pad, dtype)
        v.copy_(t)
        views.append(v)
    (yb, y), (sb, s) = strided(T, H, H + 5, dtype), strided(T, H, H + 1, dtype)
    got = rms_norm(views[0], w, EPS, residual=views[1], out=y, residual_out=s)
    assert got[0] is y and got[1] is s
    check_guard(yb, T, H, H + 5, dtype)
    check_guard(sb, T, H, H + 1, dtype)
    assert torch.equal(bits(y), bits(want_y)) and torch.equal(bits(s), bits(want_s))
    # bytes at an odd address, rows 3 bytes apart
    buf = torch.full((T * (H + 3) + 9,), 0x55, dtype=torch.uint8, device=device())
    q = buf[1:1 + T * (H + 3)].view(torch.float8_e4m3fn).view(T, H + 3)[:, :H]
    got = rms_norm_fp8(views[0], w, EPS, residual=views[1], out=q)
    assert torch.equal(q.contiguous().view(torch.uint8), want_q.view(torch.uint8))
    assert torch.equal(got[1], want_scales)
    assert int((buf != 0x55).sum()) <= T * H and bool((buf[:1] == 0x55).all())
    body = buf[1:1 + T * (H + 3)].view(T, H + 3)
    assert bool((body[:, H:] == 0x55).all()) and bool((buf[1 + T * (H + 3):] == 0x55).all())


@pytest.mark.parametrize("T,H", [(3, 500), (300, 4096), (2, 9000), (2, 40000)])
@pytest.mark.parametrize("dtype", TYPES)
def test_in_place(T, H, dtype):
    note(f"norm in place T{T} H{H} {dtype}")
    x, w, r = make(gen(H), T, H, dtype)
    want_y, want_s = rms_norm(x, w, EPS, residual=r)
    for y_in, s_in in ((None, 1), (0, 1), (1, 0), (0, None)):
        held = [x.clone(), r.clone()]
        y, s = rms_norm(held[0], w, EPS, residual=held[1],
                        out=None if y_in is None else held[y_in],
                        residual_out=None if s_in is None else held[s_in])
        assert torch.equal(bits(y), bits(want_y)) and torch.equal(bits(s), bits(want_s))
    q, scales, _ = rms_norm_fp8(x, w, EPS, residual=r)
    held = r.clone()
    got = rms_norm_fp8(x, w, EPS, residual=held, residual_out=held)
    assert torch.equal(got[0].view(torch.uint8), q.view(torch.uint8))
    assert torch.equal(got[1], scales) and torch.equal(bits(held), bits(want_s))


@pytest.mark.parametrize("H", [256, 2000, 5000, 20000, 40000])
@pytest.mark.parametrize("dtype", TYPES)
def test_zeros_infinities_nans_and_large_elements(H, dtype):
    note(f"norm edges H{H} {dtype}")
    x, w, _ = make(gen(H), 6, H, dtype)
    x[0] = 0
    x[1, H - 1] = math.inf
    x[2, H // 2] = math.nan
    x[3] *= 1e-4
    big = torch.finfo(dtype).max / 4
    x[4] = torch.where(x[4] > 0, big, -big).to(dtype)          # bf16: squares past fp32
    want = reference(x, w, None)
    y = rms_norm(x, w, EPS)
    ok = torch.tensor([0, 3, 4, 5], device=device())
    check_y(y[ok], want[ok], dtype)
    assert bool((y[0] == 0).all())
    assert bool(y[1, H - 1].isnan()) and bool((y[1, :H - 1] == 0).all())
    assert bool(y[2].isnan().all())
    for fmt in FP8:
        q, scales = rms_norm_fp8(x, w, EPS, dtype=fmt)
        check_q(q[ok[1:]], scales[ok[1:]], want[ok[1:]], fmt)
        assert float(scales[0]) == 0 and bool(scales[1:3].isnan().all())
        assert bool((q[:3].float() == 0).all())
        q, _ = rms_norm_fp8(x, w, EPS, dtype=fmt, scale=1e-3)
        assert bool(q[2].float().isnan().all()) and bool((q[0].float() == 0).all())
        assert float(q[5].float().abs().max()) == min(FP8[fmt][0], float(q[5].float().abs().max()))
    # a row whose scale has no reciprocal in fp32
    tiny = torch.full((1, H), 1.0, dtype=dtype, device=device())
    q, scales = rms_norm_fp8(tiny, (w * 0 + 1e-38).to(dtype), EPS)
    if dtype == torch.bfloat16:
        assert bool((q.float() == 448).all())
    assert bool(torch.isfinite(scales).all())


@pytest.mark.parametrize("dtype", TYPES)
def test_rows_none_and_eps(dtype):
    note(f"norm none {dtype}")
    x = torch.empty((0, 64), dtype=dtype, device=device())
    assert rms_norm(x).shape == (0, 64)
    q, scales, s = rms_norm_fp8(x, residual=x)
    assert q.shape == (0, 64) and scales.shape == (0,) and s.shape == (0, 64)
    x, w, r = make(gen(1), 4, 128, dtype)
    for eps in (0.0, 1e-3, 10.0):
        check_y(rms_norm(x, w, eps, residual=r)[0], reference(x, w, r, eps), dtype)


def test_replayed_and_on_another_stream():
    note("norm graph and stream")
    x, w, r = make(gen(2), 70, 3000, torch.bfloat16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q, scales, s = rms_norm_fp8(x, w, EPS, residual=r, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = rms_norm_fp8(x, w, EPS, residual=r)
        y = rms_norm(got[2], w, EPS)
    for k in range(3):
        graph.replay()
        torch.cuda.synchronize()
        eager = rms_norm_fp8(x, w, EPS, residual=r)
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8))
                   for a, b in zip(got, eager))
        assert torch.equal(bits(y), bits(rms_norm(eager[2], w, EPS)))
        if k == 0:
            assert torch.equal(q.view(torch.uint8), got[0].view(torch.uint8))
            assert torch.equal(scales, got[1]) and torch.equal(bits(s), bits(got[2]))
        x.mul_(-0.5)


@pytest.mark.parametrize("H", [1, 100, 1000, 4097, 9000, 40000])
@pytest.mark.parametrize("eps", [0.0, 2.0 ** -140, 2.0 ** -125, 2.0 ** -119, 2.0 ** -80])
def test_squares_below_the_range(H, eps):
    """bfloat16 rows whose squares vanish in fp32; powers of two are exact, so the tolerance is
    that of any row; what vanishes beside a mean and eps above 2^-120, 2^-30 of
    it, is far below its 32 * 2^-24."""
    note(f"norm tiny H{H} eps {eps}")
    x = torch.randn((5, H), generator=gen(H), device=device()).abs() + 0.5
    for k, e in enumerate((-132, -100, -70, -62, -55)):
        x[k] *= 2.0 ** e
    x = x.bfloat16()
    for rows in (x, x.repeat(60, 1)):
        want = reference(rows, None, None, eps)
        check_y(rms_norm(rows, None, eps), want, torch.bfloat16)
        q, scales = rms_norm_fp8(rows, None, eps)
        live = want.abs().amax(-1) > 2.0 ** -90      # scales in fp32's range
        check_q(q[live], scales[live], want[live], torch.float8_e4m3fn)
