"""CPU checks of the FP8 product with row scales: refusals before any HIP call."""
from __future__ import annotations

import pytest

from dense_gemm_18_amd import binding

OK, BAD = binding.GEMM_OK, binding.GEMM_EINVAL
# host-side integers used as addresses; never dereferenced
A, B, D, SA, SB = (0x10000000 * i for i in range(1, 6))


def call(**kw):
    a = dict(A=A, B=B, D=D, M=4, N=64, K=256, scale=1.0, a_scale=SA, b_scale=SB, a_format=0,
             b_format=1, dtype=binding.GEMM_T_BF16)
    a.update(kw)
    return binding.gemm_nt_fp8_rs(**a)


@pytest.mark.parametrize("kw", [
    dict(M=-1), dict(N=-1), dict(K=-1), dict(M=2 ** 31), dict(N=2 ** 31),
    dict(K=binding.GEMM_MAX_K + 1), dict(a_format=2), dict(b_format=-1), dict(dtype=2),
    dict(dtype=-1), dict(A=0), dict(B=0), dict(D=0), dict(D=D + 1), dict(a_scale=SA + 2),
    dict(b_scale=SB + 1), dict(D=A), dict(D=B + 2), dict(D=SA + 12), dict(D=SB + 252),
    dict(a_scale=D + 508)])
def test_refused_before_any_hip_call(kw):
    assert call(**kw) == BAD


def test_nothing_is_a_no_op():
    assert call(M=0, A=0, D=0, a_scale=0) == OK
    assert call(N=0, B=0, D=0, b_scale=0) == OK
