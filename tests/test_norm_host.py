"""CPU checks of the norm: refusals before any HIP call."""
from __future__ import annotations

import pytest
import torch

from dense_gemm_18_amd import binding, rms_norm, rms_norm_fp8

OK, BAD = binding.GEMM_OK, binding.GEMM_EINVAL
# host-side integers used as addresses; never dereferenced
X, R, W, Y, S, C = (0x10000000 * i for i in range(1, 7))
F16, E4M3 = binding.GEMM_T_F16, binding.GEMM_FP8_E4M3


def wide(**kw):
    a = dict(X=X, R=R, W=W, Y=Y, S=S, T=4, H=100, ldx=100, ldr=100, ldy=100, lds=100, eps=1e-6,
             dtype=F16)
    a.update(kw)
    return binding.rms_norm(**a)


def fp8(**kw):
    a = dict(X=X, R=R, W=W, Q=Y, scales=C, S=S, T=4, H=100, ldx=100, ldr=100, ldq=100, lds=100,
             eps=1e-6, scale=0.0, format=E4M3, dtype=F16)
    a.update({"Q" if k == "Y" else "ldq" if k == "ldy" else k: v for k, v in kw.items()})
    return binding.rms_norm_fp8(**a)


SHARED = [dict(T=-1), dict(T=2 ** 31), dict(H=0), dict(H=-1),
          dict(H=binding.GEMM_MAX_K + 1, ldx=2 ** 30, ldr=2 ** 30, ldy=2 ** 30, lds=2 ** 30),
          dict(ldx=99), dict(ldr=99), dict(ldy=99), dict(lds=99), dict(ldx=2 ** 41),
          dict(ldy=2 ** 41), dict(ldr=2 ** 41), dict(lds=2 ** 41), dict(dtype=2), dict(dtype=-1),
          dict(eps=-1e-9), dict(eps=float("inf")), dict(eps=float("nan")), dict(X=0), dict(Y=0),
          dict(X=X + 1), dict(R=R + 1), dict(W=W + 1), dict(S=S + 1), dict(R=0),
          dict(Y=X + 2), dict(Y=W + 2), dict(Y=S), dict(S=W), dict(S=X + 798), dict(S=R - 798),
          dict(S=X, lds=101), dict(S=R, ldr=101)]


@pytest.mark.parametrize("kw", SHARED + [dict(Y=Y + 1), dict(Y=X, ldy=101)])
def test_norm_refuses_before_any_hip_call(kw):
    assert wide(**kw) == BAD


@pytest.mark.parametrize("kw", SHARED + [dict(format=2), dict(format=-1), dict(Y=X), dict(Y=R),
                                         dict(scales=C + 2), dict(scales=X), dict(scales=S + 4),
                                         dict(scales=Y), dict(scales=0), dict(scales=W),
                                         dict(scales=0, scale=-1.0),
                                         dict(scales=0, scale=float("inf")),
                                         dict(scales=0, scale=float("nan"))])
def test_norm_into_8_bits_refuses_before_any_hip_call(kw):
    assert fp8(**kw) == BAD


def test_no_rows_are_a_no_op():
    assert wide(T=0, X=0, R=0, W=0, Y=0, S=0) == OK
    assert fp8(T=0, X=0, R=0, W=0, Y=0, S=0, scales=0) == OK


def test_python_refuses():
    x = torch.zeros((4, 8), dtype=torch.float16)
    with pytest.raises(ValueError):
        rms_norm(x)                                     # not on a GPU
    with pytest.raises(ValueError):
        rms_norm(x[0])
    with pytest.raises(ValueError):
        rms_norm(x[:, :0])
    with pytest.raises(TypeError):
        rms_norm(x.float())
    with pytest.raises(TypeError):
        rms_norm_fp8(x, dtype=torch.float16)
