"""GPU check that a group's scale sees every one of its elements: one element
stands out, in each place of the group and with either sign in turn."""
from __future__ import annotations

import pytest
import torch

from dense_gemm_18_amd import quantize_w4
from tests import w4_ref
from tests.gpu_util import device, note
from tests.w4_ref import TYPES

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
def test_every_element_counts_for_the_scale(group, zeros, dtype):
    note(f"quantize extremes group {group} zeros {zeros} {dtype}")
    K = 256
    g = torch.Generator().manual_seed(group)
    W = (torch.rand((2 * K, K), generator=g) * 0.02 - 0.01).to(dtype)
    at = torch.arange(K)
    W[at, at] = (1 + torch.rand(K, generator=g)).to(dtype)
    W[K + at, at] = -(1 + torch.rand(K, generator=g)).to(dtype)
    q, s, z = w4_ref.quantize(W, group, zeros)
    w = quantize_w4(W.to(device()), group=group, zeros=zeros)
    torch.cuda.synchronize()
    assert torch.equal(w.scales.cpu(), s)
    assert torch.equal(w4_ref.unpack(w.q.cpu(), K), q)
    if zeros:
        assert torch.equal(w.zeros.cpu().to(torch.int64), z)
