"""GPU check of host threads that share the 4-bit product's workspace on one
stream: every result has the bits of the same call made alone."""
from __future__ import annotations

import threading

import pytest
import torch

from dense_gemm_18_amd import W4Weight, binding, gemm_nt_w4
from tests import w4_ref
from tests.gpu_util import device, note
from tests.test_gpu_w4 import bits, gen

pytestmark = pytest.mark.gpu


def test_threads_share_a_workspace():
    note("w4 threads")
    M, N, K, group = 400, 520, 640, 64
    g = gen(6)
    ws = torch.empty(binding.gemm_nt_w4_ws_size(M, N, K), dtype=torch.uint8, device=device())
    A = torch.randn((M, K), generator=g, device=device(), dtype=torch.float16)
    ws_each = [W4Weight(*w4_ref.random_weight(g, N, K, group, True, torch.float16),
                        shape=(N, K), group=group) for _ in range(3)]
    want = [gemm_nt_w4(A, w, workspace=ws) for w in ws_each]
    torch.cuda.synchronize()
    got, start = [[] for _ in ws_each], threading.Barrier(len(ws_each))

    def work(i):
        start.wait()
        for _ in range(50):
            got[i].append(gemm_nt_w4(A, ws_each[i], workspace=ws))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(ws_each))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for w, calls in zip(want, got):
        assert len(calls) == 50
        for D in calls:
            assert torch.equal(bits(D), bits(w))
