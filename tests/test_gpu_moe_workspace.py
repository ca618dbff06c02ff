"""GPU checks of workspaces that several layers, streams or host threads share.
Tolerances: those of the layer's own tests.
"""
from __future__ import annotations

import threading

import pytest
import torch

from dense_gemm_18_amd import MoeLayer, binding
from tests.gpu_util import device, note
from tests.test_gpu_moe import Case
from tests.test_gpu_w4 import bits
from tests.w4_ref import TYPES

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("group", [0, 64])
def test_one_workspace_for_layers_of_other_sizes(group, dtype):
    # every order of short and long hidden sizes, the small one's plan first
    note(f"moe one workspace, group {group} {dtype}")
    cases = [Case(H + E, E, topk, H, 48, dtype, group) for H, E, topk in
             ((64, 8, 2), (4096, 16, 4), (256, 70, 8), (1024, 4, 1), (8192, 8, 2))]
    need = max(binding.moe_nt_ws_size(64, c.layer._weights, c.topk) for c in cases)
    ws = torch.zeros(need, dtype=torch.uint8, device=device())
    stream = torch.cuda.current_stream().cuda_stream
    for T in (1, 5, 33, 2):
        for i in (0, 1, 0, 4, 2, 1, 3, 4, 0, 1, 2, 3):
            c = cases[i]
            X = c.tokens(T)
            y = torch.full_like(X, float("nan"))
            ids = torch.empty((T, c.topk), dtype=torch.int32, device=device())
            weights = torch.empty((T, c.topk), dtype=torch.float32, device=device())
            rc = binding.moe_nt_layer(c.layer._weights, X.data_ptr(), y.data_ptr(),
                                      ids.data_ptr(), weights.data_ptr(), T, c.H, c.H, c.topk,
                                      binding.MOE_RENORMALIZE, ws.data_ptr(), need, stream)
            assert rc == binding.GEMM_OK
            c.check_route(X, ids, weights)
            c.check_y(X, ids, weights, y)


@pytest.mark.parametrize("group", [0, 64])
def test_threads_call_one_layer_on_one_stream(group):
    note(f"moe threads, group {group}")
    c = Case(11, 16, 4, 512, 256, torch.bfloat16, group)
    Xs = [c.tokens(T) for T in (1, 3, 20, 130)]
    ids = [c.layer.route(X) for X in Xs]
    want = [c.layer(X) for X in Xs]
    half = [c.layer.experts(X, *r) for X, r in zip(Xs, ids)]
    torch.cuda.synchronize()
    fresh = MoeLayer(c.router, c.layer.w13, c.layer.w2, topk=4)    # has no workspace yet
    got, errors = [[] for _ in Xs], []
    start = threading.Barrier(len(Xs))

    def work(i):
        try:
            start.wait()
            for _ in range(50):
                got[i].append((*fresh(Xs[i]), fresh.experts(Xs[i], *ids[i])))
        except Exception as e:                                  # shown by the main thread
            errors.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(Xs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for i, calls in enumerate(got):
        for y, chosen, weights, z in calls:
            assert torch.equal(bits(y), bits(want[i][0])) and torch.equal(chosen, want[i][1])
            assert torch.equal(weights, want[i][2]) and torch.equal(bits(z), bits(half[i]))
