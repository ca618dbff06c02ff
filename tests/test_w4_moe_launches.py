"""CPU checks of what the mixture of experts and the 4-bit product launch, and
with which parts of the workspace: the launches are recorded, none runs."""
from __future__ import annotations

import pytest

from tests import launch_recorder

LAYOUTS = """
result = []
WS = 0x5000000000
for hidden in (64, 256, 1024, 4096, 8192, 65536, binding.GEMM_MAX_K):
    for T in (1, 5, 64):
        w = weights(hidden=hidden, inner=64, group=GROUP, s13=0x3300000000, s2=0x4400000000)
        need = binding.moe_nt_ws_size(T, w, 2)
        before = count.value
        rc = binding.moe_nt_layer(w, 0x8000000000, 0x9000000000, 0xa000000000, 0xb000000000, T,
                                  hidden, hidden, 2, 0, WS, need)
        assert rc == binding.GEMM_OK
        inside = sorted({v - WS for x in launches()[before:] for v in x["arg"][:18]
                         if WS <= v < WS + need})
        result.append({"hidden": hidden, "T": T, "inside": inside})
"""


@pytest.mark.parametrize("group", [0, 64])
def test_counters_lie_apart_from_what_calls_of_other_sizes_write(tmp_path, group):
    """The workspace's first part counts workgroups: one word for the router and one
    for each 32 hidden rows, zero between calls.  Whatever sizes a call has, what else
    it keeps there lies behind the words of the largest one."""
    most = 4 * (1 + -(-4194303 // 32))
    for x in launch_recorder.run(tmp_path, LAYOUTS.replace("GROUP", str(group))):
        assert x["inside"][0] == 0, x
        assert x["inside"][1] >= most, x


THREADS = """
pause_us.value = 1000
WS = 0x5000000000
w = weights()
need = binding.moe_nt_ws_size(64, w, 2)

def call(kind, T, at):
    x, y = 0x8000000000 + at, 0x9000000000 + at
    ids, wts = 0xa000000000 + at, 0xb000000000 + at
    if kind == "layer":
        return binding.moe_nt_layer(w, x, y, ids, wts, T, 256, 256, 2, 0, WS, need)
    return binding.moe_nt_experts(w, x, ids, wts, y, T, 256, 256, 2, WS, need)

calls = [("layer", 5), ("experts", 9), ("layer", 130), ("layer", 1)]
alone = []
for kind, T in calls:
    before = count.value
    assert call(kind, T, 0) == binding.GEMM_OK
    alone.append(count.value - before)
before = count.value
start = threading.Barrier(len(calls))

def work(i):
    start.wait()
    for _ in range(4):
        assert call(*calls[i], (i + 1) << 28) == binding.GEMM_OK

threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
for t in threads:
    t.start()
for t in threads:
    t.join()
# which call's X a launch has; a chunk's lies a little further on
result = [alone, [(x["arg"][0] - 0x8000000000 >> 28) - 1 for x in launches()[before:]]]
"""


def test_threads_that_share_a_workspace_enqueue_whole_calls(tmp_path):
    """The launches of one call hand each other a plan, logits and products in the
    workspace, so none of another call's may come between them on the stream."""
    alone, order = launch_recorder.run(tmp_path, THREADS)
    assert sorted(set(order)) == [0, 1, 2, 3] and len(order) == 4 * sum(alone)
    while order:
        n = alone[order[0]]
        assert order[:n] == [order[0]] * n, order
        order = order[n:]


PRODUCTS = """
pause_us.value = 1000
M, N, K = 700, 512, 1024
need = binding.gemm_nt_w4_ws_size(M, N, K)
assert need > 0

def call(at):
    return binding.gemm_nt_w4(0x1000000000 + at, 0x2000000000 + at, 0x3000000000 + at, 0,
                              0x4000000000 + at, M, N, K, K, N, 128, 0, 0x5000000000, need)

assert call(0) == binding.GEMM_OK
alone = count.value
start = threading.Barrier(3)

def work(i):
    start.wait()
    for _ in range(4):
        assert call(i << 28) == binding.GEMM_OK

threads = [threading.Thread(target=work, args=(i,)) for i in range(3)]
for t in threads:
    t.start()
for t in threads:
    t.join()
result = [alone, [x["thread"] for x in launches()[alone:]]]
"""


def test_threads_that_share_a_workspace_unpack_and_multiply_together(tmp_path):
    alone, order = launch_recorder.run(tmp_path, PRODUCTS)
    assert alone == 2 and len(order) == 3 * 4 * 2 and len(set(order)) == 3
    for i in range(0, len(order), 2):
        assert order[i] == order[i + 1], order
