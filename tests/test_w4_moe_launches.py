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
