"""CPU check that the whole layer refuses every output that overlaps an input
of either half, before any HIP call."""
from __future__ import annotations

import pytest

from tests.test_w4_moe_host import BAD, layer, weights

W = dict(router=0x100000000, w13=0x200000000, w13_scales=0x300000000, w13_zeros=0x600000000,
         w2=0x400000000, w2_scales=0x500000000, w2_zeros=0x700000000)


@pytest.mark.parametrize("out", ["d", "ids", "wts", "ws"])
@pytest.mark.parametrize("part", sorted(W))
def test_layer_refuses_outputs_inside_the_model(out, part):
    assert layer(w=weights(**W), **{out: W[part]}) == BAD
    # 16-bit experts have no scales or zero points
    if part in ("router", "w13", "w2"):
        plain = weights(router=W["router"], w13=W["w13"], w2=W["w2"], w13_scales=0, w2_scales=0,
                        group=0)
        assert layer(w=plain, **{out: W[part]}) == BAD
