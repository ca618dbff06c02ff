"""GPU check of the example: quantise, 4-bit product and mixture of experts
together, eagerly and as a replayed graph.

Tolerance on its relative error: a block rounds about ten times at no more
than a half step u in the 2-norm (product, sum, two norms of two roundings,
h, y, sum), with u of the expert's inputs passing through gate, up and down:
16 u for each block, and blocks add up.
"""
from __future__ import annotations

import pytest

from examples import decode_w4_moe
from tests.gpu_util import note

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens", [1, 5])
@pytest.mark.parametrize("f16", [False, True])
def test_decode_example(tokens, f16):
    note(f"decode example tokens {tokens} f16 {f16}")
    args = ["--tokens", str(tokens), "--layers", "2", "--hidden", "384", "--inner", "192",
            "--experts", "6", "--topk", "2", "--steps", "3"] + ["--f16"] * f16
    error, same = decode_w4_moe.main(args)
    assert error <= 2 * 16 * (2.0 ** -11 if f16 else 2.0 ** -8)
    assert same
