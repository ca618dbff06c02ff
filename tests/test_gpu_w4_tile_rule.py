"""GPU check of few rows of the 4-bit product on both sides of the rule that
chooses between its resident and its chunked 16 x 64 tile: the number of tiles,
of groups and the bytes of LDS.  Tolerances: those of the product's own tests."""
from __future__ import annotations

import pytest
import torch

from tests import w4_ref
from tests.gpu_util import device, note
from tests.test_gpu_w4 import check, gen, product
from tests.w4_ref import TYPES

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K", [(1, 16321, 130), (1, 16384, 2000), (1, 16385, 2048),
                                   (2, 16400, 2049), (1, 17000, 4096), (3, 17000, 4097),
                                   (1, 16500, 8192), (1, 16500, 8200), (4, 16450, 8190),
                                   (16, 16390, 2047), (16, 33000, 100)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", TYPES)
def test_both_sides_of_the_rule(M, N, K, group, dtype):
    note(f"w4 tile rule {M}x{N}x{K} group {group} {dtype}")
    g = gen(M + N + K + group)
    A = torch.randn((M, K), generator=g, device=device(), dtype=dtype)
    Q, S, Z = w4_ref.random_weight(g, N, K, group, True, dtype)
    check(product(A, Q, S, Z, group), A, Q, S, Z, group)
