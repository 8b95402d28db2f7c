"""GPU test of a call whose list of blocks passes 2^30 entries."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import sm_b200 as K
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu


def test_block_list_past_two_to_the_thirty():
    """32772 rows of eight heads over a million keys (f32 rows: an item is one
    token's eight rows, 2^15 blocks each), every row reading all keys: the last
    rows are those that a call of their own gives."""
    D, P, n_keys, T, last = 64, 1024, 1 << 20, (1 << 15) + 4, 6
    pages = 16                                          # the sequence's pages name these in turn
    g = torch.Generator(device=DEV).manual_seed(7)
    cache = K.PagedCache(pages, 1, P, D, 4, 32, 1, DEV)
    cache.k_codes.copy_(torch.randint(0, 256, cache.k_codes.shape, generator=g, device=DEV, dtype=torch.uint8) % 0xEF)
    cache.v_codes.copy_(torch.randint(0, 256, cache.v_codes.shape, generator=g, device=DEV, dtype=torch.uint8) % 0xEF)
    cache.k_scales.uniform_(0.05, 0.2, generator=g)
    cache.v_scales.uniform_(0.05, 0.2, generator=g)
    table = (torch.arange(n_keys // P, device=DEV, dtype=torch.int32) % pages)[None].contiguous()
    q = torch.randn(T, 8, D, generator=g, device=DEV)

    def run(rows):
        x = q[-rows:].contiguous()
        i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)
        return K.paged_attend(x, cache, table, i32([n_keys]), i32([0, rows]), rows, D ** -0.5, causal=False)

    got = run(T)[-last:]
    want = run(last)
    K.check(DEV)
    # two orders of float32 sums over the same products: both within 2e-4 max|V| of float64
    top = 8 * 0.2
    assert float(want.abs().max()) > 0
    assert float((got - want).abs().max()) <= 2 * 2e-4 * top
