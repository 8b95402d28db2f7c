"""CPU test: the kernel that a query names is the one that the call picks, also
where the bound of a sequence's rows is larger than the call's rows."""

from __future__ import annotations

import ctypes
import types

import pytest
import torch

import sm_b200 as K
from tests.test_paged_abi import paged


@pytest.mark.parametrize("bits,G,dtype", [(4, 4, torch.bfloat16), (8, 8, torch.bfloat16), (4, 1, torch.bfloat16),
                                          (4, 4, torch.float32)])
def test_name_follows_the_rows_of_the_call(bits, G, dtype):
    c = paged(bits=bits, D=128)
    cache = types.SimpleNamespace(_ref=ctypes.byref(c))
    code = K.KVQ_F32 if dtype == torch.float32 else K.KVQ_BF16
    size = {}
    for rows in (1, 3, 64):                     # every kernel wants a workspace of its own size
        size[K.paged_kernel_name(cache, dtype, rows, 2 * G)] = rows
    for T in (1, 3, 5, 64):
        for max_q in (1, 3, 64, 5000):
            name = K.paged_kernel_name(cache, dtype, max_q, 2 * G, T)
            assert name == K.paged_kernel_name(cache, dtype, min(max_q, T), 2 * G)
            # what the call itself picks shows in its workspace
            ws = [K.lib.kvq_paged_workspace_size(ctypes.byref(c), code, 1, T, m, 2 * G, 0) for m in (max_q, min(max_q, T))]
            assert ws[0] == ws[1] > 0
    assert len(size) == (1 if dtype == torch.float32 else 2)
    if dtype == torch.bfloat16 and G == 4:
        assert K.paged_kernel_name(cache, dtype, 64, 8, T=3) == "paged_rows"
        assert K.paged_kernel_name(cache, dtype, 64, 8, T=64) == "paged_chunk_tcgen05"
