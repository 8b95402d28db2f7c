"""GPU test of sequences that are cut back (rejected drafts): within a group the
tail slot serves as it is, over a group's end a copy of it made before does."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import sm_b200 as K
from tests.gpu_util import DEV
from tests.test_paged_gpu import Sequences, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits,group,D,dtype", [(4, 32, 128, torch.bfloat16), (8, 8, 80, torch.float32),
                                                (4, 64, 64, torch.bfloat16)])
@pytest.mark.parametrize("over", [False, True])
def test_rejected_drafts(bits, group, D, dtype, over):
    g = group
    start = 3 * g - 2 if over else 2 * g + 1             # four drafts end in the next group, or in this one
    s = Sequences(np.random.default_rng(g), [start + 12], 2, D, bits, g, 2 * g)
    s.append([start], dtype)
    for accepted in (1, 3, 2):
        before, rows = len(s.k[0]), s.cache.k_tail.clone()
        s.append([4], dtype)                             # drafts
        k, v = s.k[0][before:before + accepted], s.v[0][before:before + accepted]
        cut = before if over else before + accepted      # what of them may stay
        s.k[0], s.v[0] = s.k[0][:cut], s.v[0][:cut]
        if over:                                         # the slot of before, and the accepted ones again
            s.cache.k_tail.copy_(rows)
            s.append([accepted], dtype, raw=np.stack([k, v]))
        else:                                            # one more token where the next goes on
            s.append([1], dtype)
    n = len(s.k[0])
    got = K.paged_gather(s.cache, i32(s.table), i32([0]), i32([0, n]), n, n)
    for x, want in zip(got, s.decoded(0)):
        np.testing.assert_array_equal(x.cpu().numpy(), want.transpose(1, 0, 2))
    K.check(DEV)
