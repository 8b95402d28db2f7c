"""GPU test of the paged calls back to back on one stream: each call's kernels
are let in while the call before drains, and buffers are written again and again
with other values, so a read that comes too early or from a stale line shows."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import sm_b200 as K
from tests import paged_ref as R
from tests.gpu_util import DEV, to_dev
from tests.test_paged_gpu import Sequences, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,bits,n", [(torch.bfloat16, 4, 64), (torch.bfloat16, 8, 150), (torch.bfloat16, 4, 1),
                                          (torch.float32, 8, 20)])
def test_steps_without_a_synchronisation(dtype, bits, n):
    """Prepare, append, attend and read back over the same buffers, 12 steps in a
    row, against the same steps with a synchronisation after every call."""
    H, G, D, P, S, steps = 2, 4, 128, 32, 3, 12
    rng = np.random.default_rng(n)
    td = to_dev(R.rope_table(n * steps, D))
    w = to_dev(1 + 0.1 * rng.standard_normal(D), dtype)
    x = [to_dev(rng.standard_normal((S * n, (G + 2) * H * D)) * 2.0 ** (i % 3), dtype) for i in range(steps)]
    cu = i32(np.arange(S + 1) * n)

    def run(wait):
        s = Sequences(np.random.default_rng(5), [n * steps] * S, H, D, bits, 32, P)
        table = i32(s.table)
        buf, lens, pos = torch.empty_like(x[0]), i32([0] * S), i32(np.zeros(S * n))
        q0 = torch.empty(S * n, G * H, D, dtype=dtype, device=DEV)
        k0 = torch.empty(S * n, H, D, dtype=dtype, device=DEV)
        o = torch.empty_like(q0)
        got = []

        def step(f, *a, **kw):
            r = f(*a, **kw)
            if wait:
                torch.cuda.synchronize()
            return r

        for i in range(steps):
            step(buf.copy_, x[i])
            step(lens.fill_, (i + 1) * n)
            step(pos.copy_, torch.arange(i * n, (i + 1) * n, device=DEV, dtype=torch.int32).repeat(S))
            q, k = buf[:, :G * H * D].unflatten(1, (G * H, D)), buf[:, G * H * D:(G + 1) * H * D].unflatten(1, (H, D))
            v = buf[:, (G + 1) * H * D:].unflatten(1, (H, D))
            step(K.qk_norm_rope, q, k, pos, td, w, w, q_out=q0, k_out=k0)
            step(K.paged_append, k0, v, s.cache, table, lens, cu, n)
            step(K.paged_attend, q0, s.cache, table, lens, cu, n, D ** -0.5, out=o)
            got.append(o.clone())
            kv = step(K.paged_gather, s.cache, table, i32([i * n] * S), cu, S * n, n)
            got.extend(kv)
        torch.cuda.synchronize()
        return got, [t.clone() for t in (s.cache.k_codes, s.cache.v_codes, s.cache.k_tail)]

    want, bytes_want = run(True)
    for _ in range(3):
        got, bytes_got = run(False)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(torch.equal(a, b) for a, b in zip(bytes_got[:2], bytes_want[:2]))
    K.check(DEV)
