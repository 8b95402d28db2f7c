"""GPU tests of the append's and the read-back's kernel instances: every row width
and group that has one of its own, over rows that lie in a wider projection on
16-byte boundaries (what the vector forms take), in single tokens and in ragged
chunks; bytes and values equal to the reference's."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import sm_b200 as K
from tests import paged_ref as R
from tests.gpu_util import DEV, bf16_values, to_dev
from tests.test_paged_gpu import Sequences, i32

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def append_aligned(s, news, dtype, table, interleaved):
    """Append news[b] random tokens from K and V views of one projection's rows."""
    T, H, D = sum(news), s.H, s.D
    raw = s.rng.standard_normal((2, T, H, D)).astype(np.float32)
    raw = bf16_values(raw) if dtype == BF16 else raw
    buf = torch.full((T, 3 * H * D + 24), float("nan"), dtype=dtype, device=DEV)
    kd, vd = buf[:, 8:8 + H * D].unflatten(1, (H, D)), buf[:, 16 + H * D:16 + 2 * H * D].unflatten(1, (H, D))
    assert kd.data_ptr() % 16 == vd.data_ptr() % 16 == buf.stride(0) * buf.element_size() % 16 == 0
    kd.copy_(to_dev(raw[0], dtype))
    vd.copy_(to_dev(raw[1], dtype))
    cu = np.concatenate([[0], np.cumsum(news)])
    for b, n in enumerate(news):
        pos = np.arange(len(s.k[b]), len(s.k[b]) + n)
        s.k[b] = np.concatenate([s.k[b], R.rotate(raw[0][cu[b]:cu[b + 1]], table, pos, interleaved)])
        s.v[b] = np.concatenate([s.v[b], raw[1][cu[b]:cu[b + 1]]])
    K.paged_append(kd, vd, s.cache, i32(s.table), i32(s.lens()), i32(cu), max(news),
                   rope=None if table is None else to_dev(table), interleaved=interleaved, slots=i32(s.slots))


APPEND = [
    # bits, group, P, D, dtype, rot, interleaved
    (4, 8, 16, 40, BF16, 32, False), (8, 8, 8, 64, F32, 64, True), (4, 16, 32, 64, BF16, 64, False),
    (8, 16, 16, 64, F32, 32, True), (4, 32, 32, 64, BF16, 16, False), (8, 32, 64, 64, F32, 64, False),
    (4, 8, 24, 128, F32, 128, False), (8, 16, 32, 128, BF16, 0, False), (4, 32, 64, 128, BF16, 128, False),
    (8, 32, 96, 128, F32, 64, True), (8, 32, 64, 96, BF16, 96, False),
    (4, 8, 8, 256, BF16, 256, False), (8, 8, 24, 256, F32, 128, True), (4, 32, 64, 256, BF16, 256, False),
    (8, 32, 32, 256, F32, 64, True), (8, 8, 16, 200, BF16, 192, False),
    # the scalar form: larger groups, groups of 16 in wide rows
    (4, 64, 64, 64, BF16, 64, False), (8, 16, 16, 192, F32, 192, False), (4, 64, 128, 128, F32, 32, True),
]


@pytest.mark.parametrize("bits,group,P,D,dtype,rot,inter", APPEND)
def test_append_instances(bits, group, P, D, dtype, rot, inter):
    g = group
    calls = [[1, 1, 1, 1], [g, 2 * g + 3, 1, g - 1], [1, 1, 1, 1], [3 * g, 1, g + 1, 2], [1, 1, 1, 1],
             [g - 1, 2 * g - 1, 4 * g + 5, 1]]
    lens = [sum(c[b] for c in calls) for b in range(4)]
    s = Sequences(np.random.default_rng(D + g), lens, 3, D, bits, g, P)
    table = R.rope_table(max(lens), rot) if rot else None
    for news in calls:
        append_aligned(s, news, dtype, table, inter)
        s.check_bytes()
    K.check(DEV)


@pytest.mark.parametrize("bits,group,P,D", [(4, 4, 12, 20), (8, 4, 8, 20), (4, 12, 24, 36), (8, 12, 12, 60),
                                            (4, 24, 48, 48), (8, 8, 16, 24), (4, 2, 6, 10), (8, 16, 32, 256)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gather_instances(bits, group, P, D, dtype):
    lens = [1, 3 * P + 5, 0, group, 2 * P]
    s = Sequences(np.random.default_rng(D), lens, 2, D, bits, group, P)
    s.append(lens)
    starts, counts = [0, P - 1, 0, group - 1, 3], [1, 2 * P + 6, 0, 1, 2 * P - 3]
    cu = np.concatenate([[0], np.cumsum(counts)])
    k, v = K.paged_gather(s.cache, i32(s.table), i32(starts), i32(cu), int(cu[-1]), max(counts), dtype)
    for b, n in enumerate(counts):
        if n:
            for got, want in zip((k, v), s.decoded(b)):
                w = want[:, starts[b]:starts[b] + n].transpose(1, 0, 2)
                w = bf16_values(w) if dtype == BF16 else w
                np.testing.assert_array_equal(got[cu[b]:cu[b + 1]].float().cpu().numpy(), w)
    K.check(DEV)
