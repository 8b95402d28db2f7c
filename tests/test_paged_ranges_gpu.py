"""GPU tests of paged attention over values of very different sizes: what lies
behind a row's position, groups of zeros among small values, keys and values
far apart.

Tolerance, per output: with p a row's float64 weights over the decoded values v,
A = sum_t p_t |v_t|.  Rounding V and the weights to 11 bits moves an output by at
most 2^-11 A each.  K's roundings move a score by at most 1.4e-3 (five deviations
of a sum of 64 or 128 products, each off by 2^-11 / sqrt(3) of itself, whose root
sum of squares is about 1 for these inputs), and an error e of the scores moves
an output by at most e sum_t p_t |v_t - o| <= 2 e A: 2.8e-3 A.  Together below
2^-8 A.  A weight times a value far below the row's largest may be lost: at most
2^-31 of the largest a key, below 2^-22 for 512 keys.  The output's own rounding
is 2^-8 of it for bf16."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import sm_b200 as K
from tests.gpu_util import DEV, bf16_values, to_dev
from tests.test_paged_gpu import Sequences, i32

pytestmark = pytest.mark.gpu


def rows64(q, k, v, scale, first):
    """q [n, H_q, D]: rows at positions first ..; k, v [H, len, D] decoded.
    Outputs and sum_t p |v| in float64, causal."""
    n, H_q, D = q.shape
    H = k.shape[0]
    G = H_q // H
    out, size = np.zeros((n, H_q, D)), np.zeros((n, H_q, D))
    for h in range(H):
        kk, vv = k[h].astype(np.float64), v[h].astype(np.float64)
        for i in range(n):
            lim = first + i + 1
            s = q[i, h * G:(h + 1) * G].astype(np.float64) @ kk[:lim].T * scale
            p = np.exp(s - s.max(-1, keepdims=True))
            p /= p.sum(-1, keepdims=True)
            out[i, h * G:(h + 1) * G] = p @ vv[:lim]
            size[i, h * G:(h + 1) * G] = p @ np.abs(vv[:lim])
    return out, size


def check(s, q, G, dtype, splits=0, scale=None, b=0):
    """The last rows of the one sequence against float64."""
    n, D = q.shape[0], s.D
    scale = scale or 1.0 / np.sqrt(D)
    if dtype == torch.bfloat16:
        q = bf16_values(q)
    length = len(s.k[b])
    got = K.paged_attend(to_dev(q, dtype), s.cache, i32(s.table), i32([length]), i32([0, n]), n, scale, splits=splits)
    K.check(DEV)
    kd, vd = s.decoded(b)
    want, size = rows64(q, kd, vd, scale, length - n)
    err = np.abs(got.double().cpu().numpy() - want)
    tol = 2.0 ** -8 * (size + (np.abs(want) if dtype == torch.bfloat16 else 0)) + 2.0 ** -22 * size.max(-1, keepdims=True)
    bad = ~(err <= tol)
    assert not bad.any(), f"{bad.sum()} of {bad.size} outputs off, first at {np.argwhere(bad)[0]}: " \
                          f"{err[bad][0]:.3e} > {tol[bad][0]:.3e}"


# rows of four heads a KV head: the kernels of few and of many
SHAPES = [(4, 128, 1, torch.bfloat16), (8, 64, 2, torch.bfloat16), (4, 128, 100, torch.bfloat16),
          (8, 128, 100, torch.bfloat16), (8, 128, 1, torch.bfloat16), (4, 64, 100, torch.bfloat16),
          (8, 64, 24, torch.bfloat16), (8, 64, 100, torch.float32),
          (4, 80, 9, torch.bfloat16), (8, 80, 5, torch.float32)]


@pytest.mark.parametrize("bits,D,n,dtype", SHAPES)
@pytest.mark.parametrize("splits", [0, 1, 7])
def test_large_values_behind_a_row(bits, D, n, dtype, splits):
    """One key's channel and one value row 2^40 times larger than the others:
    rows before them are what they are without, rows after see them."""
    rng = np.random.default_rng(41)
    s = Sequences(rng, [300], 1, D, bits, 32, 64)
    raw = rng.standard_normal((2, 300, 1, D)).astype(np.float32)
    raw[0, 270, 0, 3] = 2.0 ** 40
    raw[1, 285] *= 2.0 ** 40
    s.append([300], raw=raw)
    check(s, rng.standard_normal((n, 4, D)).astype(np.float32), 4, dtype, splits)


@pytest.mark.parametrize("bits,D,n,dtype", SHAPES)
@pytest.mark.parametrize("small", [2.0 ** -30, 2.0 ** -60])
def test_groups_of_zeros_among_small_values(bits, D, n, dtype, small):
    """A group of zeros has the scale 1, whatever the size of the others."""
    rng = np.random.default_rng(42)
    s = Sequences(rng, [200], 1, D, bits, 32, 32)
    raw = rng.standard_normal((2, 200, 1, D)).astype(np.float32) * np.float32(small)
    raw[1, 37] = 0.0
    raw[1, 150, :, :32] = 0.0
    raw[0, 64:96, :, 5] = 0.0
    raw[0, 160:192] = 0.0
    s.append([200], raw=raw)
    check(s, rng.standard_normal((n, 4, D)).astype(np.float32) / np.float32(small), 4, dtype)


@pytest.mark.parametrize("bits,D,n,dtype", SHAPES)
@pytest.mark.parametrize("splits", [0, 5])
def test_values_far_apart(bits, D, n, dtype, splits):
    """Key channels up to 2^24 apart, with queries the other way round, and
    value rows up to 2^60 apart: the largest reach the output, whichever they are."""
    rng = np.random.default_rng(43)
    s = Sequences(rng, [400], 1, D, bits, 32, 64)
    raw = rng.standard_normal((2, 400, 1, D)).astype(np.float32)
    a = 2.0 ** rng.integers(-12, 13, D)
    raw[0] *= a.astype(np.float32)
    raw[1] *= (2.0 ** rng.integers(-30, 31, 400)).astype(np.float32)[:, None, None]
    raw[1, :200] *= 2.0 ** -20                       # later keys of a row move its reference
    s.append([400], raw=raw)
    check(s, rng.standard_normal((n, 4, D)).astype(np.float32) / a.astype(np.float32), 4, dtype, splits)


@pytest.mark.parametrize("bits,D,n,dtype", SHAPES)
def test_large_value_of_no_weight(bits, D, n, dtype):
    """A value 2^60 times the others, of a key whose weight is 2^-100: the row is
    the others'."""
    rng = np.random.default_rng(44)
    s = Sequences(rng, [260], 1, D, bits, 32, 64)
    raw = rng.standard_normal((2, 260, 1, D)).astype(np.float32)
    raw[0] *= 0.1
    raw[0, 50] = -70.0 / np.sqrt(D)
    raw[1, 50] *= 2.0 ** 60
    s.append([260], raw=raw)
    q = 1.0 + 0.1 * rng.standard_normal((n, 4, D)).astype(np.float32)
    check(s, q, 4, dtype, splits=3)


def test_empty_rows_and_two_sequences_of_other_sizes():
    """A batch in which one sequence is ordinary and another is not, and a third
    has no rows."""
    rng = np.random.default_rng(45)
    lens, news, D = [500, 300, 90], [60, 80, 0], 128
    s = Sequences(rng, lens, 2, D, 4, 32, 64)
    raw = rng.standard_normal((2, sum(lens), 2, D)).astype(np.float32)
    raw[1, 500:800] *= (2.0 ** rng.integers(-30, 31, 300)).astype(np.float32)[:, None, None]
    s.append(lens, raw=raw)
    q = bf16_values(rng.standard_normal((140, 8, D)).astype(np.float32))
    for splits in (0, 1, 9):
        got = K.paged_attend(to_dev(q, torch.bfloat16), s.cache, i32(s.table), i32(lens), i32([0, 60, 140, 140]), 80,
                             D ** -0.5, splits=splits).double().cpu().numpy()
        for b, (r0, r1) in enumerate(((0, 60), (60, 140))):
            kd, vd = s.decoded(b)
            want, size = rows64(q[r0:r1], kd, vd, D ** -0.5, lens[b] - news[b])
            err = np.abs(got[r0:r1] - want)
            assert (err <= 2.0 ** -8 * (size + np.abs(want)) + 2.0 ** -22 * size.max(-1, keepdims=True)).all(), (b, splits)
    K.check(DEV)


@pytest.mark.parametrize("bits,D,n,dtype", SHAPES + [(4, 128, 3, torch.bfloat16)])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("wide", [False, True])
def test_value_scale_that_is_not_finite(bits, D, n, dtype, bad, wide):
    """It is the scale of one token's 32 features: rows that see the token are not
    finite there and as ever elsewhere, rows before it as ever."""
    rng = np.random.default_rng(47)
    s = Sequences(rng, [300], 1, D, bits, 32, 64)
    raw = rng.standard_normal((2, 300, 1, D)).astype(np.float32)
    if wide:
        raw[1, :40] *= 2.0 ** 30
    s.append([300], raw=raw)
    q = bf16_values(rng.standard_normal((n, 4, D)).astype(np.float32))
    at, hit = 300 - (n + 1) // 2, slice(32, min(D, 64))       # the token, its features

    def run(splits):
        return K.paged_attend(to_dev(q, dtype), s.cache, i32(s.table), i32([300]), i32([0, n]), n, D ** -0.5,
                              splits=splits).float()

    vs = s.cache.v_scales.view(s.cache.pages, 1, 64, -1)
    page, row = int(s.table[0, at // 64]), at % 64
    was = vs[page, 0, row, 1].clone()
    for splits in (0, 1, 6):
        want = run(splits)
        vs[page, 0, row, 1] = bad
        got = run(splits)
        vs[page, 0, row, 1] = was
        sees = n - (300 - at)                                 # the first row that does
        assert torch.equal(got[:sees], want[:sees])
        assert not torch.isfinite(got[sees:, :, hit]).any()
        got[sees:, :, hit] = want[sees:, :, hit]
        assert torch.equal(got, want)
    K.check(DEV)


@pytest.mark.parametrize("bits,D,n,dtype", SHAPES)
@pytest.mark.parametrize("size", [2.0 ** k for k in (8, 12, 14, 16, 18, 20, 30, 60)])
def test_scores_of_any_size(bits, D, n, dtype, size):
    """Scores up to 2^69: keys of whole numbers in groups of scale 1 and queries
    of powers of two, so that equal scores are equal in any precision and others
    far apart.  A row is the mean of its best keys' values."""
    rng = np.random.default_rng(46)
    top = 7 if bits == 4 else 127
    s = Sequences(rng, [200], 1, D, bits, 32, 32)
    raw = np.zeros((2, 200, 1, D), np.float32)
    raw[0, :, 0, 0] = rng.integers(-top + 1, top, 200)
    raw[0, 5::32, 0, 0] = -top                           # in every group, and no key but one at the other end
    raw[0, 77, 0, 0] = top
    raw[0, :, 0, 1] = top                                # the same for all keys
    raw[1] = rng.standard_normal((200, 1, D))
    s.append([200], raw=raw)
    q = np.zeros((n, 4, D), np.float32)
    q[..., 0] = size * rng.choice([-1.0, 1.0], (n, 4))
    q[..., 1] = size * rng.choice([-1.0, 1.0], (n, 4))
    check(s, q, 4, dtype, scale=1.0)


@pytest.mark.parametrize("bits,D,n,dtype", SHAPES)
@pytest.mark.parametrize("bad", [float("inf"), float("nan"), 2.0 ** 100])
@pytest.mark.parametrize("splits", [0, 1, 10])
def test_key_scale_behind_a_row(bits, D, n, dtype, bad, splits):
    """A key channel's scale in the last group, whatever it is: rows before the
    group are as ever."""
    rng = np.random.default_rng(48)
    s = Sequences(rng, [300], 1, D, bits, 32, 32)
    s.append([300])
    q = bf16_values(rng.standard_normal((n, 4, D)).astype(np.float32))
    s.cache.k_scales.view(s.cache.pages, 1, 1, D)[int(s.table[0, 288 // 32]), 0, 0, 5] = bad
    got = K.paged_attend(to_dev(q, dtype), s.cache, i32(s.table), i32([300]), i32([0, n]), n, D ** -0.5,
                         splits=splits).double().cpu().numpy()
    K.check(DEV)
    kd, vd = s.decoded(0)
    before = max(0, n - 12)                                   # rows at positions below 288
    want, size = rows64(q[:before], kd, vd, D ** -0.5, 300 - n)
    err = np.abs(got[:before] - want)
    assert (err <= 2.0 ** -8 * (size + np.abs(want)) + 2.0 ** -22 * size.max(-1, keepdims=True, initial=0)).all()
    if np.isnan(bad):
        assert np.isnan(got[before:]).all()
