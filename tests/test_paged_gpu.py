"""GPU tests of the paged cache: append, gather, attention, q/k preparation.

Packed bytes, scales, tails and gathered values must equal the reference's
exactly.  Attention rows: a float32 output within 2e-4 * max|V| of float64 (a
score is a sum of 128 products of which the absolute values add up to about 10
in log2 units for these inputs, so its float32 error is below 128 * 2^-24 * 10
= 8e-5, and an error d of every score moves an output by at most 2 d max|V|
ln 2); a bf16 output through its rounding interval at the library's 2e-3 *
max|V| (gpu_util).  Where the tensor-core kernel of many rows runs, Q,
K, V and the softmax's p are fp16 tiles, each rounded once (at most 2^-11 of the
value; Q is exact): V moves an output by at most 2^-11 max|V|, p by as much (a
weighted mean of the errors), and K through the scores: a score is a sum of 64
or 128 products whose independent roundings have a deviation below 2^-11 /
sqrt(3) * sqrt(sum (q k scale)^2), and for these inputs that root is about 1:
2.8e-4, five deviations 1.4e-3; an error e of the scores moves an output by at
most e max|V| / 2 for each of the keys that share the weight, p (1 - p) <= 1/4
and values differing by at most 2 max|V|: 2^-10 max|V|.  Together 2^-9 max|V|;
and over all outputs the output's own rounding has a relative deviation of at
most 2^-8 / sqrt(3) = 2.3e-3 and the three others 2.8e-4 each, 2.4e-3 together:
3e-3 is asked of the whole."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle as O
import sm_b200 as K
from tests import paged_ref as R
from tests.gpu_util import DEV, bf16_values, check_rows_rounded, to_dev

pytestmark = pytest.mark.gpu

F32_TOL = 2e-4
TILE_TOL = 2.0 ** -9
TILE_REL = 3e-3


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def poisoned(pages, H, P, D, bits, group, slots):
    """A cache whose every byte is bad: codes 0xFF, scales and tails NaN."""
    c = K.PagedCache(pages, H, P, D, bits, group, slots, DEV)
    c.k_codes.fill_(255)
    c.v_codes.fill_(255)
    for t in (c.k_scales, c.v_scales, c.k_tail):
        t.fill_(float("nan"))
    return c


class Sequences:
    """Sequences in random pages of a poisoned pool, and what they hold."""

    def __init__(self, rng, lens, H, D, bits, group, P, spare=2, slots=None, width=None):
        S = len(lens)
        self.rng, self.H, self.D, self.bits, self.group, self.P = rng, H, D, bits, group, P
        used = [-(-max(n, 1) // P) for n in lens]
        self.cols = width or max(used) + 1
        total = sum(used) + spare
        order = rng.permutation(total)
        self.table = np.full((S, self.cols), -1, np.int32)
        at = 0
        for b, n in enumerate(used):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.free = order[at:]
        self.slots = rng.permutation(S).astype(np.int32) if slots is None else np.asarray(slots, np.int32)
        self.cache = poisoned(total, H, P, D, bits, group, S)
        self.k = [np.zeros((0, H, D), np.float32) for _ in lens]     # rotated rows
        self.v = [np.zeros((0, H, D), np.float32) for _ in lens]

    def append(self, news, dtype=torch.float32, table=None, interleaved=False, fused=False, extra=0, max_new=None,
               raw=None):
        """Append news[b] random tokens to each sequence (`extra` rows past the
        last sequence's) and keep the reference rows."""
        T, H, D = sum(news) + extra, self.H, self.D
        if raw is None:
            raw = self.rng.standard_normal((2, T, H, D)).astype(np.float32)
        if dtype == torch.bfloat16:
            raw = bf16_values(raw)
        if fused:                                   # rows of a wider projection
            buf = torch.full((T, 3 * H * D + 5), float("nan"), dtype=dtype, device=DEV)
            kd, vd = buf[:, 1:1 + H * D].unflatten(1, (H, D)), buf[:, 2 + H * D:2 + 2 * H * D].unflatten(1, (H, D))
            kd.copy_(to_dev(raw[0], dtype))
            vd.copy_(to_dev(raw[1], dtype))
        else:
            kd, vd = to_dev(raw[0], dtype), to_dev(raw[1], dtype)
        cu = np.concatenate([[0], np.cumsum(news)])
        for b, n in enumerate(news):
            pos = np.arange(len(self.k[b]), len(self.k[b]) + n)
            new = R.rotate(raw[0][cu[b]:cu[b + 1]], table, pos, interleaved)
            self.k[b] = np.concatenate([self.k[b], new])
            self.v[b] = np.concatenate([self.v[b], raw[1][cu[b]:cu[b + 1]]])
        K.paged_append(kd, vd, self.cache, i32(self.table), i32(self.lens()), i32(cu), max_new or max(max(news), 1),
                       rope=None if table is None else to_dev(table), interleaved=interleaved, slots=i32(self.slots))

    def lens(self):
        return [len(x) for x in self.k]

    def packed(self, b, h):
        return (O.pack_k(self.k[b][:, h], self.bits, self.group), O.pack_v(self.v[b][:, h], self.bits, self.group))

    def decoded(self, b):
        return R.decoded_heads(self.k[b].transpose(1, 0, 2), self.v[b].transpose(1, 0, 2), self.bits, self.group)

    def check_bytes(self):
        """Every page byte: the sequences' as a whole-cache pack of their
        tokens, the others as they were."""
        c, g, P, D, H = self.cache, self.group, self.P, self.D, self.H
        Dp = -(-D // g) * g
        kc = np.full((c.pages, H, P * D * self.bits // 8), 255, np.uint8)
        vc = np.full((c.pages, H, P, Dp * self.bits // 8), 255, np.uint8)
        ks = np.full((c.pages, H, P // g, D), np.nan, np.float32)
        vs = np.full((c.pages, H, P, Dp // g), np.nan, np.float32)
        for b, n in enumerate(self.lens()):
            for h in range(H if n else 0):
                pk, pv = self.packed(b, h)
                kcodes = pk.codes.reshape(-1, g * D * self.bits // 8)          # a K group's bytes
                vcodes = pv.codes.reshape(n, -1)
                for j in range(-(-n // g)):
                    page, at = self.table[b, j * g // P], j * g % P // g
                    w = g * D * self.bits // 8
                    kc[page, h, at * w:(at + 1) * w] = kcodes[j]
                    ks[page, h, at] = pk.scales[j]
                for t in range(n):
                    vc[self.table[b, t // P], h, t % P] = vcodes[t]
                    vs[self.table[b, t // P], h, t % P] = pv.scales[t]
        for got, want, name in ((c.k_codes, kc, "k_codes"), (c.v_codes, vc, "v_codes"),
                                (c.k_scales, ks, "k_scales"), (c.v_scales, vs, "v_scales")):
            np.testing.assert_array_equal(got.cpu().numpy().reshape(want.shape), want, name)
        tail = c.k_tail.cpu().numpy()
        for b, n in enumerate(self.lens()):
            r = n % g
            if r:
                np.testing.assert_array_equal(tail[self.slots[b], :, :r], self.k[b][n - r:].transpose(1, 0, 2))


@pytest.mark.parametrize("bits,group,P,D,dtype,rot,inter,fused", [
    (4, 32, 64, 128, torch.bfloat16, 128, False, False),
    (4, 32, 32, 128, torch.float32, 64, True, True),
    (8, 32, 96, 64, torch.bfloat16, 64, False, True),
    (8, 8, 16, 80, torch.float32, 40, True, False),
    (4, 8, 8, 72, torch.bfloat16, 0, False, True),
    (4, 8, 24, 13, torch.float32, 6, False, False),
    (8, 2, 6, 5, torch.bfloat16, 4, True, False),
    (4, 32, 64, 40, torch.float32, 40, False, True),
    (4, 64, 64, 256, torch.bfloat16, 256, False, False),
])
def test_append_bytes_over_ragged_calls(bits, group, P, D, dtype, rot, inter, fused):
    rng = np.random.default_rng(bits * 1000 + group * 10 + D)
    g = group
    # per call, the new tokens of four sequences: whole prompts, single steps,
    # drafts that begin and end inside groups (one, two or more groups apart)
    calls = [[1, 0, 2 * g + 3, g], [1, g, 1, 1], [g - 1, 0, 1, 2 * g], [1, 2 * g - 1, g + 1, 3], [g, 1, 2 * g, 1],
             [1, 1, 1, 1], [3 * g + 1, 2, g - 1, 2 * g + 1]]
    lens = [sum(c[b] for c in calls) for b in range(4)]
    s = Sequences(rng, lens, 3, D, bits, g, P)
    table = R.rope_table(max(lens), rot) if rot else None
    for i, news in enumerate(calls):
        s.append(news, dtype, table, inter, fused, extra=i % 2)
        s.check_bytes()
    K.check(DEV)


def test_append_equals_pack_of_the_rotated_rows():
    """One sequence over one page per call == kvq_pack of the same rows."""
    rng = np.random.default_rng(5)
    n, H, D, g = 77, 2, 128, 32
    s = Sequences(rng, [n], H, D, 4, g, 96)
    for m in (1, 30, 3, 40, 3):
        s.append([m])
    whole = K.PackedCache(1, H, 96, D, 4, g, DEV)
    K.pack(to_dev(s.k[0].transpose(1, 0, 2)[None]), to_dev(s.v[0].transpose(1, 0, 2)[None]), whole)
    page = int(s.table[0, 0])
    for h in range(H):
        groups = -(-n // g)
        a = s.cache.k_codes.view(s.cache.pages, H, -1)[page, h, :groups * g * D // 2]
        assert torch.equal(a, whole.head_k_codes(0, h)[:groups * g * D // 2])
        b = s.cache.v_codes.view(s.cache.pages, H, -1)[page, h, :n * D // 2]
        assert torch.equal(b, whole.head_v_codes(0, h)[:n * D // 2])
    K.check(DEV)


def test_append_special_values():
    """Zero groups (scale 1), signed zeros, ties, the largest and the smallest
    floats: the same bytes as the oracle's pack."""
    rng = np.random.default_rng(6)
    s = Sequences(rng, [70], 1, 32, 4, 32, 32)
    raw = np.zeros((2, 70, 1, 32), np.float32)
    raw[:, :20] = rng.integers(-7, 8, (2, 20, 1, 32)) * 0.5
    raw[:, 3] = 3.5
    raw[:, 20:40] = -0.0
    raw[:, 40:60] = rng.standard_normal((2, 20, 1, 32)) * 1e-38
    raw[:, 60:70] = rng.standard_normal((2, 10, 1, 32)) * 1e37
    s.append([70], raw=raw)
    s.check_bytes()
    K.check(DEV)


@pytest.mark.parametrize("bits,group,P,D,dtype", [(4, 32, 32, 128, torch.float32), (8, 8, 40, 80, torch.bfloat16),
                                                  (4, 8, 8, 13, torch.float32), (8, 32, 64, 64, torch.float32)])
def test_gather_values(bits, group, P, D, dtype):
    rng = np.random.default_rng(D)
    lens = [1, 3 * P + 5, 0, group, 2 * P]
    s = Sequences(rng, lens, 2, D, bits, group, P)
    s.append(lens)
    starts, counts = [0, P - 1, 0, group - 1, 3], [1, 2 * P + 6, 0, 1, 2 * P - 3]
    cu = np.concatenate([[0], np.cumsum(counts)])
    k, v = K.paged_gather(s.cache, i32(s.table), i32(starts), i32(cu), int(cu[-1]), max(counts), dtype)
    for b, n in enumerate(counts):
        if not n:
            continue
        kd, vd = s.decoded(b)
        for got, want in ((k, kd), (v, vd)):
            w = want[:, starts[b]:starts[b] + n].transpose(1, 0, 2)
            if dtype == torch.bfloat16:
                w = bf16_values(w)
            np.testing.assert_array_equal(got[cu[b]:cu[b + 1]].float().cpu().numpy(), w)
    K.check(DEV)


def run_attend(s, news, G, dtype, causal, extra=0, splits=0, max_q=None, scale=None, q=None):
    """Attend the last news[b] positions; returns (out, list of reference rows)."""
    H, D = s.H, s.D
    T = sum(news) + extra
    scale = scale if scale is not None else 1.0 / np.sqrt(D)
    if q is None:
        q = s.rng.standard_normal((T, H * G, D)).astype(np.float32)
    if dtype == torch.bfloat16:
        q = bf16_values(q)
    cu = np.concatenate([[0], np.cumsum(news)])
    out = torch.full((T, H * G, D), 77.0, dtype=dtype, device=DEV)
    K.paged_attend(to_dev(q, dtype), s.cache, i32(s.table), i32(s.lens()), i32(cu), max_q or max(max(news), 1), scale,
                   causal=causal, out=out, splits=splits)
    out.tiles = K.paged_kernel_name(s.cache, dtype, max_q or max(max(news), 1), H * G) == "paged_chunk_tcgen05"
    want = []
    for b, n in enumerate(news):
        if n:
            kd, vd = s.decoded(b)
            want.append((R.attend_rows(q[cu[b]:cu[b + 1]], kd, vd, len(s.k[b]), scale, causal), vd))
        else:
            want.append(None)
    return out, want, cu


def check_attend(out, want, cu, dtype, what="", tiles=None):
    o = out.float().cpu().numpy()
    tiles = out.tiles if tiles is None else tiles
    off = size = 0.0
    for b, w in enumerate(want):
        if w is None:
            continue
        rows, vd = w
        got = o[cu[b]:cu[b + 1]]
        H = vd.shape[0]
        G = rows.shape[1] // H
        for h in range(H):
            a, r = got[:, h * G:(h + 1) * G], rows[:, h * G:(h + 1) * G]
            top = float(np.abs(vd[h]).max())
            if dtype == torch.bfloat16:
                check_rows_rounded(a, r, (TILE_TOL if tiles else 2e-3) * top, f"{what} b={b} h={h}")
                off, size = off + float(np.square(a - r).sum()), size + float(np.square(r).sum())
            else:
                assert np.isfinite(a).all(), f"{what} b={b} h={h}"
                err = np.abs(a - r).max()
                assert err <= F32_TOL * top, f"{what} b={b} h={h}: {err:.3e} > {F32_TOL * top:.3e}"
    assert not tiles or off <= TILE_REL ** 2 * size, f"{what}: {(off / size) ** 0.5:.2e} of the outputs' norm"
    assert (o[cu[-1]:] == 77.0).all(), f"{what}: rows behind the last sequence"


LENS = [1, 31, 32, 33, 0, 127, 128, 129, 500]

ATTEND = [
    # bits, group, P, D, H, G, dtype
    (4, 32, 32, 128, 2, 4, torch.bfloat16),
    (8, 32, 64, 128, 1, 8, torch.bfloat16),
    (4, 32, 96, 64, 2, 3, torch.float32),
    (8, 32, 32, 64, 2, 1, torch.bfloat16),
    (4, 32, 256, 128, 1, 4, torch.float32),
    (8, 32, 128, 128, 2, 2, torch.float32),
    (4, 32, 160, 128, 1, 7, torch.bfloat16),
    (4, 32, 32, 128, 1, 16, torch.bfloat16),
    (8, 32, 64, 64, 1, 20, torch.float32),
    (4, 8, 16, 128, 2, 4, torch.bfloat16),
    (8, 8, 24, 80, 1, 5, torch.float32),
    (4, 64, 64, 256, 1, 2, torch.bfloat16),
    (4, 32, 64, 256, 1, 4, torch.float32),
    (4, 32, 64, 32, 2, 4, torch.bfloat16),
    (4, 2, 6, 13, 1, 1, torch.float32),
    (8, 16, 48, 96, 3, 2, torch.bfloat16),
]


@pytest.mark.parametrize("bits,group,P,D,H,G,dtype", ATTEND)
@pytest.mark.parametrize("splits", [0, 1, 7])
def test_attend_one_row_a_sequence(bits, group, P, D, H, G, dtype, splits):
    rng = np.random.default_rng(D + G)
    s = Sequences(rng, LENS, H, D, bits, group, P)
    s.append(LENS)
    news = [1 if n else 0 for n in LENS]
    out, want, cu = run_attend(s, news, G, dtype, True, extra=2, splits=splits)
    check_attend(out, want, cu, dtype)
    K.check(DEV)


@pytest.mark.parametrize("bits,group,P,D,H,G,dtype", ATTEND)
@pytest.mark.parametrize("causal", [True, False])
def test_attend_ragged_rows(bits, group, P, D, H, G, dtype, causal):
    """Whole prompts, one row, a few and many, in one batch."""
    rng = np.random.default_rng(D + G + 1)
    s = Sequences(rng, LENS, H, D, bits, group, P)
    s.append(LENS)
    news = [1, 31, 2, 9, 0, 127, 1, 40, 65]
    out, want, cu = run_attend(s, news, G, dtype, causal, extra=1)
    check_attend(out, want, cu, dtype)
    K.check(DEV)


@pytest.mark.parametrize("bits,D,G,dtype", [(4, 128, 4, torch.bfloat16), (8, 128, 4, torch.bfloat16),
                                            (4, 64, 8, torch.bfloat16), (4, 128, 4, torch.float32),
                                            (8, 64, 2, torch.float32)])
@pytest.mark.parametrize("n", [1, 3, 8, 33, 200])
def test_attend_split_and_whole(bits, D, G, dtype, n):
    """A few long sequences: many workers to one (sequence, head), several
    items to one sequence, and one worker for everything."""
    rng = np.random.default_rng(n)
    lens = [1500, 700]
    s = Sequences(rng, lens, 2, D, bits, 32, 64)
    s.append(lens)
    q = rng.standard_normal((2 * n, 2 * G, D)).astype(np.float32)
    for splits in (0, 1, 2, 1000):
        out, want, cu = run_attend(s, [n, n], G, dtype, True, splits=splits, q=q)
        check_attend(out, want, cu, dtype, f"splits {splits}")
    K.check(DEV)


def test_attend_ignores_what_is_past_a_row():
    """Keys behind a row's position may hold anything: other values there
    leave a causal row's bits as they were."""
    rng = np.random.default_rng(9)
    for D, n, dtype in ((128, 5, torch.bfloat16), (128, 100, torch.bfloat16), (64, 4, torch.float32)):
        s = Sequences(rng, [300], 1, D, 4, 32, 64)
        s.append([300])
        q = rng.standard_normal((n, 4, D)).astype(np.float32)
        a, _, _ = run_attend(s, [n], 4, dtype, True, q=q)
        t = 300 - 1                                     # the last token: seen by the last row only
        page, at = int(s.table[0, t // 64]), t % 64
        s.cache.v_scales.view(s.cache.pages, 1, 64, -1)[page, 0, at] = float("inf")
        b, _, _ = run_attend(s, [n], 4, dtype, True, q=q)
        assert torch.equal(a[:n - 1], b[:n - 1])
        assert not torch.isfinite(b[n - 1].float()).all()
    K.check(DEV)


def test_attend_nan_query_gives_nan_rows():
    """A row whose query is not a number is not one either, split or not, and
    the other rows are as they were."""
    rng = np.random.default_rng(14)
    for D, n, dtype in ((128, 1, torch.bfloat16), (128, 50, torch.bfloat16), (64, 2, torch.float32),
                        (80, 3, torch.float32)):
        s = Sequences(rng, [600], 1, D, 4, 32 if D != 80 else 8, 64)
        s.append([600])
        q = rng.standard_normal((n, 2, D)).astype(np.float32)
        for splits in (1, 0):
            good, _, _ = run_attend(s, [n], 2, dtype, True, q=q, splits=splits)
            bad_q = q.copy()
            bad_q[n - 1, 1, 5] = np.nan
            out, _, _ = run_attend(s, [n], 2, dtype, True, q=bad_q, splits=splits)
            assert torch.isnan(out[n - 1, 1].float()).all(), (D, n, splits)
            out[n - 1, 1] = good[n - 1, 1]
            assert torch.equal(out, good), (D, n, splits)
    K.check(DEV)


def test_attend_extreme_scores():
    """Scores hundreds apart, in both orders, and a negative scale: the
    running maximum moves at every block, or never."""
    rng = np.random.default_rng(10)
    for order in (1, -1):
        for dtype in (torch.bfloat16, torch.float32):
            for n in (1, 40):
                s = Sequences(rng, [400], 1, 128, 8, 32, 64)
                raw = rng.standard_normal((2, 400, 1, 128)).astype(np.float32)
                raw[0] = 0.02 * raw[0] + (np.linspace(0, 3, 400)[::order] * 1.0)[:, None, None]
                s.append([400], raw=raw)
                q = np.ones((n, 2, 128), np.float32)
                for scale in (1.0, -1.0):
                    out, want, cu = run_attend(s, [n], 2, dtype, True, scale=scale, q=q)
                    # scores of about 400 (their absolute products add up to as much): a float32 error of up to
                    # 128 * 2^-24 * 400 * 1.44 = 4e-3 in the exponent's log2 for a running sum, and for the tensor
                    # cores' tiles K rounded to fp16 (2^-11 of 400 at most, averaged over 128 features: 0.2 / 11);
                    # one key dominates, neighbours differ by 1: an error e of a score moves the output by e max|V|
                    top = float(np.abs(want[0][1]).max())
                    err = np.abs(out.float().cpu().numpy() - want[0][0]).max()
                    assert err <= (0.05 if dtype == torch.bfloat16 else 8e-3) * top, (order, dtype, n, scale, err)
    K.check(DEV)


def test_attend_device_errors():
    rng = np.random.default_rng(11)
    for G, n in ((4, 1), (4, 40)):
        s = Sequences(rng, [100, 70], 1, 128, 4, 32, 64)
        s.append([100, 70])
        q = rng.standard_normal((2 * n, G, 128)).astype(np.float32)
        good, want, cu = run_attend(s, [n, n], G, torch.bfloat16, True, q=q)
        qd = to_dev(q, torch.bfloat16)

        def call(table=s.table, lens=(100, 70), c=cu, max_q=n):
            out = torch.full((2 * n, G, 128), 77.0, dtype=torch.bfloat16, device=DEV)
            K.paged_attend(qd, s.cache, i32(table), i32(lens), i32(c), max_q, 1 / np.sqrt(128), out=out)
            return out

        def name(**kw):
            out = call(**kw)
            with pytest.raises(K.KVQError) as e:
                K.check(DEV)
            return out, e.value.name

        for page in (-1, s.cache.pages, 2 ** 31 - 1, -2 ** 31):
            bad = s.table.copy()
            bad[0, 1] = page
            out, err = name(table=bad)
            assert err == "KVQ_ERR_INDEX"
            assert torch.equal(out[n:], good[n:])            # the other sequence is as it was
        out, err = name(lens=(0, 70))
        assert err == "KVQ_ERR_LENGTH" and (out[:n] == 0).all() and torch.equal(out[n:], good[n:])
        out, err = name(lens=(-5, 70))
        assert err == "KVQ_ERR_LENGTH" and (out[:n] == 0).all()
        out, err = name(c=[0, 3 * n, 2 * n])                  # not increasing, past T
        assert err == "KVQ_ERR_LENGTH"
        if n > 1:
            out, err = name(lens=(n - 1, 70))                 # fewer keys than rows: row 0 sees none
            assert err == "KVQ_ERR_LENGTH" and (out[0] == 0).all() and torch.isfinite(out.float()).all()
            out, err = name(max_q=n - 1)
            assert err == "KVQ_ERR_LENGTH"
        assert torch.equal(call(), good)
        K.check(DEV)


def test_append_device_errors():
    rng = np.random.default_rng(12)
    s = Sequences(rng, [40, 40], 1, 64, 4, 32, 32)
    k, v = to_dev(rng.standard_normal((10, 1, 64))), to_dev(rng.standard_normal((10, 1, 64)))

    def name(table=s.table, lens=(5, 5), cu=(0, 5, 10), mx=5, slots=(0, 1), rope=None):
        before = [t.clone() for t in (s.cache.k_codes, s.cache.v_codes)]
        K.paged_append(k, v, s.cache, i32(table), i32(lens), i32(cu), mx, slots=i32(slots), rope=rope)
        with pytest.raises(K.KVQError) as e:
            K.check(DEV)
        return e.value.name, before

    for page in (-1, s.cache.pages, 2 ** 31 - 1):
        bad = s.table.copy()
        bad[:, 0] = page
        err, before = name(table=bad)
        assert err == "KVQ_ERR_INDEX"
        assert torch.equal(before[0], s.cache.k_codes) and torch.equal(before[1], s.cache.v_codes)
    for kw in (dict(slots=(-1, 2)), dict(slots=(7, 1 << 30))):
        err, before = name(**kw)
        assert err == "KVQ_ERR_INDEX" and torch.equal(before[0], s.cache.k_codes)
    for kw in (dict(lens=(4, 3)), dict(lens=(-1, 0)), dict(lens=(10 ** 6, 2 ** 31 - 1))):
        err, before = name(**kw)
        assert err == "KVQ_ERR_LENGTH" and torch.equal(before[0], s.cache.k_codes)
    assert name(cu=(0, 50, 10))[0] == "KVQ_ERR_LENGTH"
    assert name(mx=2)[0] == "KVQ_ERR_LENGTH"
    assert name(rope=to_dev(R.rope_table(3, 64)))[0] == "KVQ_ERR_INDEX"
    K.check(DEV)


def test_gather_device_errors():
    rng = np.random.default_rng(13)
    s = Sequences(rng, [40], 1, 64, 4, 32, 32, width=2)
    s.append([40])
    for kw, want in ((dict(start=-1), "KVQ_ERR_LENGTH"), (dict(start=60), "KVQ_ERR_LENGTH"),
                     (dict(cu=(0, 40)), "KVQ_ERR_LENGTH"), (dict(page=99), "KVQ_ERR_INDEX")):
        table = s.table.copy()
        table[0, 0] = kw.get("page", table[0, 0])
        K.paged_gather(s.cache, i32(table), i32([kw.get("start", 0)]), i32(kw.get("cu", (0, 8))), 8, 8)
        with pytest.raises(K.KVQError) as e:
            K.check(DEV)
        assert e.value.name == want
    K.check(DEV)


QK = [
    # T, H_q, H_kv, D, dtype, rot, interleaved, norm, fused
    (1, 1, 1, 128, torch.bfloat16, 128, False, True, False),
    (7, 32, 8, 128, torch.bfloat16, 128, False, True, True),
    (600, 32, 8, 128, torch.bfloat16, 128, False, True, True),
    (33, 8, 2, 64, torch.bfloat16, 64, True, True, True),
    (5, 4, 4, 256, torch.float32, 128, False, True, False),
    (9, 4, 1, 128, torch.float32, 64, True, False, True),
    (4, 3, 1, 80, torch.bfloat16, 80, False, True, True),
    (4, 3, 1, 96, torch.float32, 24, True, True, False),
    (3, 2, 0, 13, torch.float32, 6, False, True, False),
    (6, 2, 1, 8, torch.bfloat16, 0, False, True, True),
    (3, 5, 2, 1000, torch.bfloat16, 500, False, True, False),
    (2, 1, 1, 2, torch.float32, 2, True, False, False),
    (3000, 12, 3, 64, torch.float32, 32, False, True, True),
    (20, 7, 1, 16, torch.bfloat16, 16, False, False, False),
]


@pytest.mark.parametrize("T,H_q,H_kv,D,dtype,rot,inter,norm,fused", QK)
def test_qk_norm_rope(T, H_q, H_kv, D, dtype, rot, inter, norm, fused):
    rng = np.random.default_rng(T + D)
    n_pos, eps = 5000, 1e-5
    wide = (H_q + H_kv) * D + (11 if fused else 0)
    x = 2.0 * rng.standard_normal((T, wide)).astype(np.float32)
    x = bf16_values(x) if dtype == torch.bfloat16 else x
    w = [(1 + 0.3 * rng.standard_normal(D)).astype(np.float32) for _ in range(2)]
    w = [bf16_values(a) if dtype == torch.bfloat16 else a for a in w] if norm else [None, None]
    pos = rng.integers(0, n_pos, T)
    table = R.rope_table(n_pos, rot) if rot else None
    xd = to_dev(x, dtype)
    q = xd[:, :H_q * D].unflatten(1, (H_q, D))
    k = xd[:, H_q * D:(H_q + H_kv) * D].unflatten(1, (H_kv, D)) if H_kv else None
    if not fused:
        q, k = q.contiguous(), k.contiguous() if H_kv else None
    td = None if table is None else to_dev(table)
    wd = [None if a is None else to_dev(a, dtype) for a in w]
    got = K.qk_norm_rope(q, k, i32(pos), td, wd[0], wd[1], eps, inter)
    K.check(DEV)
    for o, lo, heads, ww in ((got[0], 0, H_q, w[0]), (got[1], H_q * D, H_kv, w[1])):
        if not heads:
            assert o is None
            continue
        xin = x[:, lo:lo + heads * D].reshape(T, heads, D)
        want = R.norm_rope(xin, ww, eps, table, pos, inter)
        # float32: the mean of D squares, the root (2 ulp), three products and a sum, each within 2^-24 or so of
        # the operands, whose size is that of the pair (c, s <= 1): below (D / 32 + 16) * 2^-24 of the larger one
        # (a warp's sum adds D / 32 terms a lane, then 5); the output's rounding is half a step more
        a, b = R.pair_index(rot, inter) if rot else (np.zeros(0, int), np.zeros(0, int))
        size = np.abs(want)
        if rot:
            pair = np.hypot(want[..., a], want[..., b])
            size[..., a], size[..., b] = pair, pair
        tol = size * (D / 32 + 16) * 2.0 ** -24 + np.abs(want) * (2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24) + 1e-30
        err = np.abs(o.double().cpu().numpy() - want)
        assert (err <= tol).all(), float((err - tol).max())
    # in place, where the input is dense
    if not fused:
        K.qk_norm_rope(q, k, i32(pos), td, wd[0], wd[1], eps, inter, q_out=q, k_out=k)
        assert torch.equal(q, got[0]) and (k is None or torch.equal(k, got[1]))
    K.check(DEV)


def test_qk_position_error_leaves_the_row_unturned():
    x = torch.randn(3, 2, 64, device=DEV)
    t = to_dev(R.rope_table(10, 64))
    out, _ = K.qk_norm_rope(x, None, i32([1, 10, -1]), t)
    with pytest.raises(K.KVQError) as e:
        K.check(DEV)
    assert e.value.name == "KVQ_ERR_INDEX"
    assert torch.equal(out[1:], x[1:]) and not torch.equal(out[0], x[0])


@pytest.mark.parametrize("dtype,D,G,bits,P", [(torch.bfloat16, 128, 4, 4, 64), (torch.bfloat16, 64, 8, 8, 32),
                                              (torch.float32, 128, 2, 8, 96), (torch.bfloat16, 80, 2, 4, 32)])
def test_serving_steps(dtype, D, G, bits, P):
    """Prompts, chunks, drafts and single tokens: q/k norms and rotation, the
    append and the attention of each step, against the reference's own."""
    rng = np.random.default_rng(D + bits)
    H, S, eps = 2, 3, 1e-6
    steps = [[40, 1, 0], [1, 90, 5], [1, 1, 1], [4, 30, 1], [1, 1, 70], [33, 1, 1]]
    total = [sum(st[b] for st in steps) for b in range(S)]
    s = Sequences(rng, total, H, D, bits, 32, P)
    table = R.rope_table(max(total), D)
    td = to_dev(table)
    w = [bf16_values((1 + 0.1 * rng.standard_normal(D)).astype(np.float32)) for _ in range(2)]
    wd = [to_dev(a, dtype) for a in w]
    for news in steps:
        T = sum(news)
        x = 1.3 * rng.standard_normal((T, (G + 2) * H * D)).astype(np.float32)
        xd = to_dev(x, dtype)
        hq = H * G
        q = xd[:, :hq * D].unflatten(1, (hq, D))
        k = xd[:, hq * D:(hq + H) * D].unflatten(1, (H, D))
        v = xd[:, (hq + H) * D:].unflatten(1, (H, D))
        cu = np.concatenate([[0], np.cumsum(news)])
        before = s.lens()
        pos = np.concatenate([np.arange(before[b], before[b] + n) for b, n in enumerate(news)]).astype(np.int64)
        qn, kn = K.qk_norm_rope(q, k, i32(pos), td, wd[0], wd[1], eps)
        lens = [before[b] + n for b, n in enumerate(news)]
        K.paged_append(kn, v, s.cache, i32(s.table), i32(lens), i32(cu), max(news), slots=i32(s.slots))
        out = K.paged_attend(qn, s.cache, i32(s.table), i32(lens), i32(cu), max(news), 1 / np.sqrt(D))
        K.check(DEV)
        kv, vv, qv = (t.float().cpu().numpy() for t in (kn, v, qn))
        want = []
        for b, n in enumerate(news):
            s.k[b] = np.concatenate([s.k[b], kv[cu[b]:cu[b + 1]]])
            s.v[b] = np.concatenate([s.v[b], vv[cu[b]:cu[b + 1]]])
            if n:
                kd, vd = s.decoded(b)
                want.append((R.attend_rows(qv[cu[b]:cu[b + 1]], kd, vd, lens[b], 1 / np.sqrt(D), True), vd))
            else:
                want.append(None)
        s.check_bytes()
        check_attend(out, want, cu, dtype, str(news),
                     K.paged_kernel_name(s.cache, dtype, max(news), hq) == "paged_chunk_tcgen05")


def test_captured_step_replays_on_new_inputs():
    """A decode step captured once, replayed with other rows, lengths and
    pages in the same buffers, and two graphs sharing one workspace in turn."""
    rng = np.random.default_rng(21)
    H, G, D, P, S = 2, 4, 128, 64, 5
    total = [200, 64, 1, 33, 150]
    s = Sequences(rng, [n + 4 for n in total], H, D, 4, 32, P)
    s.append(total)
    table = R.rope_table(400, D)
    td = to_dev(table)
    tab, lens, cu, slots = i32(s.table), i32(total), i32(range(S + 1)), i32(s.slots)
    q = torch.zeros(S, H * G, D, dtype=torch.bfloat16, device=DEV)
    k = torch.zeros(S, H, D, dtype=torch.bfloat16, device=DEV)
    v = torch.zeros_like(k)
    out = [torch.zeros_like(q) for _ in range(2)]
    ws = torch.empty(K.paged_workspace_size(s.cache, torch.bfloat16, S, S, 1, H * G), dtype=torch.uint8, device=DEV)

    def step(o):
        K.paged_append(k, v, s.cache, tab, lens, cu, 1, rope=td, slots=slots)
        K.paged_attend(q, s.cache, tab, lens, cu, 1, 1 / np.sqrt(D), out=o, workspace=ws)

    lens.copy_(i32([n + 1 for n in total]))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(out[0])                              # warm-up on the capture stream
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for o in out:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(o)
        graphs.append(g)
    for i in range(3):
        raw = bf16_values(rng.standard_normal((3, S, H * G, D)).astype(np.float32))
        q.copy_(to_dev(raw[0], torch.bfloat16))
        k.copy_(to_dev(raw[1][:, :H], torch.bfloat16))
        v.copy_(to_dev(raw[2][:, :H], torch.bfloat16))
        lens.copy_(i32([n + 1 + i for n in total]))
        for o, g in zip(out, graphs):
            o.fill_(7)
            g.replay()                            # the same step twice: a step can be repeated
        torch.cuda.synchronize()
        want = []
        for b in range(S):
            new = R.rotate(raw[1][b:b + 1, :H], table, np.array([total[b] + i]), False)
            s.k[b] = np.concatenate([s.k[b][:total[b] + i], new])
            s.v[b] = np.concatenate([s.v[b][:total[b] + i], raw[2][b:b + 1, :H]])
            kd, vd = s.decoded(b)
            want.append((R.attend_rows(raw[0][b:b + 1], kd, vd, total[b] + i + 1, 1 / np.sqrt(D), True), vd))
        for o in out:
            check_attend(o, want, np.arange(S + 1), torch.bfloat16, f"replay {i}", False)
        s.check_bytes()
    K.check(DEV)


def test_two_streams_at_once():
    """Calls on two streams with their own buffers give what each gives alone."""
    rng = np.random.default_rng(22)
    s = Sequences(rng, [900, 350], 2, 128, 4, 32, 64)
    s.append([900, 350])
    jobs = []
    for n in (1, 40):
        q = to_dev(rng.standard_normal((2 * n, 8, 128)), torch.bfloat16)
        args = (q, s.cache, i32(s.table), i32([900, 350]), i32([0, n, 2 * n]), n, 0.1)
        jobs.append((args, K.paged_attend(*args)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(10):
        outs = []
        for st, (args, _) in zip(streams, jobs):
            with torch.cuda.stream(st):
                outs.append(K.paged_attend(*args))
        torch.cuda.synchronize()
        for o, (_, want) in zip(outs, jobs):
            assert torch.equal(o, want)
    K.check(DEV)


def test_repeated_calls_give_the_same_bits():
    rng = np.random.default_rng(23)
    s = Sequences(rng, [700, 90, 1333], 2, 128, 8, 32, 96)
    s.append([700, 90, 1333])
    for n in (1, 6, 80):
        q = to_dev(rng.standard_normal((3 * n, 8, 128)), torch.bfloat16)
        args = (q, s.cache, i32(s.table), i32([700, 90, 1333]), i32([0, n, 2 * n, 3 * n]), n, 0.09)
        a = K.paged_attend(*args)
        for _ in range(5):
            assert torch.equal(a, K.paged_attend(*args))
    K.check(DEV)


@pytest.mark.parametrize("dtype,n", [(torch.bfloat16, 1), (torch.bfloat16, 60), (torch.float32, 3)])
def test_attend_powers_of_two_leave_the_bits(dtype, n):
    """Queries, K scales and V scales far from one: powers of two move the
    exponents of the result and nothing else."""
    rng = np.random.default_rng(31)
    s = Sequences(rng, [450, 130], 2, 128, 4, 32, 64)
    s.append([450, 130])
    q = bf16_values(rng.standard_normal((2 * n, 8, 128)).astype(np.float32))
    q[0, 0] = 0.0

    def run(scale_q):
        return K.paged_attend(to_dev(q * np.float32(scale_q), dtype), s.cache, i32(s.table), i32([450, 130]),
                              i32([0, n, 2 * n]), n, 0.09)

    want = run(1.0)
    for a, b in ((40, -30), (-50, 60), (0, -80)):
        s.cache.k_scales *= 2.0 ** -a
        s.cache.v_scales *= 2.0 ** b
        got = run(2.0 ** a)
        assert torch.equal(got.float() * 2.0 ** -b, want.float()), (a, b)
        s.cache.k_scales *= 2.0 ** a
        s.cache.v_scales *= 2.0 ** -b
    K.check(DEV)


@pytest.mark.parametrize("S", [129, 1500])
def test_many_sequences(S):
    """More sequences than a warp finds in one round of loads, and than the
    plan keeps in shared memory: some without rows, rows before the first and
    behind the last."""
    rng = np.random.default_rng(S)
    H, G, D, P = 1, 4, 64, 32
    lens = rng.integers(0, 70, S)
    lens[rng.random(S) < 0.1] = 0
    lens[5] = 300
    s = Sequences(rng, [int(n) for n in lens], H, D, 4, 32, P)
    s.append([int(n) for n in lens], dtype=torch.bfloat16, extra=3)
    s.check_bytes()
    counts = np.minimum(lens, rng.integers(0, 40, S))
    starts = rng.integers(0, lens - counts + 1)
    cu = np.concatenate([[0], np.cumsum(counts)])
    k, v = K.paged_gather(s.cache, i32(s.table), i32(starts), i32(cu), int(cu[-1]), int(counts.max()), torch.float32)
    k, v = k.cpu().numpy(), v.cpu().numpy()
    for b in range(S):
        if counts[b]:
            kd, vd = s.decoded(b)
            at = slice(int(starts[b]), int(starts[b] + counts[b]))
            np.testing.assert_array_equal(k[cu[b]:cu[b + 1]], kd[:, at].transpose(1, 0, 2))
            np.testing.assert_array_equal(v[cu[b]:cu[b + 1]], vd[:, at].transpose(1, 0, 2))
    for most in (1, 50):
        news = [int(min(n, rng.integers(0, most + 1))) for n in lens]
        for dtype in (torch.bfloat16, torch.float32):
            out, want, cu = run_attend(s, news, G, dtype, True, extra=2, max_q=most)
            check_attend(out, want, cu, dtype, f"at most {most}")
    K.check(DEV)


def test_pages_behind_four_gigabytes():
    """Pages whose bytes, scales and elements lie past 2^32 of their arrays."""
    rng = np.random.default_rng(33)
    H, G, D, P, far = 8, 2, 128, 64, 70000                  # 64 KB of codes a page: 4.6 GB; scales 2^31 bytes and more
    cache = K.PagedCache(far + 8, H, P, D, 8, 32, 2, DEV)
    lens = [200, 77]
    near = Sequences(rng, lens, H, D, 8, 32, P)
    table = np.full_like(near.table, -1)
    table[near.table >= 0] = far + np.arange((near.table >= 0).sum())
    raw = bf16_values(rng.standard_normal((2, sum(lens), H, D)).astype(np.float32))
    near.append(lens, dtype=torch.bfloat16, raw=raw)
    K.paged_append(to_dev(raw[0], torch.bfloat16), to_dev(raw[1], torch.bfloat16), cache, i32(table), i32(lens),
                   i32([0, 200, 277]), 200)
    for n in (1, 30):
        for dtype in (torch.bfloat16, torch.float32):
            q = to_dev(rng.standard_normal((2 * n, H * G, D)), dtype)
            a, b = (K.paged_attend(q, c, i32(t), i32(lens), i32([0, n, 2 * n]), n, 0.1)
                    for c, t in ((cache, table), (near.cache, near.table)))
            assert torch.equal(a, b), (n, dtype)
    a, b = (K.paged_gather(c, i32(t), i32([0, 0]), i32([0, 200, 277]), 277, 200)
            for c, t in ((cache, table), (near.cache, near.table)))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    K.check(DEV)


def test_sequences_that_share_their_pages():
    """A common prefix held once: several sequences read the same pages.  (To
    the reference's tolerance: the work is divided over the whole batch, so a
    row's float32 sums come in another order than alone.)"""
    rng = np.random.default_rng(34)
    s = Sequences(rng, [256], 2, 128, 4, 32, 64)
    s.append([256])
    s.table, s.k, s.v = np.repeat(s.table, 3, 0), s.k * 3, s.v * 3
    for n in (1, 40):
        q = np.tile(rng.standard_normal((n, 8, 128)).astype(np.float32), (3, 1, 1))
        out, want, cu = run_attend(s, [n] * 3, 4, torch.bfloat16, True, q=q)
        check_attend(out, want, cu, torch.bfloat16)
    K.check(DEV)


def test_captured_chunk_replays_on_new_inputs():
    """Chunks of many rows, captured with the workspace the call takes itself:
    a replay with other queries, lengths and rows a sequence is the call's own
    result on them."""
    rng = np.random.default_rng(35)
    s = Sequences(rng, [900, 400, 260], 2, 128, 8, 32, 64)
    s.append([900, 400, 260])
    T, most = 180, 90
    q = torch.zeros(T, 8, 128, dtype=torch.bfloat16, device=DEV)
    table, lens, cu = i32(s.table), i32([900, 400, 260]), i32([0, 60, 120, 180])
    out = torch.zeros_like(q)

    def step(o):
        return K.paged_attend(q, s.cache, table, lens, cu, most, 0.09, out=o)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(out)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(out)
    for new_lens, new_cu in (([900, 400, 260], [0, 60, 120, 180]), ([300, 1, 129], [0, 90, 91, 180]),
                             ([64, 0, 250], [0, 2, 2, 70])):
        q.copy_(to_dev(rng.standard_normal((T, 8, 128)), torch.bfloat16))
        lens.copy_(i32(new_lens))
        cu.copy_(i32(new_cu))
        out.fill_(7)
        graph.replay()
        want = step(torch.full_like(out, 7))
        assert torch.equal(out, want), new_lens
    K.check(DEV)
