"""The paged chunk kernel's synchronization protocol, as a model on the CPU
(the machine of test_chunk_protocol: hardware parity semantics for every wait,
copies and MMAs that complete out of order, a version on every buffer).

What differs from the contiguous kernel: the ring holds half-units of 64 keys,
each decoded by four of the eight decode warps; a segment's item has one or two
row tiles, so the second tile's barriers count its own blocks; a lone tile has
its scores in both tiles' columns in turn, with barriers of their own for the
second, and its next scores before its values; and the Q loader leaves a segment's powers of two, four segments deep, to the decode warps and
the softmax.  A ring of odd length gives a slot to the two halves in turn,
and a decode warp sees only its own half's uses of it: the slot's full barrier
is one per half, since on a shared one a warp would wait for a phase without
having seen the one before, and a parity wait cannot tell those apart."""

import pytest

from tests.test_chunk_protocol import Bar, Model

DW, RW, DEEP = 8, 4, 4


class PagedModel(Model):
    """blocks: [(segment, first, last, tiles)]."""

    def __init__(self, blocks, n_units, seed, lag):
        super().__init__(blocks, 2, n_units, seed, lag)
        for u in range(n_units):
            self.B[("RE", u)] = Bar(DW // 2)
            for half in range(2):
                self.B[("RF", u, half)] = Bar(1)
        for i in range(DEEP):
            self.B[("X", i)] = Bar(1)
        self.B[("SF", 2)], self.B[("PF", 2)], self.B[("PD", 2)] = Bar(1), Bar(RW), Bar(1)


def roles_of(m, drop=None, shift=None, shared_full=False):
    blocks, nu = m.blocks, m.nu

    def full(n):
        """Barrier and phase of half-unit n's arrival."""
        if shared_full:
            return ("RF", n % nu), n // nu
        return ("RF", n % nu, n % 2), (n // nu) // (2 if nu % 2 else 1)

    nb = len(blocks)
    segs = []
    for b in blocks:
        if b[1]:
            segs.append([])
        segs[-1].append(b)
    seg_blocks = [[i for i, b in enumerate(blocks) if b[0] == s[0][0]] for s in segs]
    tiles = [b[3] for b in blocks]
    # what a tile uses in a block: 0 and 1, the tiles; 2, a lone tile's other S
    use = []
    for k, b in enumerate(blocks):
        use.append([0, 1] if b[3] == 2 else [0 if b[1] else 2 - use[-1][0]])

    def nth(u, k):
        return sum(1 for x in use[:k] if u in x)

    def tile_at(u, k):
        """The tile whose block k's S is in the columns of u."""
        return 0 if tiles[k] == 1 else min(u, 1)
    units = [("K", 0)]
    for v in range(nb):
        if v + 1 < nb:
            units.append(("K", v + 1))
        units.append(("V", v))

    def wait(name, bar, k):
        return [] if drop == name else [("wait", bar, k + (shift == name))]

    def producer():
        n = 0
        for typ, blk in units:
            for half in range(2):
                if n + half >= nu:
                    yield from wait("ring_empty", ("RE", (n + half) % nu), (n + half) // nu - 1)
            for half in range(2):
                slot = n % nu
                yield ("expect_tx", full(n)[0])
                yield ("copy", full(n)[0], lambda slot=slot, v=(typ, blk, half): m.write(
                    ("ring", slot), v, lambda p: {("dec", w) for w in range(4 * p[2], 4 * p[2] + 4)}))
                n += 1

    def qloader():
        for s in range(len(segs)):
            yield ("do", lambda s=s: m.write(("X", s % DEEP), s, lambda p: {("dec", w) for w in range(DW)} | {
                ("sm", t, w) for t in range(segs[p][0][3]) for w in range(RW)}))
            yield ("arrive", ("X", s % DEEP))
            if s > 0:
                yield from wait("q_free", "QF", s - 1)
            yield ("expect_tx", "QR")
            yield ("copy", "QR", lambda s=s: m.write(
                "Q", s, lambda p: {("qk", t, i) for i in seg_blocks[p] for t in range(tiles[i])}))

    def decode(w):
        half = w // 4
        n = half
        count = {"K": 0, "V": 0}
        for typ, blk in units:
            slot, x = n % nu, count[typ]
            if typ == "K" and blocks[blk][1]:
                yield from wait("powers", ("X", blocks[blk][0] % DEEP), blocks[blk][0] // DEEP)
                yield ("do", lambda s=blocks[blk][0]: m.read(("X", s % DEEP), s, ("dec", w)))
            yield from wait("ring_full", *full(n))
            if typ == "K" and x >= 2:
                yield from wait("k_free", ("KF", x & 1), (x >> 1) - 1)
            if typ == "V" and x >= 1:
                yield from wait("v_free", "VF", x - 1)
            buf = x & 1 if typ == "K" else 0
            readers = ((lambda p: {("qk", t, p) for t in range(tiles[p])}) if typ == "K"
                       else (lambda p: {("pv", t, p) for t in range(tiles[p])}))
            yield ("do", lambda slot=slot, v=(typ, blk, half), readers=readers, buf=buf: (
                m.read(("ring", slot), v, ("dec", w)),
                m.write((v[0], buf, w), v[1], readers)))
            yield ("arrive", ("KR", buf) if typ == "K" else "VR")
            yield ("arrive", ("RE", slot))
            n += 2
            count[typ] += 1

    def qk(u, k):
        t, at = u & 1, min(u, 1)

        def fn():
            m.read("Q", next(i for i, s in enumerate(seg_blocks) if k in s), ("qk", t, k))
            for w in range(DW):
                m.read(("K", k & 1, w), k, ("qk", t, k))
            m.write(("S", at), k, lambda p: {("pv", tile_at(at, p), p)} | {
                ("sm", tile_at(at, p), p, w) for w in range(RW)})
        return [("mma", ("S", at), fn), ("commit", ("SF", u))]

    def pv(u, k):
        t, at = u & 1, min(u, 1)

        def fn():
            for w in range(RW):
                m.read(("P", at, w), k, ("pv", t, k))
            for w in range(DW):
                m.read(("V", 0, w), k, ("pv", t, k))
            m.reads.setdefault(("S", at), set()).add(("pv", t, k))
            for w in range(RW):
                o = ("O", t, w)
                if blocks[k][1]:
                    prev = m.buf.get(o)
                    assert prev is None or ("epi", t, prev) in m.reads.get(o, set()), "O overwritten unread"
                else:
                    assert m.buf.get(o) == k - 1, f"P V({k}) accumulates onto O v{m.buf.get(o)}"
                m.buf[o] = k
                m.reads[o] = set()
        return [("mma", ("O", t), fn), ("commit", ("PD", u))]

    def mma():
        done = [0, 0, 0]

        def product(u, k):
            yield from wait("p_full", ("PF", u), done[u])
            yield from pv(u, k)
            done[u] += 1

        def pv_done(u):
            for x in ([0] if u == 0 else [1, 2]):
                if done[x] > 0:
                    yield from wait("pv_done", ("PD", x), done[x] - 1)

        def scores(u, k):
            yield from pv_done(u)
            yield from qk(u, k)

        def freed(k):
            yield ("commit", ("KF", k & 1))
            if blocks[k][2]:
                yield ("commit", "QF")

        sq = 0
        for k in range(-1, nb):
            have, nxt = k >= 0, k + 1 < nb
            boundary = nxt and blocks[k + 1][1]
            lone = have and nxt and not boundary and tiles[k + 1] == 1
            if lone:
                yield from wait("k_ready", ("KR", (k + 1) & 1), (k + 1) >> 1)
                yield from scores(use[k + 1][0], k + 1)
                yield from freed(k + 1)
            if have:
                yield from wait("v_ready", "VR", k)
                yield from product(use[k][0], k)
            for step in range(2):
                if step == boundary:
                    if nxt and not lone:
                        if boundary:
                            yield from wait("q_ready", "QR", sq)
                            sq += 1
                        yield from wait("k_ready", ("KR", (k + 1) & 1), (k + 1) >> 1)
                        yield from scores(0, k + 1)
                elif have:
                    if tiles[k] == 2:
                        yield from product(1, k)
                    yield ("commit", "VF")
            if nxt and not lone:
                if tiles[k + 1] == 2:
                    yield from scores(1, k + 1)
                yield from freed(k + 1)

    def softmax(t, w):
        for k in range(nb):
            if tiles[k] <= t:
                continue
            u = use[k][t]
            n = nth(u, k)
            yield from wait("s_full", ("SF", u), n)
            if tiles[k] == 1 and not blocks[k][1]:          # (as if O were rescaled every time)
                yield from wait("rescale", ("PD", 2 - u), nth(2 - u, k) - 1)

            def f(k=k, u=u):
                m.read(("S", min(u, 1)), k, ("sm", t, k, w))
                if blocks[k][1]:
                    m.read(("X", blocks[k][0] % DEEP), blocks[k][0], ("sm", t, w))
                else:
                    assert m.buf.get(("O", t, w)) == k - 1, "rescale before the previous P V finished"
                m.buf[("P", min(u, 1), w)] = k
            yield ("do", f)
            yield ("arrive", ("PF", u))
            if blocks[k][2]:
                yield from wait("epilogue_pv", ("PD", u), n)
                yield ("do", lambda k=k: m.read(("O", t, w), k, ("epi", t, k)))

    roles = {"producer": producer(), "q": qloader(), "mma": mma()}
    for w in range(DW):
        roles[f"decode{w}"] = decode(w)
    for t in range(2):
        for w in range(RW):
            roles[f"softmax{t}.{w}"] = softmax(t, w)
    return roles


def block_list(segments):
    """segments: [(blocks, tiles)]."""
    return [(s, j == 0, j == n - 1, t) for s, (n, t) in enumerate(segments) for j in range(n)]


SEGMENTS = [[(1, 1)], [(1, 2)], [(3, 2)], [(28, 2)], [(5, 2), (23, 2)], [(1, 1), (1, 2), (1, 1), (1, 2)],
            [(27, 2), (1, 1)], [(1, 2), (27, 1)], [(2, 2), (2, 1), (2, 2), (2, 1), (3, 2)], [(13, 1), (14, 1)],
            [(4, 1), (2, 2), (5, 1), (1, 2), (1, 1), (7, 1)]]


@pytest.mark.parametrize("segments", SEGMENTS, ids=lambda s: "-".join(f"{n}x{t}" for n, t in s))
@pytest.mark.parametrize("n_units", [3, 6, 11, 12])
def test_protocol_holds(segments, n_units):
    for seed in range(10):
        m = PagedModel(block_list(segments), n_units, seed, lag=(seed % 4) * 0.3)
        m.run(roles_of(m))


@pytest.mark.parametrize("drop", ["ring_empty", "q_free", "k_free", "v_free", "pv_done", "epilogue_pv",
                                  "p_full", "v_ready", "k_ready", "s_full", "powers", "rescale"])
def test_every_wait_is_needed(drop):
    for segments in ([(3, 2)], [(5, 2), (23, 2)], [(27, 2), (1, 1)], [(9, 1), (9, 2), (9, 1)]):
        for seed in range(60):
            m = PagedModel(block_list(segments), 3, seed, lag=(seed % 4) * 0.3)
            try:
                m.run(roles_of(m, drop=drop))
            except AssertionError:
                return
    raise AssertionError(f"leaving out the {drop} wait went unnoticed")


@pytest.mark.parametrize("shift", ["ring_empty", "ring_full", "k_free", "v_free", "pv_done", "p_full",
                                   "v_ready", "k_ready", "s_full", "q_ready", "powers"])
def test_every_phase_is_right(shift):
    with pytest.raises(AssertionError):
        for seed in range(10):
            m = PagedModel(block_list([(5, 2), (18, 1), (5, 2)]), 3, seed, lag=0.3)
            m.run(roles_of(m, shift=shift))


def test_a_full_barrier_shared_by_the_halves_of_an_odd_ring_aliases():
    with pytest.raises(AssertionError, match="parity alias"):
        for seed in range(200):
            m = PagedModel(block_list([(28, 2)]), 3, seed, lag=(seed % 4) * 0.3)
            m.run(roles_of(m, shared_full=True))
