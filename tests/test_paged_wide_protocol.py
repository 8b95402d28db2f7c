"""The paged chunk kernel's wide form in the CPU model of its barriers
(test_paged_chunk_protocol): the decode warps leave each key's power beside the K
tile and V's exponents beside the V tile, and the softmax reads both, waiting for
V's tile first.  Segments of both forms follow one another in a CTA."""

import pytest

from tests.test_paged_chunk_protocol import DEEP, DW, RW, SEGMENTS, PagedModel, block_list, roles_of

KEYS = 4                                        # K tiles whose powers are kept


def with_wide(m, is_wide, keys=KEYS, wait_v=True):
    """roles_of with the wide form's reads, writes and waits: is_wide(segment)."""
    blocks, roles = m.blocks, roles_of(m)

    def readers(p):
        return {("sm", t, w) for t in range(blocks[p][3]) for w in range(RW)}

    def decode(steps, w):
        x = {"K": 0, "V": 0}
        for op in steps:
            typ = {"KR": "K", "VR": "V"}.get(op[1] if op[1] == "VR" else op[1][0]) if op[0] == "arrive" else None
            if typ:
                k = x[typ]
                x[typ] += 1
                if is_wide(blocks[k][0]):
                    place = ("keys", k % keys, w) if typ == "K" else ("values", w)
                    yield ("do", lambda place=place, k=k: m.write(place, k, readers))
            yield op

    def softmax(steps, t):
        mine = iter([k for k in range(len(blocks)) if blocks[k][3] > t])
        for op in steps:
            yield op
            if op[0] == "wait" and op[1][0] == "SF":
                k = next(mine)
                # the segment's form is read at every block
                yield ("do", lambda k=k: m.read(("X", blocks[k][0] % DEEP), blocks[k][0], ("form", t)))
                if is_wide(blocks[k][0]):
                    if wait_v:
                        yield ("wait", "VR", k)

                    def f(k=k, w=w_of[id(steps)]):
                        for d in range(DW):
                            m.read(("keys", k % keys, d), k, ("sm", t, w))
                            m.read(("values", d), k, ("sm", t, w))
                    yield ("do", f)

    w_of = {id(roles[f"softmax{t}.{w}"]): w for t in range(2) for w in range(RW)}
    out = dict(roles)
    for w in range(DW):
        out[f"decode{w}"] = decode(roles[f"decode{w}"], w)
    for t in range(2):
        for w in range(RW):
            out[f"softmax{t}.{w}"] = softmax(roles[f"softmax{t}.{w}"], t)
    return out


@pytest.mark.parametrize("segments", SEGMENTS, ids=lambda s: "-".join(f"{n}x{t}" for n, t in s))
@pytest.mark.parametrize("n_units", [3, 6, 11, 12])
@pytest.mark.parametrize("form", ["all", "even", "odd"])
def test_wide_form_holds(segments, n_units, form):
    is_wide = {"all": lambda s: True, "even": lambda s: s % 2 == 0, "odd": lambda s: s % 2 == 1}[form]
    for seed in range(5):
        m = PagedModel(block_list(segments), n_units, seed, lag=(seed % 4) * 0.3)
        m.run(with_wide(m, is_wide))


@pytest.mark.parametrize("fault", [dict(wait_v=False), dict(keys=2)])
def test_the_wait_and_the_depth_are_needed(fault):
    for segments in ([(28, 2)], [(27, 1)], [(9, 1), (9, 2), (9, 1)]):
        for seed in range(60):
            m = PagedModel(block_list(segments), 12, seed, lag=(seed % 4) * 0.3)
            try:
                m.run(with_wide(m, lambda s: True, **fault))
            except AssertionError:
                return
    raise AssertionError(f"{fault} went unnoticed")
