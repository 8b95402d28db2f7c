"""CPU tests of the paged calls' argument rules: every refusal is found on the
host before any launch (the fake pointers are never touched)."""

from __future__ import annotations

import ctypes

import pytest
import torch

import sm_b200 as K

ARG, ALIGN, WORKSPACE, UNSUPPORTED = 1, 3, 4, 8


def paged(bits=4, group=32, pages=8, H=2, P=64, D=64, ptr=0x10000, tail=0x900000, slots=4):
    return K._Paged(K._Cache(bits, group, pages, H, P, D, ptr, ptr + 0x100000, ptr + 0x200000, ptr + 0x300000),
                    tail, slots)


def rope(table=0x700000, n_pos=128, rot=64, inter=0):
    return ctypes.byref(K._Rope(table, n_pos, rot, inter))


def append(c=None, k=0x1000, ks=128, v=0x2000, vs=128, dt=K.KVQ_BF16, tab=0x3000, mp=4, lens=0x4000, cu=0x5000,
           slots=None, S=2, T=6, mx=4, r=None):
    c = paged() if c is None else c
    return K.lib.kvq_paged_append(ctypes.byref(c), k, ks, v, vs, dt, tab, mp, lens, cu, slots, S, T, mx, r, None)


def gather(c=None, tab=0x3000, mp=4, st=0x4000, cu=0x5000, S=2, T=6, mx=4, k=0x6000, v=0x7000, dt=K.KVQ_F32):
    c = paged() if c is None else c
    return K.lib.kvq_paged_gather(ctypes.byref(c), tab, mp, st, cu, S, T, mx, k, v, dt, None)


def attend(c=None, q=0x1000, dt=K.KVQ_BF16, tab=0x3000, mp=4, lens=0x4000, cu=0x5000, S=2, T=6, mx=4, hq=4, o=0x6000,
           ws=0x8000, wsb=1 << 40, splits=0):
    c = paged() if c is None else c
    return K.lib.kvq_paged_attend(q, dt, ctypes.byref(c), tab, mp, lens, cu, S, T, mx, hq, 1.0, 1, o, ws, wsb, splits,
                                  None)


def qk(q=0x1000, qs=256, k=0x2000, ks=128, dt=K.KVQ_BF16, T=3, hq=4, hk=2, D=64, qw=0x3000, kw=0x4000, eps=1e-6,
       pos=0x5000, r=None, qo=0x6000, ko=0x7000):
    return K.lib.kvq_qk_norm_rope(q, qs, k, ks, dt, T, hq, hk, D, qw, kw, eps, pos, rope() if r is None else r, qo, ko,
                                  None)


@pytest.mark.parametrize("bad", [dict(bits=5), dict(group=7), dict(group=0), dict(pages=0), dict(H=0), dict(P=0),
                                 dict(D=0), dict(P=48), dict(group=8, P=36), dict(ptr=0)])
def test_bad_pool(bad):
    c = paged(**bad)
    if bad == dict(ptr=0):
        c.pages.k_codes = None
    assert append(c) == ARG
    assert gather(c) == ARG
    assert attend(c) == ARG
    if bad != dict(ptr=0):
        assert K.lib.kvq_paged_workspace_size(ctypes.byref(c), K.KVQ_BF16, 2, 6, 4, 4, 0) == 0
        assert K.lib.kvq_paged_kernel_name(ctypes.byref(c), K.KVQ_BF16, 1, 4) == b"invalid"


@pytest.mark.parametrize("call", [append, gather, attend])
def test_batch_rules(call):
    lens = "st" if call is gather else "lens"
    for kw in (dict(S=0), dict(T=0), dict(mx=0), dict(mp=0), dict(tab=0), {lens: 0}, dict(cu=0), dict(dt=5),
               dict(mp=1 << 30)):
        assert call(**kw) == ARG, kw
    for kw in (dict(tab=0x3002), {lens: 0x4001}, dict(cu=0x5002), dict(c=paged(ptr=0x10008))):
        assert call(**kw) == ALIGN, kw
    assert call(S=8193, T=9000) == UNSUPPORTED
    assert call(c=paged(D=258)) in (ARG, UNSUPPORTED)


def test_append_rules():
    for kw in (dict(k=0), dict(v=0), dict(ks=127), dict(vs=10), dict(c=paged(tail=0)), dict(c=paged(slots=0)),
               dict(r=rope(rot=0)), dict(r=rope(rot=3)), dict(r=rope(rot=66)), dict(r=rope(n_pos=0))):
        assert append(**kw) == ARG, kw
    for kw in (dict(k=0x1001), dict(v=0x2001), dict(dt=K.KVQ_F32, k=0x1002), dict(slots=0x8001),
               dict(c=paged(tail=0x900004)), dict(r=rope(table=0x700002))):
        assert append(**kw) == ALIGN, kw
    assert append(c=paged(group=256, P=256, D=256), ks=512, vs=512) == UNSUPPORTED
    assert append(c=paged(D=258), ks=600, vs=600) == UNSUPPORTED


def test_gather_rules():
    assert gather(k=0, v=0) == ARG
    assert gather(k=0x6008) == ALIGN and gather(v=0x7004) == ALIGN


def test_attend_rules():
    for kw in (dict(q=0), dict(o=0), dict(hq=3), dict(hq=0), dict(splits=-1)):
        assert attend(**kw) == ARG, kw
    for kw in (dict(q=0x1008), dict(o=0x6002), dict(ws=0x8008)):
        assert attend(**kw) == ALIGN, kw
    assert attend(ws=0) == WORKSPACE and attend(wsb=16) == WORKSPACE
    assert attend(c=paged(D=258)) == UNSUPPORTED


def test_qk_rules():
    for kw in (dict(q=0), dict(qo=0), dict(k=0), dict(ko=0), dict(T=0), dict(hq=0), dict(hk=0), dict(D=0), dict(qs=255),
               dict(ks=127), dict(dt=9), dict(eps=-1.0), dict(eps=float("nan")), dict(r=rope(rot=66)),
               dict(r=rope(rot=5)), dict(r=rope(n_pos=0)), dict(pos=0)):
        assert qk(**kw) == ARG, kw
    for kw in (dict(q=0x1001), dict(k=0x2001), dict(qw=0x3001), dict(kw=0x4001), dict(qo=0x6001), dict(ko=0x7001),
               dict(pos=0x5002), dict(r=rope(table=0x700002))):
        assert qk(**kw) == ALIGN, kw
    assert qk(D=1026, qs=1 << 20, ks=1 << 20) == UNSUPPORTED


def test_workspace_grows_with_splits_and_covers_any_batch():
    c = paged(D=128)
    f = lambda **k: K.lib.kvq_paged_workspace_size(ctypes.byref(c), k.get("dt", K.KVQ_BF16), k.get("S", 4), k.get("T", 4),
                                                   k.get("mx", 1), k.get("hq", 8), k.get("splits", 3))
    assert 0 < f() < f(splits=300)
    assert f(splits=-1) == 0 and f(hq=3) == 0 and f(S=0) == 0 and f(dt=7) == 0
    assert f(T=4000, mx=1000) > 0


def test_binding_refuses_on_the_host():
    cpu = "cpu"
    with pytest.raises(ValueError):
        K.PagedCache(4, 2, 48, 64, device=cpu)                      # page not a multiple of the group
    with pytest.raises(K.KVQError):
        K.PagedCache(4, 2, 64, 64, bits=3, device=cpu)
    with pytest.raises(ValueError):
        K.PagedCache(4, 2, 64, 64, slots=0, device=cpu)
    with pytest.raises(ValueError):
        K.rope_table(16, 7, device=cpu)
    with pytest.raises(ValueError):
        K.qk_norm_rope(torch.zeros(2, 4, 64), None, None, None)     # not on a GPU
    with pytest.raises(TypeError):
        K.qk_norm_rope(3, None, None, None)
    with pytest.raises(TypeError):
        K._calls.paged_append(1)
    with pytest.raises(ValueError):                                 # given buffers must be on the cache's GPU
        K.PagedCache(4, 2, 64, 64, device=cpu, buffers=[torch.zeros(1, dtype=torch.uint8)] * 5)


def test_rope_table_far_positions_keep_their_phase():
    t = K.rope_table(70000, 8, device="cpu").double()
    a = torch.arange(70000, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, 8, 2, dtype=torch.float64) / 8)
    # one rounding of a value of at most 1 to float32
    assert (t[:, :4] - a.cos()).abs().max() <= 2.0 ** -24 and (t[:, 4:] - a.sin()).abs().max() <= 2.0 ** -24
