"""CPU test: each call of the paged cache refuses what the header says it does."""

from __future__ import annotations

import pytest

from tests.test_paged_abi import ARG, UNSUPPORTED, append, attend, gather, paged


@pytest.mark.parametrize("call", [append, gather, attend])
def test_limits_of_every_call(call):
    assert call(S=8193, T=9000) == UNSUPPORTED
    wide = dict(ks=1 << 23, vs=1 << 23) if call is append else dict(hq=65536) if call is attend else {}
    assert call(c=paged(H=65536, D=32), **wide) == UNSUPPORTED
    wide = dict(ks=1 << 20, vs=1 << 20) if call is append else {}
    assert call(c=paged(D=288), **wide) == UNSUPPORTED
    assert call(c=paged(P=64), mp=(2 ** 31 - 256) // 64 + 1) == ARG
    assert call(c=paged(P=1 << 20, group=32), mp=2048) == ARG


def test_limits_of_one_call():
    assert append(c=paged(group=256, P=256, D=256), ks=512, vs=512) == UNSUPPORTED
    assert attend(T=1 << 29, hq=2, mx=1 << 29) == UNSUPPORTED
