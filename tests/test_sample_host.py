"""Sampling's refusal of probabilities laid over the logits, against a model that compares every byte (no GPU:
only calls that are refused before any launch are made; the pointers are never dereferenced)."""
import ctypes

import pytest

BASE = 1 << 20
WS = ctypes.c_void_p(1 << 21)


@pytest.fixture(scope="module")
def irm():
    from mla_position_independent_gb300 import build
    build.build()
    import mla_position_independent_gb300 as m
    m.lib()
    return m


def shares_a_byte(off, each, ld, pld, V, T):
    mine = {t * ld * each + i for t in range(T) for i in range(V * each)}
    return any(off + t * pld * 4 + i in mine for t in range(T) for i in range(V * 4))


@pytest.mark.parametrize("type,each", [(0, 4), (1, 2)])
@pytest.mark.parametrize("V,T,ld,pld", [(10, 1, 10, 10), (10, 3, 40, 20), (10, 3, 60, 30), (10, 3, 30, 30), (10, 4, 20, 10), (7, 3, 64, 32), (9, 2, 23, 9)])
def test_every_overlap_is_refused(irm, type, each, V, T, ld, pld):
    refused = 0
    for off in range(-4 * T * pld - 8, each * T * ld + 8, 4):
        if not shares_a_byte(off, each, ld, pld, V, T):
            continue
        st = irm.lib().irm_sample(ctypes.c_void_p(BASE), type, ld, T, V, None, None, None, None, ctypes.c_void_p(BASE << 2), ctypes.c_void_p(BASE << 3),
                                  ctypes.c_void_p(BASE + off), pld, WS, 256, None)
        assert st == -1 and b"overlap" in irm.lib().irm_last_error(), off
        refused += 1
    assert refused > V // 4
