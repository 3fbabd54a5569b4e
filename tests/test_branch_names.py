"""CPU checks of append at positions: a refused call names itself, and sizes whose product
passes 64 bits are refused."""
import ctypes

import pytest

from long_context_flashattention_gb300 import dfa
from test_branch_refusals import BASE, I3, L, append_at, cache  # noqa: F401


@pytest.mark.parametrize("kw", [dict(pos=None), dict(spec=False), dict(T=0), dict(k=None),
                                dict(k=BASE + 2), dict(v=None), dict(v=BASE + 2), dict(ws=None),
                                dict(n=255), dict(c=cache(d=96)), dict(c=cache(k=None)),
                                dict(c=cache(B=1 << 20), T=1 << 20)])
def test_append_at_names_itself(L, kw):  # noqa: F811
    assert append_at(L, **kw) != 0
    assert b"dfa_cache_append_at" in L.dfa_last_error(), L.dfa_last_error()


def test_append_still_names_itself(L):  # noqa: F811
    for k, v in ((BASE + 2, BASE), (BASE, BASE + 2)):
        assert L.dfa_cache_append(ctypes.byref(cache()), None, 4, None, k, None, v, None, 0, None,
                                  None, None, None, BASE, 256, None) == 2
        assert L.dfa_last_error().startswith(b"dfa_cache_append: ")


def test_append_at_names_its_queries(L):  # noqa: F811
    spec = dfa.rope_spec(64)
    for Hq, q, out in ((0, BASE, BASE), (4, BASE + 2, BASE), (4, BASE, BASE + 2), (4, BASE, None),
                       (4, BASE, BASE + 16)):
        assert L.dfa_cache_append_at(ctypes.byref(cache()), ctypes.byref(spec), 4, None, BASE,
                                     BASE, None, BASE, None, Hq, q, None, out, None, BASE, 256,
                                     None) != 0
        assert b"dfa_cache_append_at" in L.dfa_last_error()


def test_append_refuses_sizes_past_64_bits(L):  # noqa: F811
    """2^20 sequences of 2^29 tokens and 2 * 2^14 heads: 2^64 rows."""
    c = cache(B=1 << 20, Hkv=1 << 14)
    spec = dfa.rope_spec(64)
    rows = (BASE, I3(0, 0, 0), BASE, I3(0, 0, 0), 0, None, None, None, None, BASE, 256, None)
    assert L.dfa_cache_append(ctypes.byref(c), None, 1 << 29, None, *rows) == 2
    assert L.dfa_cache_append_at(ctypes.byref(c), ctypes.byref(spec), 1 << 29, None, BASE,
                                 *rows) == 2
