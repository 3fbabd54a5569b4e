"""CPU checks of a paged cache's status word: where the device's errors of calls
without a workspace go."""
import ctypes

import pytest
import torch

from long_context_flashattention_gb300 import dfa


def paged_cache():
    kv = torch.zeros(8, 2, 16, 64, dtype=torch.bfloat16)
    return dfa.PagedCache(kv, kv.clone(), torch.zeros(2, 4, dtype=torch.int32),
                          torch.zeros(2, dtype=torch.int32))


def test_a_cache_has_a_status_of_its_own():
    c = paged_cache()
    assert c.status.dtype == torch.uint8 and c.status.numel() == 256 and not c.status.any()
    with pytest.raises(AttributeError, match="contents"):
        c.status = torch.zeros(256, dtype=torch.uint8)
    # given a workspace, calls report to that; without one, to the cache
    assert not c.desc.status
    ws, ref = dfa._ws(torch.zeros(256, dtype=torch.uint8), 256, c, None)
    assert ref is c._ref
    ws, ref = dfa._ws(None, 256, c, None)
    assert ref._obj.status == c.status.data_ptr() and ref._obj.k == c.k.data_ptr()


def test_a_misaligned_status_is_refused():
    buf = (ctypes.c_uint8 * 4096)()
    base = (ctypes.addressof(buf) + 255) & ~255
    c = dfa.PagedCacheDesc(0, 16, 2, 64, 8, 0, base, base, None, None, 2, 4, base, base, base + 16)
    assert dfa.lib().dfa_cache_gather(ctypes.byref(c), 0, 4, base, base, base, 256, None) == 1
    assert b"status" in dfa.lib().dfa_last_error()
