"""CPU checks: outputs of the paged-cache calls that share memory are refused, since the
kernels' blocks read and write them side by side."""
import ctypes

import torch

from long_context_flashattention_gb300 import dfa

BUF = (ctypes.c_uint8 * (1 << 16))()
BASE = (ctypes.addressof(BUF) + 255) & ~255
FAR = BASE + (1 << 15)
I3 = ctypes.c_int64 * 3


def cache():
    return ctypes.byref(dfa.PagedCacheDesc(0, 16, 2, 64, 8, 0, BASE, BASE, None, None, 2, 4, BASE,
                                           BASE))


def test_decode_refuses_an_output_among_its_queries():
    L, B, Hq, T, d = dfa.lib(), 2, 4, 1, 64
    for fp32 in (False, True):
        desc = dfa.make_desc(B, Hq, 2, 1, d, o_fp32=fp32)
        span = B * Hq * T * d * 2
        for o in (BASE, BASE + 16, BASE + span - 16):
            assert L.dfa_decode_paged(ctypes.byref(desc), cache(), T, None, BASE, None, o, FAR, FAR,
                                      1 << 40, None) == 1
            assert b"overlap" in L.dfa_last_error()
        # behind one another they pass the check (and then want a device)
        if not torch.cuda.is_available():
            L.dfa_decode_paged(ctypes.byref(desc), cache(), T, None, BASE, None, BASE + span, FAR,
                               FAR, 1 << 40, None)
            assert b"overlap" not in L.dfa_last_error()
        # heads of a wider buffer: up to the last row's end
        wide = I3(10 * d, d, d)
        last = BASE + (10 * d + 3 * d + d) * 2
        assert L.dfa_decode_paged(ctypes.byref(desc), cache(), T, None, BASE, wide, last - 16, FAR,
                                  FAR, 1 << 40, None) == 1


def test_gather_refuses_outputs_on_top_of_one_another():
    L = dfa.lib()
    span = 2 * 2 * 8 * 64 * 2
    for v in (BASE, BASE + 256, BASE + span - 16):
        assert L.dfa_cache_gather(cache(), 0, 8, BASE, v, FAR, 256, None) == 1
        assert b"overlap" in L.dfa_last_error()
    if not torch.cuda.is_available():
        L.dfa_cache_gather(cache(), 0, 8, BASE, BASE + span, FAR, 256, None)
        assert b"overlap" not in L.dfa_last_error()
    assert L.dfa_cache_gather(cache(), 64, 8, BASE, BASE, FAR, 256, None) == 0   # no such rows
