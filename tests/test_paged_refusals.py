"""CPU checks of the rotary and paged-cache calls: the C entries refuse bad
arguments before any device work, and the binding refuses tensors that the
calls do not take."""
import ctypes

import pytest
import torch

from long_context_flashattention_gb300 import dfa

_BUF = (ctypes.c_uint8 * 8192)()
BASE = (ctypes.addressof(_BUF) + 255) & ~255
I3 = ctypes.c_int64 * 3


@pytest.fixture(scope="module")
def L():
    return dfa.lib()


def spec(**kw):
    s = dict(layout="half", rot_dim=64)
    return dfa.rope_spec(64, **{**s, **kw})


def cache(**kw):
    c = dict(dtype=1, page=16, Hkv=2, d=64, npages=8, page_stride=0, k=BASE, v=BASE,
             k_scale=BASE, v_scale=BASE, B=2, max_pages=4, block_table=BASE, seq_lens=BASE)
    return dfa.PagedCacheDesc(**{**c, **kw})


def rope(L, s=None, B=1, H=2, n=8, d=64, fp32=0, x=BASE, xs=None, out=BASE + 4096, os_=None,
         m=None, pos=None, inverse=0):
    s = spec() if s is None else s
    return L.dfa_rope(ctypes.byref(s), B, H, n, d, fp32, x, xs, out, os_,
                      None if m is None else ctypes.byref(m), pos, inverse, None)


def test_rope_refuses(L):
    bad = dfa.RopeSpec(2, 64, 0, 0, 1e4, 1, 0, 0, 0, 1)
    assert rope(L, bad) == 1 and b"layout" in L.dfa_last_error()
    for kw, code in ((dict(rot_dim=128), 1), (dict(rot_dim=24), 2), (dict(rot_dim=0), 1),
                     (dict(rot_dim=15), 1), (dict(theta_base=1.0), 1),
                     (dict(theta_base=float("nan")), 1), (dict(gain=-1.0), 1),
                     (dict(gain=float("inf")), 1), (dict(scaling="linear", factor=0.0), 1),
                     (dict(scaling="bands", factor=2.0, orig_len=0.0, low=1.0, high=4.0), 1),
                     (dict(scaling="bands", factor=2.0, orig_len=99.0, low=4.0, high=4.0), 1),
                     (dict(scaling="bands", factor=2.0, orig_len=99.0, low=-1.0, high=4.0), 1)):
        assert rope(L, spec(**kw)) == code, kw
    bad = dfa.RopeSpec(0, 64, 3, 0, 1e4, 1, 0, 0, 0, 1)
    assert rope(L, bad) == 1 and b"scaling" in L.dfa_last_error()
    assert L.dfa_rope(None, 1, 2, 8, 64, 0, BASE, None, BASE + 4096, None, None, None, 0,
                      None) == 1
    for kw, code in ((dict(d=96), 2), (dict(B=0), 1), (dict(H=0), 1), (dict(n=-1), 1),
                     (dict(n=1 << 30), 2), (dict(fp32=2), 1), (dict(inverse=2), 1),
                     (dict(x=None), 1), (dict(out=None), 1), (dict(x=BASE + 8), 2),
                     (dict(out=BASE + 2), 2), (dict(xs=I3(1024, 512, 60)), 2),
                     (dict(xs=I3(1024, -512, 64)), 1),
                     (dict(os_=I3(1024, 0, 64)), 1),         # heads on top of one another
                     (dict(os_=I3(1024, 64, 64)), 1),
                     (dict(out=BASE + 128), 1),              # overlaps x, not the same
                     (dict(out=BASE, os_=I3(1024, 64, 128)), 1)):
        assert rope(L, **kw) == code, kw
    assert rope(L, n=0, x=None, out=None) == 0               # nothing to do
    for m, code in ((dfa.pos_map(1, (7, 0), (0, 0)), 1), (dfa.pos_map(3, (8, 0), (0, 0)), 1),
                    (dfa.pos_map(2, (9, -1), (0, 0)), 1),
                    (dfa.pos_map(1, (8, 0), (-1, 0)), 2),
                    (dfa.pos_map(1, (8, 0), (2 ** 31 - 5, 0)), 2),
                    (dfa.pos_map(1, (8, 0), (0, 0), 2, 1), 2),
                    (dfa.pos_map(1, (8, 0), (0, 0), 1, 2 ** 40), 2)):
        assert rope(L, m=m) == code


CACHE_BAD = [(dict(dtype=2), 1), (dict(d=96), 2), (dict(page=8), 2), (dict(page=48), 2),
             (dict(Hkv=0), 1), (dict(B=0), 1), (dict(max_pages=0), 1),
             (dict(max_pages=1 << 27), 1), (dict(npages=0), 1), (dict(npages=1 << 31), 1),
             (dict(page_stride=100), 1), (dict(page_stride=2 * 16 * 64 + 8), 2),
             (dict(k=None), 1), (dict(v=None), 1), (dict(k_scale=None), 1),
             (dict(v_scale=None), 1), (dict(block_table=None), 1), (dict(seq_lens=None), 1),
             (dict(k=BASE + 8), 2), (dict(v=BASE + 1), 2)]


def append(L, c=None, s=None, T=4, k=BASE, ks=None, v=BASE, vs=None, Hq=0, q=None, qs=None,
           qo=None, qos=None, ws=BASE, n=256):
    return L.dfa_cache_append(None if c is False else ctypes.byref(c or cache()),
                              None if s is None else ctypes.byref(s), T, None, k, ks, v, vs, Hq,
                              q, qs, qo, qos, ws, n, None)


def gather(L, c=None, pos0=0, n=4, k=BASE, v=BASE, ws=BASE, wn=256):
    return L.dfa_cache_gather(None if c is False else ctypes.byref(c or cache()), pos0, n, k, v,
                              ws, wn, None)


def decode(L, c=None, T=1, q=BASE, qs=None, o=BASE, lse=BASE, ws=BASE, n=1 << 40, desc=None,
           **kw):
    if desc is None:
        desc = dfa.make_desc(**{**dict(B=2, Hq=4, Hkv=2, N=1, d=64), **kw})
    return L.dfa_decode_paged(ctypes.byref(desc), None if c is False else ctypes.byref(c or cache()),
                              T, None, q, qs, o, lse, ws, n, None)


@pytest.mark.parametrize("kw,code", CACHE_BAD)
def test_every_call_refuses_a_bad_cache(L, kw, code):
    assert append(L, cache(**kw)) == code and L.dfa_last_error()
    assert gather(L, cache(**kw)) == code
    d = {k: v for k, v in kw.items() if k in ("d", "Hkv", "B")}
    assert decode(L, cache(**kw)) == (code if not d else code)


def test_append_refuses(L):
    assert append(L, False) == 1
    far = BASE + 4096
    for kw, code in ((dict(T=0), 1), (dict(T=1 << 30), 1), (dict(k=None), 1), (dict(v=None), 1),
                     (dict(k=BASE + 2), 2), (dict(ks=I3(512, 256, 60)), 2),
                     (dict(vs=I3(512, 252, 64)), 2), (dict(ws=None), 3), (dict(n=255), 3),
                     (dict(ws=BASE + 16), 3), (dict(s=spec(rot_dim=24)), 2),
                     (dict(q=BASE, qo=far, Hq=2), 1),                  # queries, no rotation
                     (dict(q=BASE, qo=far, Hq=0, s=spec()), 1),
                     (dict(q=BASE, qo=None, Hq=2, s=spec()), 1),
                     (dict(q=BASE, qo=BASE + 256, Hq=2, s=spec()), 1)):
        assert append(L, **kw) == code, kw


def test_gather_refuses(L):
    assert gather(L, False) == 1
    for kw, code in ((dict(pos0=-1), 1), (dict(n=-1), 1), (dict(n=1 << 30), 1),
                     (dict(k=BASE + 8), 2), (dict(ws=None), 3), (dict(wn=10), 3)):
        assert gather(L, **kw) == code, kw
    assert gather(L, n=0) == 0 and gather(L, pos0=64) == 0   # no such rows
    assert gather(L, k=None, v=None) == 0


def test_decode_refuses(L):
    assert decode(L, False) == 1
    for kw, code in ((dict(T=0), 1), (dict(T=513), 2), (dict(Hq=3), 1), (dict(B=3), 1),
                     (dict(Hkv=4), 1), (dict(d=128), 1), (dict(scale=0.0), 1),
                     (dict(scale=float("nan")), 1), (dict(q=None), 1), (dict(q=BASE + 2), 2),
                     (dict(qs=I3(256, 64, 60), T=2), 2), (dict(o=None), 1), (dict(lse=None), 1),
                     (dict(o=BASE + 8), 2), (dict(ws=None), 3), (dict(n=100), 3)):
        assert decode(L, **kw) == code, kw
    desc = dfa.make_desc(2, 4, 2, 1, 64)
    desc.ndocs, desc.doc_bounds = 1, BASE
    assert decode(L, desc=desc) == 2
    for f, x in (("causal", 2), ("o_fp32", 3)):
        desc = dfa.make_desc(2, 4, 2, 1, 64)
        setattr(desc, f, x)
        assert decode(L, desc=desc) == 1
    assert L.dfa_decode_paged(None, ctypes.byref(cache()), 1, None, BASE, None, BASE, BASE, BASE,
                              1 << 40, None) == 1


def test_decode_workspace_size(L):
    def size(T, **kw):
        desc = dfa.make_desc(**{**dict(B=2, Hq=4, Hkv=2, N=1, d=64), **kw})
        return L.dfa_decode_paged_workspace_size(ctypes.byref(desc), T)
    assert size(1) >= 256 and size(1, B=1000) == size(1)   # whatever the batch
    assert size(0) == 0 and size(513) == 0 and size(1, d=96) == 0 and size(1, Hq=3) == 0
    assert L.dfa_decode_paged_workspace_size(None, 1) == 0


def test_binding_refuses():
    """Host tensors, wrong dtypes, shapes and strides, before any device work."""
    bf = torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device"):
        dfa.rope(bf, spec())
    e4 = torch.zeros(8, 2, 16, 64).to(torch.float8_e4m3fn)
    table, lens = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    sc = torch.ones(8, 2)
    ok = dfa.PagedCache(e4, e4, table, lens, k_scale=sc, v_scale=sc)
    assert ok.desc.page == 16 and ok.desc.npages == 8 and ok.desc.page_stride == 2 * 16 * 64
    for call in (lambda: dfa.cache_append(ok, bf, bf), lambda: dfa.cache_gather(ok, 4),
                 lambda: dfa.decode_paged(ok, bf)):
        with pytest.raises(ValueError, match="device"):
            call()
    bad = [
        (e4.float(), e4.float(), table, lens, sc, sc),            # dtype
        (e4, e4, table, lens, None, None),                        # no scales
        (e4, e4, table, lens, sc, None),
        (e4.to(torch.bfloat16), e4.to(torch.bfloat16), table, lens, sc, sc),
        (e4, e4[:4], table, lens, sc, sc),                        # k and v differ
        (e4.transpose(1, 2), e4.transpose(1, 2), table, lens, sc, sc),
        (e4, e4, table.long(), lens, sc, sc), (e4, e4, table[0], lens, sc, sc),
        (e4, e4, table, lens[:1], sc, sc), (e4, e4, table.t(), lens, sc, sc),
        (e4, e4, table, lens, sc[:4], sc), (e4, e4, table, lens, sc.double(), sc),
        (e4[0], e4[0], table, lens, sc, sc),
    ]
    for k, v, t, n, ks, vs in bad:
        with pytest.raises(ValueError):
            dfa.PagedCache(k, v, t, n, k_scale=ks, v_scale=vs)
    with pytest.raises(KeyError):
        dfa.rope_spec(64, layout="thirds")


def test_rope_refuses_what_fp32_cannot_hold(L):
    """A gain that is zero or infinite in fp32, frequencies that are not finite."""
    for kw in (dict(gain=1e-60), dict(gain=1e60), dict(scaling="linear", factor=1e-310),
               dict(scaling="bands", factor=1e-316, orig_len=512.0, low=1.0, high=4.0)):
        assert rope(L, spec(**kw)) == 1, kw
    assert decode(L, scale=3e38) == 1                         # times log2(e) is not finite


def test_a_cache_keeps_its_tensors():
    """Rebinding a cache's tensor would leave the calls with the old memory."""
    e4 = torch.zeros(8, 2, 16, 64).to(torch.bfloat16)
    table, lens = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    c = dfa.PagedCache(e4, e4, table, lens)
    with pytest.raises(AttributeError, match="contents"):
        c.seq_lens = lens + 1
    with pytest.raises(AttributeError, match="contents"):
        c.k = e4.clone()
    with pytest.raises(AttributeError, match="contents"):
        del c.block_table
    c.seq_lens += 1                                           # in place
    assert lens.tolist() == [1, 1] and c.desc.seq_lens == lens.data_ptr()


def test_plain_forms_of_the_tests():
    """The tests' own fp64 forms: rotation keeps lengths, its inverse undoes it,
    the two layouts are one map under a reordering, scales are tight."""
    import paged_ref as ref
    g = torch.Generator().manual_seed(1)
    x = torch.randn(3, 5, 64, generator=g, dtype=torch.float64)
    pos = torch.tensor([0, 1, 77, 1000, 123456])
    for layout in ("half", "interleaved"):
        y = ref.rope(x, pos, layout, 48)
        assert torch.allclose(y.norm(dim=-1), x.norm(dim=-1), rtol=1e-12)
        assert torch.allclose(ref.rope(y, pos, layout, 48, inverse=True), x, atol=1e-12)
    idx = torch.arange(48).view(2, 24).t().flatten()
    a = ref.rope(x[..., idx], pos, "interleaved", 48)
    b = ref.rope(x[..., :48], pos, "half", 48)[..., idx]
    assert torch.allclose(a, b, atol=1e-13)
    for amax in (0.0, 1.0, 448.0, 448.1, 1.75, 1.76, 1e-40, 1e38):
        s = ref.pow2_scale(amax)
        assert amax <= 448 * s and (s == 2.0 ** -100 or amax > 224 * s)
