"""CPU checks of the calls around branching sequences: the C entries refuse bad arguments
before any device work, the binding refuses tensors that the calls do not take, and the
plain forms of the tests agree with one another."""
import ctypes

import pytest
import torch

import branch_ref as bref
import paged_ref as ref
from long_context_flashattention_gb300 import dfa

_BUF = (ctypes.c_uint8 * (1 << 16))()
BASE = (ctypes.addressof(_BUF) + 255) & ~255
FAR = BASE + (1 << 14)
END = BASE + (1 << 15)
I3 = ctypes.c_int64 * 3


@pytest.fixture(scope="module")
def L():
    return dfa.lib()


def cache(**kw):
    c = dict(dtype=1, page=16, Hkv=2, d=64, npages=8, page_stride=0, k=BASE, v=BASE,
             k_scale=BASE, v_scale=BASE, B=2, max_pages=4, block_table=BASE, seq_lens=BASE)
    return dfa.PagedCacheDesc(**{**c, **kw})


def plan(L, c=None, T=4, parents=BASE, mask=FAR, pos=END, ws=BASE, n=256):
    return L.dfa_tree_plan(None if c is False else ctypes.byref(c or cache()), T, None, parents,
                           mask, pos, ws, n, None)


def tree(L, c=None, T=4, mask=BASE, q=BASE, qs=None, o=FAR, lse=END, ws=BASE, n=1 << 40,
         desc=None, **kw):
    if desc is None:
        desc = dfa.make_desc(**{**dict(B=2, Hq=4, Hkv=2, N=1, d=64), **kw})
    return L.dfa_decode_tree(ctypes.byref(desc), None if c is False else ctypes.byref(c or cache()),
                             T, None, mask, q, qs, o, lse, ws, n, None)


def compact(L, c=None, T=8, A=4, kept=BASE, ws=BASE, n=256):
    return L.dfa_cache_compact(None if c is False else ctypes.byref(c or cache()), T, None, A,
                               kept, None, ws, n, None)


def copy(L, c=None, jobs=BASE, J=4, info=BASE, ws=BASE, n=256):
    return L.dfa_cache_copy(None if c is False else ctypes.byref(c or cache()), jobs, J, info, ws,
                            n, None)


def append_at(L, c=None, pos=BASE, spec=True, T=4, k=BASE, v=BASE, ws=BASE, n=256):
    s = dfa.rope_spec(64)
    return L.dfa_cache_append_at(ctypes.byref(c or cache()), ctypes.byref(s) if spec else None, T,
                                 None, pos, k, None, v, None, 0, None, None, None, None, ws, n,
                                 None)


CACHE_BAD = [(dict(dtype=2), 1), (dict(d=96), 2), (dict(page=8), 2), (dict(page=48), 2),
             (dict(Hkv=0), 1), (dict(B=0), 1), (dict(max_pages=0), 1),
             (dict(max_pages=1 << 27), 1), (dict(npages=0), 1), (dict(npages=1 << 31), 1),
             (dict(page_stride=100), 1), (dict(page_stride=2 * 16 * 64 + 8), 2),
             (dict(k=None), 1), (dict(v=None), 1), (dict(k_scale=None), 1),
             (dict(v_scale=None), 1), (dict(block_table=None), 1), (dict(seq_lens=None), 1),
             (dict(k=BASE + 8), 2), (dict(v=BASE + 1), 2), (dict(status=BASE + 16), 1)]


@pytest.mark.parametrize("kw,code", CACHE_BAD)
def test_every_call_refuses_a_bad_cache(L, kw, code):
    for call in (plan, tree, compact, copy, append_at):
        assert call(L, cache(**kw)) == code and L.dfa_last_error(), call.__name__
    for call in (plan, tree, compact, copy):
        assert call(L, False) == 1


def test_plan_refuses(L):
    for kw, code in ((dict(T=0), 1), (dict(T=1025), 2), (dict(parents=None), 1),
                     (dict(mask=None), 1), (dict(pos=None), 1), (dict(ws=None), 3),
                     (dict(n=255), 3), (dict(ws=BASE + 16), 3), (dict(mask=BASE), 1),
                     (dict(mask=BASE + 28), 1), (dict(pos=BASE + 4), 1), (dict(pos=FAR), 1)):
        assert plan(L, **kw) == code, kw


def test_tree_refuses(L):
    for kw, code in ((dict(T=0), 1), (dict(T=513), 2), (dict(Hq=3), 1), (dict(B=3), 1),
                     (dict(Hkv=4), 1), (dict(d=128), 1), (dict(scale=0.0), 1),
                     (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1), (dict(scale=3e38), 1),
                     (dict(q=None), 1), (dict(q=BASE + 2), 2), (dict(qs=I3(1024, 64, 60)), 2),
                     (dict(qs=I3(1024, -64, 64)), 1), (dict(mask=None), 1), (dict(o=None), 1),
                     (dict(lse=None), 1), (dict(o=FAR + 8), 2), (dict(ws=None), 3),
                     (dict(n=100), 3), (dict(ws=BASE + 64), 3)):
        assert tree(L, **kw) == code, kw
    # outputs on top of one another or of what the call reads
    span = 2 * 4 * 4 * 64 * 2
    for kw in (dict(o=BASE), dict(o=BASE + span - 16), dict(lse=BASE), dict(lse=FAR + span - 4),
               dict(mask=END, o=END), dict(mask=END), dict(mask=FAR + span - 4)):
        assert tree(L, **kw) == 1 and b"overlap" in L.dfa_last_error(), kw
    desc = dfa.make_desc(2, 4, 2, 1, 64)
    desc.ndocs, desc.doc_bounds = 1, BASE
    assert tree(L, desc=desc) == 2
    desc = dfa.make_desc(2, 4, 2, 1, 64)
    desc.o_fp32 = 3
    assert tree(L, desc=desc) == 1
    assert L.dfa_decode_tree(None, ctypes.byref(cache()), 1, None, BASE, BASE, None, FAR, END,
                             BASE, 1 << 40, None) == 1


def test_tree_workspace_size(L):
    def size(T, **kw):
        desc = dfa.make_desc(**{**dict(B=2, Hq=4, Hkv=2, N=1, d=64), **kw})
        return L.dfa_decode_tree_workspace_size(ctypes.byref(desc), T)
    assert size(1) >= 256 and size(1, B=1000) == size(1)   # whatever the batch
    assert size(0) == 0 and size(513) == 0 and size(1, d=96) == 0 and size(1, Hq=3) == 0
    assert L.dfa_decode_tree_workspace_size(None, 1) == 0


def test_append_at_refuses(L):
    for kw, code in ((dict(pos=None), 1), (dict(spec=False), 1), (dict(T=0), 1), (dict(k=None), 1),
                     (dict(v=BASE + 2), 2), (dict(ws=None), 3)):
        assert append_at(L, **kw) == code, kw


def test_compact_refuses(L):
    for kw, code in ((dict(T=0), 1), (dict(T=1 << 30), 1), (dict(A=0), 1), (dict(A=9), 1),
                     (dict(kept=None), 1), (dict(ws=None), 3), (dict(n=255), 3),
                     (dict(c=cache(B=1 << 20, Hkv=2048)), 2)):
        assert compact(L, **kw) == code, kw


def test_copy_refuses(L):
    for kw, code in ((dict(J=0), 1), (dict(J=1 << 30), 1), (dict(jobs=None), 1),
                     (dict(info=None), 1), (dict(jobs=BASE + 4), 2), (dict(ws=None), 3),
                     (dict(n=255), 3)):
        assert copy(L, **kw) == code, kw


def pool(**kw):
    p = dict(page=16, B=2, max_pages=4, npages=8, block_table=BASE, held=BASE, refs=BASE,
             seq_lens=BASE)
    return dfa.PagePoolDesc(**{**p, **kw})


def fork(L, p=None, src=BASE, ws=BASE, n=1 << 40):
    return L.dfa_pages_fork(None if p is False else ctypes.byref(p or pool()), src, ws, n, None)


def reserve(L, p=None, T=4, jobs=BASE, J=4, info=BASE, ws=BASE, n=1 << 40):
    return L.dfa_pages_reserve(None if p is False else ctypes.byref(p or pool()), T, None, jobs, J,
                               info, ws, n, None)


def trim(L, p=None, ws=BASE, n=256):
    return L.dfa_pages_trim(None if p is False else ctypes.byref(p or pool()), ws, n, None)


POOL_BAD = [(dict(page=8), 2), (dict(page=0), 2), (dict(B=0), 1), (dict(B=(1 << 20) + 1), 1),
            (dict(max_pages=0), 1), (dict(max_pages=1 << 27), 1),
            (dict(B=1 << 20, max_pages=1 << 11), 1), (dict(npages=0), 1), (dict(npages=1 << 31), 1),
            (dict(block_table=None), 1), (dict(held=None), 1), (dict(refs=None), 1),
            (dict(seq_lens=None), 1), (dict(status=BASE + 8), 1)]


@pytest.mark.parametrize("kw,code", POOL_BAD)
def test_every_call_refuses_a_bad_pool(L, kw, code):
    for call in (fork, reserve, trim):
        assert call(L, pool(**kw)) == code and L.dfa_last_error(), call.__name__
        assert call(L, False) == 1


def test_pool_calls_refuse(L):
    need = L.dfa_pages_workspace_size(ctypes.byref(pool()))
    assert need > 256 and L.dfa_pages_workspace_size(None) == 0
    assert L.dfa_pages_workspace_size(ctypes.byref(pool(B=0))) == 0
    for kw, code in ((dict(src=None), 1), (dict(ws=None), 3), (dict(n=256), 3),
                     (dict(ws=BASE + 8), 3)):
        assert fork(L, **kw) == code, kw
    for kw, code in ((dict(T=-1), 1), (dict(T=1 << 30), 1), (dict(jobs=None), 1),
                     (dict(J=-1), 1), (dict(info=None), 1), (dict(jobs=BASE + 4), 2),
                     (dict(ws=None), 3), (dict(n=256), 3)):
        assert reserve(L, **kw) == code, kw
    for kw, code in ((dict(ws=None), 3), (dict(n=255), 3)):
        assert trim(L, **kw) == code, kw


def test_binding_refuses():
    """Host tensors, wrong dtypes, shapes and strides, before any device work."""
    kv = torch.zeros(8, 2, 16, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    c = dfa.PagedCache(kv, kv.clone(), table, lens)
    p = dfa.PagePool(table, lens, 16, npages=8)
    q = torch.zeros(2, 4, 3, 64, dtype=torch.bfloat16)
    ints = torch.zeros(2, 3, dtype=torch.int32)
    for call in (lambda: dfa.tree_plan(c, ints), lambda: dfa.decode_tree(c, q, ints),
                 lambda: dfa.cache_compact(c, ints, T=3), lambda: dfa.cache_copy(c, ints, lens),
                 lambda: dfa.pages_fork(p, lens), lambda: dfa.pages_reserve(p, 1),
                 lambda: dfa.pages_trim(p)):
        with pytest.raises(ValueError, match="device"):
            call()
    for kw in (dict(), dict(held=lens), dict(refs=lens), dict(held=lens, refs=lens, npages=2),
               dict(held=lens[:1], refs=lens), dict(held=lens.long(), refs=lens),
               dict(held=lens, refs=lens[None])):
        with pytest.raises(ValueError):
            dfa.PagePool(table, lens, 16, **kw)
    with pytest.raises(ValueError):
        dfa.PagePool(table[0], lens, 16, npages=8)
    with pytest.raises(ValueError):
        dfa.PagePool(table, lens[:1], 16, npages=8)
    with pytest.raises(AttributeError, match="contents"):
        p.refs = lens
    with pytest.raises(AttributeError, match="contents"):
        del p.held
    assert p.npages == 8 and p.status.numel() == 256 and not p.desc.status


def test_plain_forms_of_the_tests():
    """Masks by parents and by their closure; a model pool that conserves its pages; a
    compacted cache whose rows are the kept ones."""
    parents = bref.random_parents(3, 50, seed=1)
    sees = bref.sees_of(parents)
    step = torch.zeros(3, 50, 50, dtype=torch.bool)
    for b in range(3):
        for t in range(50):
            if parents[b, t] >= 0:
                step[b, t, int(parents[b, t])] = True
    closure = torch.eye(50, dtype=torch.bool).repeat(3, 1, 1)
    for _ in range(50):
        closure = closure | (step.float() @ closure.float() > 0)
    assert torch.equal(sees, closure)
    words = bref.pack(sees)
    assert words.shape == (3, 50, 2)
    for t in (0, 31, 32, 49):
        assert torch.equal((words[:, :, t // 32].long() >> (t % 32)) & 1, sees[:, :, t].long())
    m = bref.Pool(3, 4, 9, 16)
    m.lens = [40, 0, 1]
    assert m.reserve([40, 0, 1]) == ([], 4, 0) and m.pages == [[0, 1, 2], [], [3]]
    m.fork([0, 0, 2])
    m.lens = [41, 41, 2]
    assert m.reserve([1, 1, 1]) == ([[2, 4]], 1, 0)
    assert m.pages == [[0, 1, 4], [0, 1, 2], [3]] and sum(m.refs()) == 7
    m.lens = [0, 20, 2]
    m.trim()
    assert m.pages == [[], [0, 1], [3]]
    c = ref.Cache(torch.bfloat16, 1, 1, 64, 16, 3, [40], seed=2)
    kept = torch.tensor([[1, 2, 9, 20, 29]], dtype=torch.int32)
    want = bref.rows(c, "k", 0, 40)[:, [*range(10), 11, 12, 19, 30, 39]]
    c.cells["k"] = bref.compact(c, kept, [5], [30])["k"][0].to(torch.bfloat16)
    assert torch.equal(bref.rows(c, "k", 0, 15), want)
