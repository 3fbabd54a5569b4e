"""Trees, kept rows and copies in pages that begin beyond 2^32 bytes (and elements) of the
cells: the same bits as in a cache of a few pages."""
import pytest
import torch

import branch_ref as bref
import paged_ref as ref
from long_context_flashattention_gb300 import dfa
from test_gpu_tree import i32, randn, some

pytestmark = pytest.mark.gpu
BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    dfa.lib()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


@pytest.mark.parametrize("cells", [BF16, E4M3])
@pytest.mark.parametrize("strided", [False, True])
def test_pages_beyond_32_bits(cells, strided):
    B, Hkv, G, T, d, page, width = 2, 2, 4, 20, 128, 64, 6
    lens = [350, 200]
    c = ref.Cache(cells, B, Hkv, d, page, width, lens, seed=1)
    near = c.cuda()
    # the same pages, far behind: one after the other, or far apart
    apart = (1 << 28) if strided else Hkv * page * d
    extra = (1 << 32) // apart + 1
    kw, far = {}, []
    for name in "kv":
        base = torch.empty((extra + c.npages) * apart, dtype=cells, device="cuda")
        x = base.view(-1, apart)[:, :Hkv * page * d].unflatten(1, (Hkv, page, d))
        x[extra:] = c.cells[name].cuda()
        far.append(x)
        if cells is E4M3:
            s = torch.ones(extra + c.npages, Hkv, device="cuda")
            s[extra:] = c.scales[name].cuda()
            kw[name + "_scale"] = s
    cache = dfa.PagedCache(*far, near.block_table + extra, near.seq_lens.clone(), **kw)
    assert extra * apart >= 1 << 32
    q = randn(B, Hkv * G, T, d, seed=2).cuda()
    k, v = (randn(B, Hkv, T, d, seed=3 + i).cuda() for i in range(2))
    parents = bref.random_parents(B, T, seed=5).cuda()
    kept = torch.stack([some(T, 7, b) for b in range(B)]).to(torch.int32).cuda()
    jobs = torch.tensor([[0, c.npages - 1], [1, c.npages - 2]], dtype=torch.int32, device="cuda")
    got = []
    for h, first in ((near, 0), (cache, extra)):
        out = []
        mask, pos = dfa.tree_plan(h, parents)
        qr = dfa.cache_append(h, k, v, rope=dfa.rope_spec(d), q=q, positions=pos)
        for fp32 in (False, True):
            out += dfa.decode_tree(h, qr, mask, out_fp32=fp32)
        dfa.cache_compact(h, kept, T=T)
        dfa.cache_copy(h, jobs + first, i32([2, 0, 0, 0]))
        dfa.stream_status(h.status)
        for t in (h.k, h.v):
            out.append(t[first:].contiguous().view(torch.uint8))
        got.append(out)
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert got[0][0].isfinite().all()
