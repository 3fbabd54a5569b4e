"""Trees over contexts of more tiles than a sum of products has before it is set apart: several
such sums to a block, with scores and values that rise within them, at their borders and
after them, both outputs."""
import pytest
import torch

import branch_ref as bref
import paged_ref as ref
from long_context_flashattention_gb300 import dfa
from test_gpu_tree import randn

pytestmark = pytest.mark.gpu
BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    dfa.lib()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("cells", [BF16, E4M3])
@pytest.mark.parametrize("G,T", [(1, 3), (8, 17)])
@pytest.mark.parametrize("rises", [[], [256], [100, 255, 257, 511, 513], [514], [1, 512]])
def test_contexts_of_many_chains(cells, G, T, rises):
    """550 tiles and a bit, of 80 sequences with two heads: a block has about one of them.
    Louder from those tiles on: scores by 6.5, or in 8 bits by 4 and values by 2^17."""
    L, d, page, copies = 550 * 128 + 77, 64, 128, 80
    c = ref.Cache(cells, 1, 2, d, page, -(-L // page), [L], seed=9)
    q = randn(1, 2 * G, T, d, seed=10)
    q[..., 0] = 32.0                                  # (scale 1/8)
    k = c.cells["k"].float()
    for p in range(c.table.shape[1]):
        at, up = int(c.table[0, p]), sum(p >= r for r in rises)
        k[at, :, :, 0] = 0.0
        if cells is E4M3:
            c.scales["k"][at] = 1 / 64
            k[at, :, :, 0] = 64.0 * up
            c.scales["v"][at] *= 2.0 ** (17 * up)
        else:
            k[at, :, :, 0] = 1.625 * up
    c.cells["k"] = k.to(cells)
    sees = bref.sees_of(bref.random_parents(1, T, seed=11))
    w = {f: 2.0 ** -11 if cells is E4M3 and not f else 2.0 ** -16 for f in (False, True)}
    want = {f: bref.attention(c, q, sees, weight=w[f]) for f in w}
    assert want[True][0].isfinite().all()
    c.B, c.table, c.lens = copies, c.table.repeat(copies, 1), c.lens.repeat(copies)
    dev, mask = c.cuda(), bref.pack(sees).repeat(copies, 1, 1).cuda()
    for f, (O, LSE, tO, tL) in want.items():
        o, lse = dfa.decode_tree(dev, q.repeat(copies, 1, 1, 1).cuda(), mask, out_fp32=f)
        many = lambda x: x.expand(copies, *x.shape[1:])  # noqa: E731
        ref.check(o, many(O), many(tO), torch.float32 if f else BF16, f)
        ref.check(lse, many(LSE), many(tL), torch.float32, f)
    dfa.stream_status(dev.status)
