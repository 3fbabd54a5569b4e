"""Trees over bf16 cells with values far from 1 behind scores that rise: weights relative to an
early reference do not carry large values out of fp32's range, nor small ones."""
import pytest
import torch

import branch_ref as bref
import paged_ref as ref
from long_context_flashattention_gb300 import dfa
from test_gpu_tree import check_tree

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    dfa.lib()
    yield
    torch.cuda.synchronize()


def check_rising(L, d, page, gain, scores, G, T, copies, seed):
    """A context whose key j has the score scores(j) under a query of ones in feature 0, and
    values of size `gain`; `copies` sequences of it, so that blocks have more or fewer of
    its tiles, against one plain form."""
    c = ref.Cache(BF16, 1, 2, d, page, -(-L // page), [L], seed=seed)
    k = torch.zeros_like(c.cells["k"].float())
    for j in range(L):
        k[int(c.table[0, j // page]), :, j % page, 0] = scores(j)
    c.cells["k"] = k.to(BF16)
    c.cells["v"] = (c.cells["v"].float() * gain).to(BF16)
    q = torch.zeros(1, 2 * G, T, d, dtype=BF16)
    q[..., 0] = 1.0
    sees = bref.sees_of(bref.random_parents(1, T, seed=seed + 1))
    O, LSE, tO, tL = bref.attention(c, q, sees, scale=1.0, weight=2.0 ** -16)
    c.table, c.lens = c.table.repeat(copies, 1), c.lens.repeat(copies)
    dev, mask = c.cuda(), bref.pack(sees).repeat(copies, 1, 1).cuda()
    for fp32 in (False, True):
        o, lse = dfa.decode_tree(dev, q.repeat(copies, 1, 1, 1).cuda(), mask, scale=1.0,
                                 out_fp32=fp32)
        many = lambda x: x.expand(copies, *x.shape[1:])  # noqa: E731
        ref.check(o, many(O), many(tO), torch.float32 if fp32 else BF16, fp32)
        ref.check(lse, many(LSE), many(tL), torch.float32, fp32)
    dfa.stream_status(dev.status)


# up to 64 rows a head and more; a tile or two to a block, all of a sequence's
@pytest.mark.parametrize("G,T", [(1, 3), (8, 17)])
@pytest.mark.parametrize("copies", [1, 150])
@pytest.mark.parametrize("gain", [2.0 ** 66, 2.0 ** 100, 2.0 ** 106, 2.0 ** -110])
@pytest.mark.parametrize("step,d", [(3.0, 64), (5.5, 128), (20.0, 64), (41.0, 128), (60.0, 64)])
def test_values_behind_rising_scores(G, T, copies, gain, step, d):
    """Scores go up by `step` from one tile to the next: below, at and above what the
    reference is left behind by.  (700 rows of 2^106 times 6: 2^118, below the 2^120 that
    they may be.)"""
    check_rising(700, d, 64, gain, lambda j: step * (j // 128), G, T, copies, seed=1)


@pytest.mark.parametrize("G,T", [(1, 3), (8, 17)])
@pytest.mark.parametrize("L,copies", [(500, 1), (500, 150), (20000, 1), (5000, 40)])
@pytest.mark.parametrize("above", [5.0, 41.0])
def test_one_late_key_of_large_values(G, T, L, copies, above):
    """A single key far above all others, in the last tile but one and in the first."""
    for late in (L - 200, 70):
        check_rising(L, 64, 128, 2.0 ** 100, lambda j: above if j == late else 0.0, G, T, copies,
                     seed=3)


@pytest.mark.parametrize("G,T", [(4, 2), (8, 17)])
def test_rises_over_chains(G, T):
    """More than 40 tiles to a block and scores that rise before and after a sum is set
    apart, fp32 outputs, large values."""
    B, Hkv, d, page, L = 20, 8, 64, 64, 5900
    c = ref.Cache(BF16, 1, Hkv, d, page, -(-L // page), [L], seed=5)
    k = c.cells["k"].float()
    for p in range(c.table.shape[1]):
        k[int(c.table[0, p]), :, :, 0] = 6.0 * (p // 20)
    c.cells["k"] = k.to(BF16)
    c.cells["v"] = (c.cells["v"].float() * 2.0 ** 98).to(BF16)
    lens = [L - 31 * b for b in range(B)]
    c.B, c.table, c.lens = B, c.table.repeat(B, 1), torch.tensor(lens, dtype=torch.int32)
    g = torch.Generator().manual_seed(6)
    q = torch.randn(B, Hkv * G, T, d, generator=g)
    q[..., 0] = 8.0                         # scale 1/8: a score of 6 every 20 pages
    check_tree(c, c.cuda(), q.to(BF16), bref.sees_of(bref.random_parents(B, T, seed=7)),
               fp32=(True,))
