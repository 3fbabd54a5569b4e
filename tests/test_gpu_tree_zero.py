"""Trees in 8 bits whose score factors underflow: queries of zeros over pages of zeros, which
have the smallest scale, with keys in those pages that a node does not see.  Every score
is 0 then, so that what is seen has equal weights."""
import math

import pytest
import torch

import branch_ref as bref
import paged_ref as ref
from long_context_flashattention_gb300 import dfa
from test_gpu_tree import check_tree, randn

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn
# rows a head: a few (one term beside half of the keys, or two in the operand's rows), and
# more than 64
ROWS = [(2, 9), (8, 17)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    dfa.lib()
    yield
    torch.cuda.synchronize()


def zero_pages(c, names, pages, scale=2.0 ** -100):
    for name in names:
        x = c.cells[name].float()
        for b in range(c.B):
            for p in pages:
                x[int(c.table[b, p])] = 0.0
                c.scales[name][int(c.table[b, p])] = scale
        c.cells[name] = x.to(E4M3)


@pytest.mark.parametrize("G,T", ROWS)
@pytest.mark.parametrize("names", ["k", "kv"])       # (the values' scale, too: far from others)
@pytest.mark.parametrize("zeros", ["all", "some"])
@pytest.mark.parametrize("d", [64, 128])
def test_zero_queries_over_zero_pages(G, T, names, zeros, d):
    """The sequence's end and hidden nodes lie in pages of zeros; rows of queries without a
    nonzero element, all or every other one."""
    lens = [150, 64 + T, 203]
    c = ref.Cache(E4M3, 3, 1, d, 16, 13, lens, seed=1 + T)
    q = randn(3, G, T, d, seed=2)
    if zeros == "all":
        q.zero_()
    else:
        q[:, :, ::2] = 0
    # from the page that the tree begins in on
    for b, L in enumerate(lens):
        for name in names:
            x = c.cells[name].float()
            for p in range((L - T) // 16, -(-L // 16)):
                x[int(c.table[b, p])] = 0.0
                c.scales[name][int(c.table[b, p])] = 2.0 ** -100
            c.cells[name] = x.to(E4M3)
    sees = bref.sees_of(bref.random_parents(3, T, seed=3))
    check_tree(c, c.cuda(), q, sees)


@pytest.mark.parametrize("G,T", ROWS)
@pytest.mark.parametrize("tiny", [2.0 ** -33, 2.0 ** -60, 2.0 ** -126])
def test_factors_next_to_the_smallest(G, T, tiny):
    """Key scales down to fp32's smallest, under queries of zeros and of tiny numbers."""
    c = ref.Cache(E4M3, 2, 1, 64, 16, 10, [150, 40], seed=4)
    c.scales["k"][:] = tiny
    sees = bref.sees_of(bref.random_parents(2, T, seed=5))
    for size in (0.0, 2.0 ** -90, 1.0):
        check_tree(c, c.cuda(), randn(2, G, T, 64, seed=6) * size, sees)


@pytest.mark.parametrize("fp32", [False, True])
def test_a_step_of_zeros(fp32):
    """What a warm-up or a padded slot computes: zeros appended and attended to."""
    B, Hkv, G, T, d, page = 2, 2, 4, 12, 128, 16
    k, v = (torch.zeros(8, Hkv, page, d, device="cuda").to(E4M3) for _ in "kv")
    ks, vs = (torch.ones(8, Hkv, device="cuda") for _ in "kv")
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(B, 4)
    cache = dfa.PagedCache(k, v, table, torch.full((B,), T, dtype=torch.int32, device="cuda"),
                           k_scale=ks, v_scale=vs)
    x = torch.zeros(B, Hkv, T, d, dtype=torch.bfloat16, device="cuda")
    parents = torch.full((B, T), -1, dtype=torch.int32)     # no node sees another
    mask, pos = dfa.tree_plan(cache, parents.cuda())
    q = dfa.cache_append(cache, x, x, rope=dfa.rope_spec(d), q=x.repeat(1, G, 1, 1), positions=pos)
    o, lse = dfa.decode_tree(cache, q, mask, out_fp32=fp32)
    assert (o == 0).all() and (lse == 0).all()              # one key each, of score 0
    parents = (torch.arange(T, dtype=torch.int32) - 1).repeat(B, 1)
    mask, _ = dfa.tree_plan(cache, parents.cuda())
    o, lse = dfa.decode_tree(cache, q, mask, out_fp32=fp32)
    want = torch.arange(1, T + 1).double().log()
    # the logarithm to 2^-22 of itself, times ln 2 in fp32
    assert (o == 0).all() and (lse.cpu().double() - want).abs().max() <= 2.0 ** -21 * math.log(T)
    dfa.stream_status(cache.status)
