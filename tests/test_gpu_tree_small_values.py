"""Trees in 8 bits over value scales down to fp32's smallest normal number, and larger ones
behind them: the weights' common exponent is then far below that of ordinary values."""
import pytest
import torch

import branch_ref as bref
import paged_ref as ref
from long_context_flashattention_gb300 import dfa
from test_gpu_tree import check_tree, randn

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    dfa.lib()
    yield
    torch.cuda.synchronize()


# rows a head: up to 64, more
@pytest.mark.parametrize("G", [1, 4])
@pytest.mark.parametrize("small", [[1], [0, 1]])
@pytest.mark.parametrize("d", [64, 128])
def test_nothing_seen_behind_tiny_values(G, small, d):
    """Pages of 64 rows, two to a tile: tiny values in the first tile's second page (or in
    both), then a tile that ends before its second page."""
    T = 16
    c = ref.Cache(E4M3, 1, 1, d, 64, 4, [128 + 40], seed=1)
    for p in small:
        c.scales["v"][int(c.table[0, p])] = 2.0 ** -126
    q = randn(1, G, T, d, seed=2)
    check_tree(c, c.cuda(), q, bref.sees_of(bref.random_parents(1, T, seed=3)))


@pytest.mark.parametrize("G", [1, 2])
@pytest.mark.parametrize("up", [0, 20])
def test_hidden_nodes_behind_tiny_values(G, up):
    """The second tile's second page is the tree, whose nodes see nothing of it, or some."""
    T = 64
    c = ref.Cache(E4M3, 1, 1, 64, 64, 4, [256], seed=4)
    c.scales["v"][int(c.table[0, 1])] = 2.0 ** -126
    c.scales["v"][int(c.table[0, 3])] = 2.0 ** up
    q = randn(1, G, T, 64, seed=5)
    sees = torch.zeros(1, T, T, dtype=torch.bool)
    check_tree(c, c.cuda(), q, sees)
    check_tree(c, c.cuda(), q, sees | (torch.arange(T) % 2 == 0)[:, None] & torch.eye(T).bool())


@pytest.mark.parametrize("G", [1, 40])
@pytest.mark.parametrize("below", [96.0, 104.0])
def test_far_larger_values_at_far_lower_scores(G, below):
    """Values of 2^40 with weights of e^-104 are what counts beside values of 2^-126: the
    powers of two of the scores alone are below fp32's range."""
    T, d = 2, 64
    c = ref.Cache(E4M3, 1, 1, d, 64, 4, [250], seed=6)
    c.scales["k"][:] = 1.0
    k = torch.zeros_like(c.cells["k"].float())
    for p in range(4):
        k[int(c.table[0, p]), 0, :, 0] = 0.0 if p < 2 else -below
        c.scales["v"][int(c.table[0, p])] = 2.0 ** -126 if p < 2 else 2.0 ** 40
    # (the nodes among the last rows)
    c.cells["k"] = k.to(E4M3)
    q = torch.zeros(1, G, T, d, dtype=torch.bfloat16)
    q[..., 0] = 1.0
    check_tree(c, c.cuda(), q, bref.sees_of(bref.random_parents(1, T, seed=7)), scale=1.0)
