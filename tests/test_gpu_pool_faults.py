"""Page pools whose numbers cannot be: each is reported, and its entry or sequence passed
over, so that later calls find the pool as it was."""
import pytest
import torch

from long_context_flashattention_gb300 import dfa
from test_gpu_pages import i32, new_pool, reserve, same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    dfa.lib()
    yield
    torch.cuda.synchronize()


def fresh(lens=(20, 30, 5)):
    pool, model = new_pool(3, 4, 20, 16)
    pool.seq_lens.copy_(i32(list(lens)))
    model.lens = list(lens)
    reserve(pool, model, list(lens), max(lens))
    return pool, model


def reported(pool):
    with pytest.raises(dfa.DfaError) as e:
        dfa.stream_status(pool.status)
    assert e.value.code == 6


@pytest.mark.parametrize("call", ["trim", "fork"])
@pytest.mark.parametrize("left", [0, -3])
def test_a_page_released_more_often_than_held_keeps_its_count(call, left):
    pool, model = fresh()
    pages = pool.block_table[0, :2].long()
    pool.refs[pages] = left
    refs = pool.refs.clone()
    if call == "trim":
        pool.seq_lens[0] = 0
        dfa.pages_trim(pool)
    else:
        dfa.pages_fork(pool, i32([-1, 1, 2]))
    reported(pool)
    assert torch.equal(pool.refs, refs) and int(pool.held[0]) == 0
    # what is free is free, and what is held afterwards is not
    pool.refs[pages] = 0
    model.pages[0], model.lens[0] = [], 40
    pool.seq_lens[0] = 40
    reserve(pool, model, [40, 0, 0], 40)
    same(pool, model)
    dfa.stream_status(pool.status)


def test_releases_of_one_page_by_many_stop_at_nothing():
    """Forty sequences give back a page that counts three holders."""
    B = 40
    pool, model = new_pool(B, 2, 50, 16)
    pool.seq_lens.copy_(i32([16] + [0] * (B - 1)))
    model.lens = [16] + [0] * (B - 1)
    reserve(pool, model, model.lens, 16)
    dfa.pages_fork(pool, i32([0] * B))
    page = int(pool.block_table[0, 0])
    assert int(pool.refs[page]) == B
    pool.refs[page] = 3
    pool.seq_lens.zero_()
    dfa.pages_trim(pool)
    reported(pool)
    assert int(pool.refs.abs().sum()) == 0 and int(pool.held.sum()) == 0


@pytest.mark.parametrize("n", [65, 66, 2 ** 31 - 1, -1, -2 ** 31])
def test_trim_reports_a_length(n):
    pool, model = fresh()
    before = [x.clone() for x in (pool.block_table, pool.held, pool.refs)]
    pool.seq_lens[1] = n
    dfa.pages_trim(pool)
    reported(pool)
    assert all(torch.equal(a, b) for a, b in zip(before, (pool.block_table, pool.held, pool.refs)))
    pool.seq_lens[1] = 64                       # all that a sequence can have: no fault
    dfa.pages_trim(pool)
    dfa.stream_status(pool.status)


@pytest.mark.parametrize("B,width", [(3, 4), (40, 4), (3, 1100)])      # one launch, or two
@pytest.mark.parametrize("n", [-1, -2 ** 31, 65, 2 ** 31 - 1])
def test_fork_reports_the_length_of_a_source(B, width, n):
    pool, model = new_pool(B, width, 3 * B, 16)
    lens = [20] * B
    pool.seq_lens.copy_(i32(lens))
    model.lens = lens
    reserve(pool, model, lens, 20)
    if n == 65:
        n = 16 * width + 1
    pool.seq_lens[1] = n
    model.lens[1] = n
    dfa.pages_fork(pool, i32([1, 1] + list(range(2, B))))
    reported(pool)
    same(pool, model)                           # sequence 0 stays
    dfa.pages_fork(pool, i32([0, 0] + list(range(2, B))))
    model.fork([0, 0] + list(range(2, B)))      # a good one takes the other's place
    same(pool, model)
    dfa.stream_status(pool.status)
