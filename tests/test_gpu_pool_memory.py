"""What a page pool makes for itself outlives the calls on other streams that use it."""
import pytest
import torch

from long_context_flashattention_gb300 import dfa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    dfa.lib()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("named", [True, False])
@pytest.mark.parametrize("own_ws", [True, False])
def test_counts_of_a_pool_that_goes_while_a_call_waits(named, own_ws):
    """A call waits on its stream; its pool goes, and what is made next on the first stream
    stays as it was made."""
    B, npages = 9, 300
    table = torch.zeros(B, 6, dtype=torch.int32, device="cuda")
    lens = torch.full((B,), 20, dtype=torch.int32, device="cuda")
    pool = dfa.PagePool(table, lens, 16, npages=npages)
    ws = dfa.pages_workspace(pool) if own_ws else None
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(100_000_000)                  # some 50 ms
        jobs = torch.zeros(B * 3, 2, dtype=torch.int32, device="cuda")
        info = torch.zeros(4, dtype=torch.int32, device="cuda")
    kw = {"stream": s} if named else {}
    with torch.cuda.stream(torch.cuda.current_stream() if named else s):
        dfa.pages_reserve(pool, 20, jobs=jobs, info=info, ws=ws, **kw)
    del pool
    made = [torch.zeros(n, dtype=torch.int32, device="cuda") for n in (B, npages, 64) * 40]
    torch.cuda.synchronize()
    assert info.tolist() == [0, 2 * B, 0, 0] and int(table.max()) == 2 * B - 1
    assert all(int(t.abs().max()) == 0 for t in made)
