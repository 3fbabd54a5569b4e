"""The steps of the usage notes, run as they stand there, with a pool that has too few pages:
nothing that other sequences hold is written, and the step after it goes on."""
import os
import re
import textwrap

import pytest
import torch

import branch_ref as bref
from long_context_flashattention_gb300 import dfa

pytestmark = pytest.mark.gpu
BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn
NOTES = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    dfa.lib()
    yield
    torch.cuda.synchronize()


def step(which):
    """The code of a step in the usage notes: from its comment to the next step's."""
    text = open(NOTES).read()
    block = re.search(r"### Trees of drafted tokens, beams\n+```python\n(.*?)```", text, re.S)[1]
    parts = re.split(r"^# one step of ", block, flags=re.M)
    return compile(textwrap.dedent("# " + next(p for p in parts if p.startswith(which))), NOTES,
                   "exec")


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class State:
    """Two sequences in a full pool of four pages.  Sequence 0 has been longer: the third
    entry of its row of the table still names a page that sequence 1 has got since."""

    def __init__(self, dtype, npages=4, spare=0):
        B, Hkv, d, page, width = 2, 2, 64, 16, 8
        g = torch.Generator().manual_seed(1)
        cells = [torch.randn(npages, Hkv, page, d, generator=g).to(dtype).cuda() for _ in "kv"]
        kw = {}
        if dtype is E4M3:
            kw = {n: torch.full((npages, Hkv), 0.5, device="cuda") for n in ("k_scale", "v_scale")}
        self.table = torch.zeros(B, width, dtype=torch.int32, device="cuda")
        self.lens = i32([33, 0])
        self.pool = dfa.PagePool(self.table, self.lens, page, npages=npages)
        self.cache = dfa.PagedCache(*cells, self.table, self.lens, **kw)
        dfa.pages_reserve(self.pool, 33, new_lens=i32([33, 0]))
        self.lens.copy_(i32([30, 0]))
        dfa.pages_trim(self.pool)
        self.lens.copy_(i32([30, 20]))
        dfa.pages_reserve(self.pool, 20, new_lens=i32([0, 20]))
        assert self.table[0, 2] == self.table[1, 0] and self.pool.held.tolist() == [2, 2]
        dfa.stream_status(self.pool.status)
        T = 16
        x = lambda h, s: torch.randn(B, h, T, d, generator=g).to(BF16).cuda()  # noqa: E731
        self.names = dict(dfa=dfa, torch=torch, B=B, T=T, cache=self.cache, pool=self.pool,
                          lens=self.lens, page=page, npages=npages, Hq=4,
                          rope=dfa.rope_spec(d, layout="half"), ws=dfa.tree_workspace(self.cache, 4, T),
                          parents=bref.random_parents(B, T, seed=2).cuda(), k_new=x(Hkv, 0),
                          v_new=x(Hkv, 0), q=x(4, 0), kept=i32([[1, 2, 5], [0, 3, 4]]),
                          kept_lens=i32([3, 2]), src=i32([0, 0]))

    def all(self):
        c, p = self.cache, self.pool
        t = [c.k, c.v, p.block_table, p.held, p.refs, p.seq_lens]
        if c.k_scale is not None:
            t += [c.k_scale, c.v_scale]
        return [x.contiguous().view(torch.uint8).clone() for x in t]


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("dtype", [E4M3, BF16])
def test_a_refused_step_of_drafted_tokens_changes_nothing(dtype, captured):
    s = State(dtype)
    code = step("speculative decoding")
    was = s.all()
    if captured:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            exec(code, s.names)
        g.replay()
    else:
        exec(code, s.names)
    torch.cuda.synchronize()
    assert s.names["info"].tolist()[2] == 1
    with pytest.raises(dfa.DfaError):
        dfa.stream_status(s.pool.status)
    dfa.stream_status(s.names["ws"])
    dfa.stream_status(s.cache.status)
    for a, b in zip(was, s.all()):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [E4M3, BF16])
def test_a_step_of_drafted_tokens_with_pages_enough(dtype):
    """The same code where nothing is refused: the kept rows are there."""
    s = State(dtype, npages=8)
    exec(step("speculative decoding"), s.names)
    torch.cuda.synchronize()
    assert s.names["info"].tolist()[2] == 0
    assert s.lens.tolist() == [33, 22] and s.pool.held.tolist() == [3, 2]
    o, lse = s.names["o"], s.names["lse"]
    assert o.isfinite().all() and lse.isfinite().all()
    for st in (s.pool.status, s.names["ws"], s.cache.status):
        dfa.stream_status(st)


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("dtype", [E4M3, BF16])
def test_a_refused_step_of_beams_writes_no_row(dtype, captured):
    """Both beams go on from one, whose last page both would write to; no page is free."""
    s = State(dtype, npages=4)
    # as many holders for two more pages as keeps them from being free
    s.lens[1] = 0
    dfa.pages_trim(s.pool)                              # sequence 0 alone: two pages of four
    s.pool.refs[:] = s.pool.refs.clamp(min=1)
    s.names.update(k_new=s.names["k_new"][:, :, :1], v_new=s.names["v_new"][:, :, :1],
                   q=s.names["q"][:, :, :1])
    code = step("beam search")
    cells = s.all()[:2] + s.all()[6:]
    if captured:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            exec(code, s.names)
        g.replay()
    else:
        exec(code, s.names)
    torch.cuda.synchronize()
    assert s.names["info"].tolist()[2] == 1
    with pytest.raises(dfa.DfaError):
        dfa.stream_status(s.pool.status)
    dfa.stream_status(s.cache.status)
    assert s.lens.tolist() == [30, 30]                  # forked, and no row longer
    for a, b in zip(cells, s.all()[:2] + s.all()[6:]):
        assert torch.equal(a, b)
