"""GPU parity of the page pool (fork, reserve, trim) and of copied pages against a plain
model that goes page by page: what is held, how many hold it, which free pages are taken,
what is copied; refusals on the device; graphs."""
import random

import pytest
import torch

import branch_ref as bref
from long_context_flashattention_gb300 import dfa

pytestmark = pytest.mark.gpu
BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    dfa.lib()
    yield
    torch.cuda.synchronize()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def new_pool(B, width, npages, page):
    return (dfa.PagePool(torch.full((B, width), -1, dtype=torch.int32, device="cuda"),
                         torch.zeros(B, dtype=torch.int32, device="cuda"), page, npages=npages),
            bref.Pool(B, width, npages, page))


def same(pool, model):
    assert pool.held.tolist() == [len(p) for p in model.pages]
    assert pool.refs.tolist() == model.refs()
    assert pool.seq_lens.tolist() == model.lens
    table = pool.block_table.tolist()
    for b, p in enumerate(model.pages):
        assert table[b][:len(p)] == p


def reserve(pool, model, new, T, ws=None, max_jobs=None):
    kw = {}
    if max_jobs is not None:
        kw["jobs"] = torch.full((max_jobs, 2), -7, dtype=torch.int32, device="cuda")
    jobs, info = dfa.pages_reserve(pool, T, new_lens=i32(new), ws=ws, **kw)
    want, taken, refused = model.reserve(new, jobs.shape[0])
    assert info.tolist() == [len(want), taken, refused, 0]
    assert jobs[:len(want)].tolist() == want
    return jobs, info, refused


@pytest.mark.parametrize("B,width,npages,page", [(1, 1, 1, 16), (3, 8, 40, 16), (17, 5, 200, 128),
                                                 (64, 40, 5000, 32), (1100, 4, 9000, 64)])
def test_pool_over_many_steps(B, width, npages, page):
    """Sequences grow, fork, shrink and end at random; the pool and the model agree after
    every call."""
    rng = random.Random(B)
    pool, model = new_pool(B, width, npages, page)
    ws = dfa.pages_workspace(pool)
    for step in range(12):
        T = rng.choice((1, 1, 7, page, 3 * page))
        new = [rng.randint(0, min(T, width * page - n)) if rng.random() < 0.8 else 0
               for n in model.lens]
        model.lens = [n + m for n, m in zip(model.lens, new)]
        pool.seq_lens += i32(new)
        if reserve(pool, model, new, T, ws)[2]:
            with pytest.raises(dfa.DfaError):
                dfa.stream_status(ws)
            model.lens = [n - m for n, m in zip(model.lens, new)]
            pool.seq_lens -= i32(new)
        same(pool, model)
        if rng.random() < 0.7:
            src = [b if rng.random() < 0.5 else rng.choice((-1, rng.randrange(B)))
                   for b in range(B)]
            dfa.pages_fork(pool, i32(src), ws=ws)
            model.fork(src)
            same(pool, model)
        if rng.random() < 0.5:
            model.lens = [rng.randint(0, n) if rng.random() < 0.5 else n for n in model.lens]
            pool.seq_lens.copy_(i32(model.lens))
            dfa.pages_trim(pool, ws=ws)
            model.trim()
            same(pool, model)
        dfa.stream_status(ws)


def test_shared_page_is_kept_by_its_last_writer():
    """Four sequences on one page: all write, and the last keeps it; two write, and nobody
    does."""
    for writers, copies in (([1, 1, 1, 1], 3), ([1, 0, 1, 0], 2), ([0, 0, 0, 1], 1),
                            ([0, 0, 0, 0], 0)):
        pool, model = new_pool(4, 4, 40, 16)
        pool.seq_lens.copy_(i32([20, 0, 0, 0]))
        model.lens = [20, 0, 0, 0]
        reserve(pool, model, [20, 0, 0, 0], 20)
        dfa.pages_fork(pool, i32([0, 0, 0, 0]))
        model.fork([0] * 4)
        same(pool, model)
        pool.seq_lens += i32(writers)
        model.lens = [20 + w for w in writers]
        jobs, info, _ = reserve(pool, model, writers, 1)
        assert int(info[0]) == copies
        same(pool, model)
        dfa.stream_status(pool.status)


def test_reserve_is_all_or_nothing():
    """Too few pages, or too little room for jobs: nothing changes, and it is reported."""
    pool, model = new_pool(3, 8, 10, 16)
    pool.seq_lens.copy_(i32([60, 60, 40]))              # 4 + 4 + 3 pages
    before = [x.clone() for x in (pool.block_table, pool.held, pool.refs)]
    jobs, info = dfa.pages_reserve(pool, 60, new_lens=i32([60, 60, 40]))
    assert info.tolist() == [0, 11, 1, 0]
    with pytest.raises(dfa.DfaError):
        dfa.stream_status(pool.status)
    assert all(torch.equal(a, b) for a, b in zip(before, (pool.block_table, pool.held, pool.refs)))
    pool.seq_lens.copy_(i32([60, 60, 32]))              # ten: all there are
    model.lens = [60, 60, 32]
    reserve(pool, model, [60, 60, 32], 60)
    same(pool, model)
    dfa.stream_status(pool.status)
    pool, model = new_pool(3, 8, 30, 16)
    pool.seq_lens.copy_(i32([20, 0, 0]))
    model.lens = [20, 0, 0]
    reserve(pool, model, [20, 0, 0], 20)
    dfa.pages_fork(pool, i32([0, 0, 0]))
    model.fork([0, 0, 0])
    pool.seq_lens += 1
    model.lens = [21] * 3
    for room in (0, 1):
        _, _, refused = reserve(pool, model, [1, 1, 1], 1, max_jobs=room)
        assert refused
        same(pool, model)
        with pytest.raises(dfa.DfaError):
            dfa.stream_status(pool.status)
    assert not reserve(pool, model, [1, 1, 1], 1, max_jobs=2)[2]
    same(pool, model)


def test_pool_reports_what_cannot_be():
    """Lengths, counts, sources and pages outside their ranges: reported, and nothing is
    written through them."""
    def fresh():
        pool, model = new_pool(3, 4, 20, 16)
        pool.seq_lens.copy_(i32([20, 30, 5]))
        model.lens = [20, 30, 5]
        reserve(pool, model, [20, 30, 5], 30)
        return pool, model

    def reported(pool):
        with pytest.raises(dfa.DfaError) as e:
            dfa.stream_status(pool.status)
        assert e.value.code == 6

    for src in ([0, 3, 2], [0, -2, 2], [2 ** 31 - 1, 1, 2]):
        pool, model = fresh()
        dfa.pages_fork(pool, i32(src))
        same(pool, model)                               # stays
        reported(pool)
    for held in (-1, 5, 2 ** 31 - 1):
        pool, model = fresh()
        pool.held[1] = held
        refs = pool.refs.clone()
        dfa.pages_fork(pool, i32([1, 1, 2]))            # from what cannot be
        reported(pool)
        dfa.pages_fork(pool, i32([0, 0, 2]))            # onto it
        reported(pool)
        dfa.pages_reserve(pool, 1)
        reported(pool)
        dfa.pages_trim(pool)
        reported(pool)
        assert torch.equal(pool.refs, refs) and int(pool.held[1]) == held
    for n in (-1, 65, 2 ** 31 - 1):
        pool, model = fresh()
        pool.seq_lens[1] = n
        refs = pool.refs.clone()
        dfa.pages_reserve(pool, 1)
        reported(pool)
        assert torch.equal(pool.refs, refs)
        dfa.pages_trim(pool)
        if n < 0:
            reported(pool)
        assert torch.equal(pool.refs, refs)
    for page in (-1, 20, 2 ** 31 - 1):
        pool, model = fresh()
        pool.block_table[1, 1] = page
        dfa.pages_reserve(pool, 14)                     # row 16 on: that page is written to
        reported(pool)
        dfa.pages_fork(pool, i32([0, 1, 1]))
        reported(pool)
        dfa.pages_fork(pool, i32([0, -1, 2]))
        reported(pool)
    pool, model = fresh()
    pool.refs.zero_()                                   # released more often than held
    pool.seq_lens.zero_()
    dfa.pages_trim(pool)
    reported(pool)


@pytest.mark.parametrize("dtype", [E4M3, BF16])
@pytest.mark.parametrize("Hkv,page,d,strided", [(1, 16, 64, False), (3, 32, 128, True),
                                                (8, 128, 128, False), (5, 64, 64, True)])
def test_copy(dtype, Hkv, page, d, strided):
    """Whole pages with their scales, as many as the device's count says, and no others."""
    npages = 12
    g = torch.Generator().manual_seed(Hkv)
    both = torch.randn(npages, 2, Hkv, page, d, generator=g).to(dtype).cuda()
    k, v = both[:, 0], both[:, 1]
    if not strided:
        k, v = k.contiguous(), v.contiguous()
    kw = {}
    if dtype is E4M3:
        kw = {n: torch.rand(npages, Hkv, generator=g).cuda() + 0.5 for n in ("k_scale", "v_scale")}
    cache = dfa.PagedCache(k, v, torch.zeros(1, 4, dtype=torch.int32, device="cuda"), i32([0]),
                           **kw)
    jobs = i32([[3, 7], [3, 0], [11, 10], [5, 4], [1, 2]])
    for count in (0, 1, 4, 5, 9, -3):
        want = {n: x.clone() for n, x in dict(k=k, v=v, **kw).items()}
        for a, b in jobs[:max(0, count)].tolist():
            for x in want.values():
                x[b] = x[a]
        dfa.cache_copy(cache, jobs, i32([count, 0, 0, 0]))
        dfa.stream_status(cache.status)
        for n, x in dict(k=k, v=v, **kw).items():
            assert torch.equal(x.contiguous().view(torch.uint8),
                               want[n].contiguous().view(torch.uint8)), (n, count)
    for pair in ([-1, 3], [3, 12], [2 ** 31 - 1, 1], [0, -2 ** 31]):
        want = k.clone()
        want[9] = want[8]
        dfa.cache_copy(cache, i32([pair, [8, 9]]), i32([2, 0, 0, 0]))
        with pytest.raises(dfa.DfaError) as e:
            dfa.stream_status(cache.status)
        assert e.value.code == 6
        assert torch.equal(k.contiguous().view(torch.uint8), want.contiguous().view(torch.uint8))


@pytest.mark.parametrize("dtype", [E4M3, BF16])
def test_beams_read_what_they_wrote(dtype):
    """Beams fork, take pages of their own, append and read back: every beam's cached rows
    are those of the tokens along its own history."""
    B, Hkv, d, page, width = 6, 2, 64, 16, 8
    npages = B * width
    cells = [torch.zeros(npages, Hkv, page, d, device="cuda").to(dtype) for _ in "kv"]
    kw = ({n: torch.ones(npages, Hkv, device="cuda") for n in ("k_scale", "v_scale")}
          if dtype is E4M3 else {})
    table = torch.zeros(B, width, dtype=torch.int32, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    pool = dfa.PagePool(table, lens, page, npages=npages)
    cache = dfa.PagedCache(*cells, table, lens, **kw)
    g = torch.Generator().manual_seed(3)
    history = [[] for _ in range(B)]
    rng = random.Random(4)
    for step in range(25):
        T = 21 if step == 0 else 1
        # small whole numbers: exact in 8 bits under any of these scales
        x = torch.randint(-7, 8, (B, Hkv, T, d), generator=g).float()
        if step:
            src = [rng.randrange(B) for _ in range(B)]
            dfa.pages_fork(pool, i32(src))
            history = [list(history[s]) for s in src]
        lens += T
        jobs, info = dfa.pages_reserve(pool, T)
        dfa.cache_copy(cache, jobs, info)
        dfa.cache_append(cache, x.to(BF16).cuda(), (-x).to(BF16).cuda())
        for b in range(B):
            history[b].append(x[b])
        n = int(lens[0])
        k, v = dfa.cache_gather(cache, n)
        for b in range(B):
            want = torch.cat(history[b], 1)
            assert torch.equal(k[b].float().cpu(), want), (step, b)
            assert torch.equal(v[b].float().cpu(), -want), (step, b)
    dfa.stream_status(pool.status)
    dfa.stream_status(cache.status)


def test_pool_captured_and_replayed():
    """One step of beams as a graph: each replay goes on from the state it finds."""
    B, width, page, npages = 5, 6, 16, 60
    pool, model = new_pool(B, width, npages, page)
    pool.seq_lens.copy_(i32([30] * B))
    model.lens = [30] * B
    reserve(pool, model, [30] * B, 30)
    src = i32(list(range(B)))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dfa.pages_fork(pool, src)
        pool.seq_lens.add_(1)
        jobs, info = dfa.pages_reserve(pool, 1)
    rng = random.Random(9)
    for _ in range(20):
        s = [rng.randrange(B) for _ in range(B)]
        src.copy_(i32(s))
        g.replay()
        model.fork(s)
        model.lens = [n + 1 for n in model.lens]
        want, taken, refused = model.reserve([1] * B)
        assert info.tolist() == [len(want), taken, refused, 0]
        assert jobs[:len(want)].tolist() == want
        same(pool, model)
    dfa.stream_status(pool.status)


def test_pool_on_other_streams():
    """The calls go to their stream or the current one; a pool may go while they run."""
    first = torch.cuda.current_stream()
    for named in (True, False):
        s = torch.cuda.Stream()
        pool, model = new_pool(9, 6, 80, 16)
        pool.seq_lens.copy_(i32([20] * 9))
        model.lens = [20] * 9
        src, tensors = i32([0] * 9), (pool.held, pool.refs, pool.block_table, pool.seq_lens)
        s.wait_stream(first)
        kw = {"stream": s} if named else {}
        with torch.cuda.stream(first if named else s):
            jobs, info = dfa.pages_reserve(pool, 20, **kw)
            dfa.pages_fork(pool, src, **kw)
            with torch.cuda.stream(s):
                pool.seq_lens.add_(1)
            jobs, info = dfa.pages_reserve(pool, 1, **kw)
            dfa.pages_trim(pool, **kw)
        want, taken, _ = model.reserve([20] * 9, 100)
        model.fork([0] * 9)
        model.lens = [21] * 9
        want, taken, refused = model.reserve([1] * 9, 100)
        model.trim()
        desc = pool.desc
        del pool
        junk = [torch.full((1 << 16,), 255, dtype=torch.uint8, device="cuda") for _ in range(8)]
        torch.cuda.synchronize()
        assert info.tolist() == [len(want), taken, refused, 0]
        assert jobs[:len(want)].tolist() == want
        held, refs, table, lens = (t.tolist() for t in tensors)
        assert held == [len(p) for p in model.pages] and refs == model.refs()
        assert lens == model.lens and desc.B == 9 and len(junk) == 8
        for b, p in enumerate(model.pages):
            assert table[b][:len(p)] == p
