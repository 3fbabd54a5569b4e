"""The ends of the serving operators' ranges, against plain fp64 forms: numbers far
apart, very large or very small, and what the device reports."""
import math

import pytest
import torch

import paged_ref as ref
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


def randn(*shape, seed=0, dtype=BF16):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


# ---------------------------------------------------------------------------
# 8-bit decode: the weights
# ---------------------------------------------------------------------------
def fine_tol(s, k, x, v, u, scale, terms=2):
    """For one query row that sees keys k [n, d], values v with scales u [n], and has
    the scores s (fp64): bounds on O's deviation relative to sum p |v|, and an
    absolute one per feature.
      dl   a score: d products summed in fp32, and its scaling; 2^x to two steps of
           2^-23; a lane's sum takes two of every 64 keys one after the other, then
           is joined over lanes, warps and blocks (64 additions);
      acc  a tile is two products (the weights' two terms), each of which cuts the
           sum off at 2^-23 once for its own terms and once for the total; as many
           again as 16 tiles for the joins;
      w    a weight as two fp16 terms, 2^-22, or as one, 2^-11; below fp16's normal
           numbers half a step is 2^-25, where the largest weight is 2^11 or more."""
    n, d = k.shape
    tiles = -(-n // 64)
    ds = (d + 4) * 2.0 ** -24 * scale * float((k.abs() @ x.abs()).max())
    dl = ds + 2.0 ** -22 + (2 * tiles + 64) * 2.0 ** -24
    acc = 4 * (tiles + 16) * 2.0 ** -23
    p = torch.softmax(s, 0)
    return (2 * dl + acc + 2.0 ** (-22 if terms == 2 else -11),
            2.0 ** -36 * float((p * u).max()) * (v.abs() / u[:, None]).sum(0))


@pytest.mark.parametrize("B,n", [(1, 131072), (600, 32768), (600, 2048)])
@pytest.mark.parametrize("Hq", [4, 12])
@pytest.mark.parametrize("p_sink,loud", [(0.9, 0), (0.99, 0), (0.996, 0), (0.99, 6), (0.996, -6)])
def test_decode_tail_behind_a_sink(B, n, Hq, p_sink, loud):
    """One key takes nearly all the probability and has a value of zero: the output
    is the tail's, whose weights lie 2^9 to 2^25 below the largest.  A page in the
    middle has louder or quieter values.  (All sequences read the same pages; with
    600 of them most are not cut.)"""
    d, page, scale = 64, 64, 0.125
    g = torch.Generator().manual_seed(n + Hq)
    pages = n // page
    k = torch.randn(pages, 1, page, d, generator=g)
    k[..., 0] = 0.0
    v = 1.0 + torch.rand(pages, 1, page, d, generator=g)
    k[0, 0, 0], v[0, 0, 0] = 0.0, 0.0
    k[0, 0, 0, 0] = 1.0
    vs = torch.ones(pages, 1)
    vs[pages // 2] = 2.0 ** loud
    k, v = k.to(E4M3), v.to(E4M3)
    q = torch.randn(Hq, d, generator=g) * 0.5
    # the tail's logits are normal with variance (63 / 64) / 4: E exp = exp(var / 2)
    q[:, 0] = (math.log(n) + 0.123 + math.log(p_sink / (1 - p_sink))) / scale
    q = q.to(BF16)
    c = dfa.PagedCache(k.cuda(), v.cuda(),
                       torch.arange(pages, dtype=torch.int32).repeat(B, 1).cuda(),
                       torch.full((B,), n, dtype=torch.int32, device="cuda"),
                       k_scale=torch.ones(pages, 1, device="cuda"), v_scale=vs.cuda())
    K, V = k.double().view(n, d), v.double().view(n, d) * vs.double().repeat_interleave(page, 0)
    u = vs.double().repeat_interleave(page, 0)[:, 0]
    qs = q.view(1, Hq, 1, d).expand(B, Hq, 1, d).contiguous().cuda()
    for fp32 in (True, False):
        o, lse = dfa.decode_paged(c, qs, scale=scale, out_fp32=fp32)
        o, lse = o.cpu().double()[:, :, 0], lse.cpu().double()[:, :, 0]
        for h in range(Hq):
            x = q[h].double()
            s = scale * (K @ x)
            want = torch.softmax(s, 0) @ V
            rel, floor = fine_tol(s, K, x, V, u, scale, 2 if fp32 or Hq <= 8 else 1)
            tol = rel * want + floor
            tol = tol + ref.HALF_STEP[torch.float32 if fp32 else BF16] * (want + tol)
            err = (o[:, h] - want).abs()
            assert (err <= tol).all(), (h, fp32, float((err / want).max()))
            rel = fine_tol(s, K, x, V, u, scale)[0]
            off = (lse[:, h] - torch.logsumexp(s, 0)).abs()
            assert (off <= rel + 2.0 ** -23 * float(lse.max())).all()


@pytest.mark.parametrize("T", [1, 3])
@pytest.mark.parametrize("d,page,lens", [(64, 16, [1, 200, 64]), (128, 64, [333, 17, 129]),
                                         (128, 16, [90, 5, 700])])
def test_decode_8_bit_in_fp32(d, page, lens, T):
    """An fp32 output has fp32's accuracy: the weights are not rounded to fp16."""
    c = ref.Cache(E4M3, 3, 2, d, page, -(-max(lens) // page), lens, seed=200 + d + page)
    q, scale = randn(3, 8, T, d, seed=201), 1 / math.sqrt(d)
    ql = [min(T, n) for n in lens]
    O, LSE, _, _ = ref.attention(c, q, ql)
    o, lse = dfa.decode_paged(c.cuda(), q.cuda(), out_fp32=True,
                              q_lens=torch.tensor(ql, dtype=torch.int32, device="cuda"))
    for b, L in enumerate(lens):
        K, V = c.rows("k", b, L), c.rows("v", b, L)
        pg = c.table[b, torch.arange(L) // page].long()
        for h in range(8):
            u = c.scales["v"][pg, h // 4].double()
            for t in range(ql[b]):
                n = L - ql[b] + t + 1
                k, v, x = K[h // 4, :n], V[h // 4, :n], q[b, h, t].double()
                s = scale * (k @ x)
                rel, floor = fine_tol(s, k, x, v, u[:n], scale)
                tol = rel * (torch.softmax(s, 0) @ v.abs()) + floor
                ref.check(o[b, h, t], O[b, h, t], tol, torch.float32, (b, h, t))
                assert abs(float(lse[b, h, t]) - float(LSE[b, h, t])) <= (
                    rel + 2.0 ** -23 * abs(float(LSE[b, h, t])))


# ---------------------------------------------------------------------------
# decode: scores far from zero
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [E4M3, BF16])
@pytest.mark.parametrize("Hq,T", [(2, 1), (12, 2)])
@pytest.mark.parametrize("n,width", [(200, 13), (200, 40), (5000, 313)])
@pytest.mark.parametrize("score", [-3e6, 7.3e8, -7.3e8, 1e25, -1e25])
def test_decode_equal_scores_far_from_zero(dtype, Hq, T, n, width, score):
    """Every score the same, very high or very low: the softmax is uniform over what
    a token sees, in tables whose segments are cut and in short ones."""
    uniform_over_equal_scores(dtype, Hq, T, n, width, score)


def uniform_over_equal_scores(dtype, Hq, T, n, width, score):
    d, page = 64, 16
    c = ref.Cache(dtype, 1, 1, d, page, width, [n], seed=210)
    k = torch.zeros(c.npages, 1, page, d)
    k[..., 5] = -1.0 if dtype is E4M3 else -2.0 ** 60
    c.cells["k"] = k.to(dtype)
    if dtype is E4M3:
        c.scales["k"][:] = 2.0 ** 60
        c.scales["v"][:] = 0.25      # (equal: the kernel adds their logarithms to the scores)
    q = torch.zeros(1, Hq, T, d)
    q[..., 5] = -score / 2.0 ** 60
    q = q.to(BF16)
    x = -float(q[0, 0, 0, 5]) * 2.0 ** 60
    o, lse = dfa.decode_paged(c.cuda(), q.cuda(), scale=1.0, out_fp32=True)
    V = c.rows("v", 0, n)[0]
    for t in range(T):
        m = n - T + t + 1
        want = V[:m].mean(0).expand(Hq, d)
        # equal weights: an exact one, at most 2^8 below its reference, so that bf16's two
        # terms and fp16's are exact too; m values summed in fp32 (as in fine_tol)
        rel = 4 * (m / 64 + 17) * 2.0 ** -23 + (m + 64) * 2.0 ** -24
        ref.check(o[0, :, t], want, rel * V[:m].abs().mean(0), torch.float32, t)
        tol = 2.0 ** -21 * abs(x) + 2.0 ** -16   # log m to fp32's steps, and below
        assert ((lse[0, :, t].cpu().double() - x - math.log(m)).abs() <= tol).all()


@pytest.mark.parametrize("dtype", [E4M3, BF16])
@pytest.mark.parametrize("Hq,T", [(1, 1), (4, 3), (12, 2)])
@pytest.mark.parametrize("n,width", [(3, 1), (1, 1), (200, 13), (200, 40), (5000, 313)])
@pytest.mark.parametrize("score", [-3e30, -1.5e38, 1.5e38])
def test_decode_lowest_scores_are_seen(dtype, Hq, T, n, width, score):
    """Finite scores next to fp32's own lowest and highest count like any others (a row
    without a visible key alone gives 0 and -inf)."""
    if n < T:
        pytest.skip("more tokens than rows")
    uniform_over_equal_scores(dtype, Hq, T, n, width, score)


@pytest.mark.parametrize("dtype", [E4M3, BF16])
def test_decode_lowest_scores_are_told_apart(dtype):
    """One key a little less far down than the others takes all the weight."""
    c = ref.Cache(dtype, 1, 1, 64, 16, 8, [120], seed=211)
    k = torch.zeros(c.npages, 1, 16, 64)
    k[..., 5] = -2.0
    k[int(c.table[0, 4]), 0, 3, 5] = -1.75
    if dtype is BF16:
        k *= 2.0 ** 60
    else:
        c.scales["k"][:] = 2.0 ** 60
    c.cells["k"] = k.to(dtype)
    q = torch.zeros(1, 2, 1, 64, dtype=BF16)
    q[..., 5] = 2.0 ** 45
    o, lse = dfa.decode_paged(c.cuda(), q.cuda(), scale=1.0, out_fp32=True)
    # the one weight is a power of two, its value has few bits: O is exact
    assert torch.equal(o[0, 0, 0].cpu().double(), c.rows("v", 0, 120)[0, 67])
    assert abs(float(lse[0, 0, 0]) / (-1.75 * 2.0 ** 105) - 1) <= 2.0 ** -21


@pytest.mark.parametrize("dtype", [E4M3, BF16])
@pytest.mark.parametrize("Hq,T", [(2, 1), (12, 2)])
@pytest.mark.parametrize("loud", [13, 20, 24, 28, 40, 90])
@pytest.mark.parametrize("exps", [[0], [0, -100, 3], [-100, 50], [-30, 30, -35]])
def test_decode_one_key_far_above_the_others(dtype, Hq, T, loud, exps):
    """Scores of up to 2^90 either way, and in 8 bits pages whose values are louder or
    quieter by as much as 2^100: O is the value of the key with the highest score."""
    if dtype is BF16 and len(exps) > 1:
        pytest.skip("bf16 cells have no scales")
    d, page, width, n = 64, 16, 40, 630
    c = ref.Cache(dtype, 1, 1, d, page, width, [n], seed=214)
    if dtype is E4M3:
        e = torch.tensor([float(exps[i % len(exps)]) for i in range(width)])
        c.scales["v"][c.table[0].long(), 0] = torch.exp2(e)
    q = (randn(1, Hq, T, d, seed=215).float() * 2.0 ** loud).to(BF16)
    K, V = c.rows("k", 0, n)[0], c.rows("v", 0, n)[0]
    o, lse = dfa.decode_paged(c.cuda(), q.cuda(), scale=1.0, out_fp32=True)
    o, lse = o.cpu().double(), lse.cpu().double()
    told = 0
    for h in range(Hq):
        for t in range(T):
            m, x = n - T + t + 1, q[0, h, t].double()
            s = K[:m] @ x
            two = torch.topk(s, 2).values
            ds = (d + 4) * 2.0 ** -24 * float((K[:m].abs() @ x.abs()).max())
            if two[0] - two[1] <= 2 * ds + 100:   # 2^-100 / ln 2: times any other value nothing
                continue
            told += 1
            want = V[int(s.argmax())]
            # the weight is at most 2^15 and its own sum: O = (w c) 2^D / w, and two roundings
            assert ((o[0, h, t] - want).abs() <= 2.0 ** -20 * want.abs() + 1e-20).all(), (h, t)
            assert abs(float(lse[0, h, t]) - float(two[0])) <= ds + 2.0 ** -22 * abs(float(two[0]))
    assert told >= 1


# ---------------------------------------------------------------------------
# an append and the decode that is launched while it runs
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("d,page", [(64, 16), (128, 64)])
def test_captured_behind_an_append_that_raises_scales(d, page):
    """A step's append raises the scales of the page that the decode behind it reads,
    moves on to new pages, and the lengths advance just before: 60 replays of one
    graph, each against the same calls made one at a time."""
    B, Hq, Hkv = 2, 4, 2
    c = ref.Cache(E4M3, B, Hkv, d, page, 12, [3, page], seed=240)
    a, b = c.cuda(), c.cuda()
    ws = dfa.paged_workspace(a, Hq, 1)
    ins = [torch.zeros(B, h, 1, d, dtype=BF16, device="cuda") for h in (Hq, Hkv, Hkv)]
    spec = dfa.rope_spec(d, layout="half")
    out, lse = torch.empty_like(ins[0]), torch.empty(B, Hq, 1, device="cuda")
    qr = torch.empty_like(ins[0])
    steps = 60

    def step(cache, sync):
        cache.seq_lens.add_(1)
        dfa.cache_append(cache, ins[1], ins[2], rope=spec, q=ins[0], q_out=qr, ws=ws)
        if sync:
            torch.cuda.synchronize()
        dfa.decode_paged(cache, qr, out=out, lse=lse, ws=ws)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(a, False)
    for i in range(steps):
        for j, t in enumerate(ins):
            # louder and louder within a page, then quiet again
            t.copy_(randn(*t.shape, seed=241 + 3 * i + j) * (2.0 ** (i % page) if j else 1.0))
        g.replay()
        got = out.clone(), lse.clone()
        step(b, True)
        assert torch.equal(out, got[0]) and torch.equal(lse, got[1]), i
    dfa.stream_status(ws)
    for n in ("k_scale", "v_scale"):
        assert torch.equal(getattr(a, n), getattr(b, n))


# ---------------------------------------------------------------------------
# cells
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("d,page", [(64, 16), (128, 64)])
def test_largest_values_stay_finite(d, page):
    """bf16's largest values, either sign, in an 8-bit page: the scale is 2^120 and
    the largest finite multiple of it in a cell 240, since 256 * 2^120 is an
    infinity.  Rows stored before are raised to the same scale; infinities and NaN
    are still NaN."""
    big = float(torch.finfo(BF16).max)
    c = ref.Cache(E4M3, 2, 2, d, page, 2, [page + 4, 9], seed=220)
    dev = c.cuda()
    ws = dfa.paged_workspace(dev, 4, 1)
    v = randn(2, 2, 6, d, seed=221)
    edge = [big, -big, 1.9375 * 2.0 ** 127, -1.9375 * 2.0 ** 127, 1.9296875 * 2.0 ** 127,
            1.875 * 2.0 ** 127, 448 * 2.0 ** 119, -2.0 ** 127]
    want = [240.0, -240.0, 240.0, -240.0, 240.0, 240.0, 224.0, -128.0]
    v[:, :, 3, :8] = torch.tensor(edge).to(BF16)
    v[:, :, 4] = big
    v[0, :, 5, 3], v[0, :, 5, 4] = float("nan"), float("inf")
    dev.seq_lens -= 6
    old = torch.full((2, 2, 2, d), 3e38, dtype=BF16)     # (scale 2^120) behind a page's beginning
    dfa.cache_append(dev, old.cuda(), old.cuda(), ws=ws)
    dev.seq_lens += 6
    dfa.cache_append(dev, v.cuda(), v.cuda(), ws=ws)
    dfa.stream_status(ws)
    k_out, v_out = dfa.cache_gather(dev, page + 4, ws=ws)
    for name, got in (("k", k_out), ("v", v_out)):
        for b, L in enumerate([page + 4, 9]):
            for j in (3, 4):
                at = L - 6 + j
                pg = int(c.table[b, at // page])
                row = getattr(dev, name)[pg, :, at % page].float().cpu()
                assert (getattr(dev, name + "_scale")[pg].cpu() == 2.0 ** 120).all()
                assert (row == 240.0).all() if j == 4 else row[:, :8].tolist() == [want] * 2
                assert torch.equal(got[b, :, at].double().cpu(), row.double() * 2.0 ** 120)
            assert got[b, :, L - 6:L].isfinite().sum() == 2 * 6 * d - (4 if b == 0 else 0)
    # a token that sees row 4 of the second sequence alone next to quiet ones
    one = dfa.PagedCache(dev.k, dev.v, dev.block_table[1:].contiguous(),
                         torch.tensor([8], dtype=torch.int32, device="cuda"),
                         k_scale=torch.ones_like(dev.k_scale), v_scale=dev.v_scale)
    q = torch.zeros(1, 2, 1, d, dtype=BF16, device="cuda")
    o, lse = dfa.decode_paged(one, q, out_fp32=True)
    V = v_out[1, :, :8].double().cpu()
    assert o.isfinite().all()
    ref.check(o[0, :, 0], V.mean(1), 2.0 ** -18 * V.abs().mean(1), torch.float32)
    assert (lse.cpu().double() - math.log(8)).abs().max() <= 2.0 ** -20


# ---------------------------------------------------------------------------
# errors of the device
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [E4M3, BF16])
def test_errors_without_a_workspace_are_kept(dtype):
    """Calls that were given no workspace report bad pages and lengths to the cache's
    own status word; with a workspace, to that."""
    c = ref.Cache(dtype, 2, 2, 64, 16, 3, [40, 40], seed=230)
    dev = c.cuda()
    k, q = randn(2, 2, 2, 64, seed=231).cuda(), randn(2, 4, 1, 64, seed=232).cuda()
    calls = (lambda **kw: dfa.cache_append(dev, k, k, **kw),
             lambda **kw: dfa.cache_gather(dev, 48, **kw),
             lambda **kw: dfa.decode_paged(dev, q, **kw))
    ws = dfa.paged_workspace(dev, 4, 1)
    for bad in ("page", "length"):
        for f in calls:
            f()
            dfa.stream_status(dev.status)
        if bad == "page":
            keep = int(dev.block_table[1, 2])
            dev.block_table[1, 2] = c.npages
        else:
            dev.seq_lens[1] = 49
        for f in calls:
            f()
            with pytest.raises(dfa.DfaError) as e:
                dfa.stream_status(dev.status)
            assert e.value.code == 6
            dfa.stream_status(dev.status)  # read and cleared
            f(ws=ws)
            dfa.stream_status(dev.status)
            with pytest.raises(dfa.DfaError):
                dfa.stream_status(ws)
        if bad == "page":
            dev.block_table[1, 2] = keep
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            calls[2]()
        g.replay()
        if bad == "length":
            with pytest.raises(dfa.DfaError):
                dfa.stream_status(dev.status)
            dev.seq_lens[1] = 40
        dfa.stream_status(dev.status)


# ---------------------------------------------------------------------------
# 8-bit decode: the queries
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("T", [1, 9])
@pytest.mark.parametrize("loud", [12, 18, 26])
def test_decode_queries_with_one_loud_element(loud, T):
    """An element 2^26 times the others, where the keys are zero: the others count
    in full."""
    d, lens = 128, [70, 300]
    c = ref.Cache(E4M3, 2, 1, d, 16, 19, lens, seed=212)
    x = c.cells["k"].float()
    x[..., 7] = torch.where(x[..., 7].isnan(), x[..., 7], torch.tensor(0.0))
    c.cells["k"] = x.to(E4M3)
    q = randn(2, 2, T, d, seed=213)
    q[..., 7] = 1.5 * 2.0 ** loud
    O, LSE, _, _ = ref.attention(c, q)
    o, lse = dfa.decode_paged(c.cuda(), q.cuda(), out_fp32=True)
    for b, L in enumerate(lens):
        K, V = c.rows("k", b, L)[0], c.rows("v", b, L)[0]
        u = c.scales["v"][c.table[b, torch.arange(L) // 16].long(), 0].double()
        for h in range(2):
            for t in range(T):
                n, x = L - T + t + 1, q[b, h, t].double()
                s = (K[:n] @ x) / math.sqrt(d)
                rel, floor = fine_tol(s, K[:n], x, V[:n], u[:n], 1 / math.sqrt(d))
                tol = rel * (torch.softmax(s, 0) @ V[:n].abs()) + floor
                ref.check(o[b, h, t], O[b, h, t], tol, torch.float32, (b, h, t))
                assert abs(float(lse[b, h, t]) - float(LSE[b, h, t])) <= (
                    rel + 2.0 ** -23 * abs(float(LSE[b, h, t])))


# ---------------------------------------------------------------------------
# angles
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("d,H", [(128, 1), (64, 3), (128, 40)])
def test_rope_cos_and_sin(layout, d, H):
    """Rotated unit vectors are the cos and sin themselves.  Every quarter of the
    turn, small and large positions.  The bound: what is left of the angle after
    whole quarter turns is at most pi / 4 and has 24 bits, 2.4e-8; its cos and sin are
    off by at most 7.5e-8 more; the frequency (fp64) by |position| f 2^-52."""
    L = 4099
    x = torch.zeros(1, H, L, d)
    first = slice(0, d // 2) if layout == "half" else slice(0, d, 2)
    x[..., first] = 1.0
    pos = torch.randint(-20000, 20000, (1, L), generator=torch.Generator().manual_seed(d + H),
                        dtype=torch.int32)
    pos[0, :5] = torch.tensor([0, 1, -1, 2, 3])
    got = dfa.rope(x.cuda(), dfa.rope_spec(d, layout=layout), positions=pos.cuda()).cpu().double()
    want = ref.rope(x, pos[:, None], layout, d)
    err = (got - want).abs().max()
    assert err <= 1.0e-7 + 20000 * 2.0 ** -51, float(err)
