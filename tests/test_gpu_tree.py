"""GPU parity of trees of drafted tokens over a paged cache (plan, positions of appended
rows, attention, kept rows) against plain fp64 forms: cells of both types, every page
size, one to 1024 query rows a head, lengths around the tiles' borders, masks that leave
rows empty, NaN wherever a node may not look, numbers far apart, refused and reported
arguments, graphs, streams, and a whole step of speculative decoding."""
import math

import pytest
import torch

import branch_ref as bref
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


def i32(x, dev="cuda"):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device=dev)


# ---------------------------------------------------------------------------
# the plan
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("B,T,lens", [(1, 1, [1]), (3, 7, [7, 30, 5]), (2, 32, [40, 32]),
                                      (2, 33, [1000, 33]), (1, 64, [64]), (2, 200, [333, 200]),
                                      (1, 1023, [1500]), (1, 1024, [1024])])
@pytest.mark.parametrize("shape", ["tree", "chain", "star"])
def test_plan(B, T, lens, shape):
    if shape == "tree":
        parents = bref.random_parents(B, T, seed=T)
    else:
        parents = (torch.arange(T) - 1 if shape == "chain" else torch.full((T,), -1)).to(
            torch.int32).repeat(B, 1)
    n = [min(T, L) for L in lens]
    if T == 7:
        n = [0, 7, 5]
    c = ref.Cache(BF16, B, 1, 64, 128, 12, [0] * B)
    c.lens = i32(lens, "cpu")
    dev = c.cuda()
    W = -(-T // 32)
    mask = torch.full((B, T, W), 7, dtype=torch.int32, device="cuda")
    pos = torch.full((B, T), 7, dtype=torch.int32, device="cuda")
    ws = dfa.paged_workspace(dev)
    r = dfa.tree_plan(dev, parents.cuda(), q_lens=i32(n), mask=mask, positions=pos, ws=ws)
    dfa.stream_status(ws)
    assert r[0] is mask and r[1] is pos
    sees = bref.sees_of(parents)
    for b in range(B):
        assert torch.equal(mask[b, :n[b]].cpu(), bref.pack(sees[b, :n[b]]))
        want = lens[b] - n[b] + sees[b, :n[b]].sum(-1) - 1
        assert torch.equal(pos[b, :n[b]].cpu().long(), want)
        assert (mask[b, n[b]:] == 7).all() and (pos[b, n[b]:] == 7).all()


def test_plan_reports_a_parent_that_cannot_be():
    c = ref.Cache(BF16, 3, 1, 64, 16, 2, [5, 5, 5])
    dev = c.cuda()
    good = [-1, 0, 0, 2, 1]
    for bad, at in ((3, 3), (5, 1), (-2, 4), (2 ** 31 - 1, 2), (-2 ** 31, 0)):
        parents = torch.tensor([good] * 3, dtype=torch.int32)
        parents[1, at] = bad
        mask, pos = dfa.tree_plan(dev, parents.cuda())
        with pytest.raises(dfa.DfaError) as e:
            dfa.stream_status(dev.status)
        assert e.value.code == 6
        parents[1, at] = -1                      # taken for the context
        assert torch.equal(mask.cpu(), bref.pack(bref.sees_of(parents)))


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def rows_max(c):
    return max(float(bref.rows(c, "v", b, int(c.lens[b])).abs().max()) for b in range(c.B))


def check_tree(c, dev, q, sees, q_lens=None, scale=None, fp32=(False, True), ws=None, **kw):
    B, Hq, T, d = q.shape
    if ws is None:
        ws = dfa.tree_workspace(dev, Hq, T)
    mask = bref.pack(sees).cuda()
    qd = q.cuda() if not q.is_cuda else q
    for f in fp32:
        # weights in fp16 (2^-11) for 8-bit cells and a bf16 output, else in two terms
        w = 2.0 ** -11 if c.dtype is E4M3 and not f else 2.0 ** -16
        O, LSE, tO, tL = bref.attention(c, q.cpu(), sees, q_lens, scale, w)
        dt = torch.float32 if f else BF16
        out = torch.full((B, Hq, T, d), 7.0, dtype=dt, device="cuda")
        lse = torch.full((B, Hq, T), 7.0, device="cuda")
        got = dfa.decode_tree(dev, qd, mask, q_lens=i32(q_lens), scale=scale, out_fp32=f, ws=ws,
                              out=out, lse=lse, **kw)
        assert got[0] is out and got[1] is lse
        dfa.stream_status(ws)
        gone = O.isnan().all(-1)
        for b in range(B):
            n = T if q_lens is None else q_lens[b]
            assert (out[b, :, n:] == 7).all() and (lse[b, :, n:] == 7).all()
            ref.check(out[b, :, :n], O[b, :, :n], tO[b, :, :n], dt, ("O", b, f))
            ref.check(lse[b, :, :n], LSE[b, :, :n], tL[b, :, :n], torch.float32, ("LSE", b, f))
    return gone


@pytest.mark.parametrize("dtype", [E4M3, BF16])
@pytest.mark.parametrize("page,d", [(16, 64), (16, 128), (32, 128), (64, 64), (64, 128),
                                    (128, 64), (128, 128)])
def test_tree_page_sizes(dtype, page, d):
    """Trees that begin in one page and tile and end in another, none, one of the whole
    sequence."""
    lens = [9, 127, 128, 129, 140, 260, 1]
    n = [9, 5, 9, 3, 9, 0, 1]
    c = ref.Cache(dtype, 7, 2, d, page, -(-260 // page), lens, seed=page + d)
    q = randn(7, 6, 9, d, seed=1)
    check_tree(c, c.cuda(), q, bref.sees_of(bref.random_parents(7, 9, seed=2)), n)


@pytest.mark.parametrize("dtype", [E4M3, BF16])
@pytest.mark.parametrize("Hkv,G,T", [(1, 1, 1), (2, 1, 2), (1, 3, 5), (1, 8, 2), (2, 4, 4),
                                     (1, 1, 17), (1, 5, 25), (1, 4, 32), (1, 2, 65), (1, 3, 43),
                                     (1, 8, 32), (1, 1, 257), (1, 16, 31), (1, 1, 1024),
                                     (1, 1024, 1), (2, 8, 37)])
def test_tree_rows(dtype, Hkv, G, T):
    """One to 1024 query rows a head; the tree in more than one tile."""
    lens = [T + 130, T, T + 1000]
    c = ref.Cache(dtype, 3, Hkv, 64, 64, -(-(T + 1000) // 64), lens, seed=T)
    q = randn(3, Hkv * G, T, 64, seed=G)
    sees = bref.sees_of(bref.random_parents(3, T, seed=G + T))
    check_tree(c, c.cuda(), q, sees, [T, T, max(0, T - 3)], fp32=(T % 2 == 0,))


@pytest.mark.parametrize("dtype", [E4M3, BF16])
def test_tree_any_mask(dtype):
    """Bits without any order, nodes that see nothing of the tree, no context: rows
    without a key."""
    T = 40
    g = torch.Generator().manual_seed(5)
    sees = torch.rand(4, T, T, generator=g) < 0.4
    sees[:, 3] = False
    sees[:, 17] = False
    sees[:, :, 20] = False                     # a node that nobody sees
    lens, n = [T, T + 100, 30, 137], [T, T, 30, 37]
    c = ref.Cache(dtype, 4, 2, 128, 32, 5, lens, seed=6)
    q = randn(4, 8, T, 128, seed=7)
    check_tree(c, c.cuda(), q, sees, n)
    sees[:] = False
    check_tree(c, c.cuda(), q, sees, n, fp32=(False,))


@pytest.mark.parametrize("dtype", [E4M3, BF16])
@pytest.mark.parametrize("B,Hkv,G,T,L,page,d", [(1, 1, 4, 8, 40000, 64, 128),
                                                (1, 2, 1, 3, 20011, 16, 64),
                                                (3, 3, 4, 60, 5003, 128, 128),
                                                (40, 8, 4, 5, 300, 16, 128)])
def test_tree_long_and_many(dtype, B, Hkv, G, T, L, page, d):
    """Sequences cut over many blocks and joined; many short ones."""
    lens = [max(T, L - 97 * b % L) for b in range(B)]
    c = ref.Cache(dtype, 1, Hkv, d, page, -(-L // page), [L], seed=L)
    if B > 1:                                  # sequences that share their pages
        c.B, c.table, c.lens = B, c.table.repeat(B, 1), i32(lens, "cpu")
    check = slice(0, B)
    q = randn(B, Hkv * G, T, d, seed=8)
    sees = bref.sees_of(bref.random_parents(B, T, seed=9))
    check_tree(c, c.cuda(), q[check], sees, fp32=(False,))


@pytest.mark.parametrize("dtype", [E4M3, BF16])
@pytest.mark.parametrize("G,T", [(1, 2), (8, 16)])
@pytest.mark.parametrize("louder", [False, True])
def test_tree_fp32_over_many_tiles(dtype, G, T, louder):
    """More than 40 tiles to a block, whose sums are set apart on the way; scores (or, in 8
    bits, values) that rise before and after that, by steps which what came before them
    outlives and does not."""
    B, Hkv, d, page = 20, 8, 64, 64
    lens = [5900 - 31 * b for b in range(B)]
    c = ref.Cache(dtype, 1, Hkv, d, page, -(-5900 // page), [5900], seed=T)
    if louder:
        for p in range(c.table.shape[1]):
            at = int(c.table[0, p])
            if dtype is E4M3:
                c.scales["v"][at] *= 2.0 ** (p // 4)
                c.scales["k"][at] *= 2.0 ** (3 * (p >= 25) + 2 * (p >= 75))
            else:
                x = c.cells["k"][at].float() * 2.0 ** (4 * (p >= 25) + 2 * (p >= 75))
                c.cells["k"][at] = x.to(dtype)
    c.B, c.table, c.lens = B, c.table.repeat(B, 1), i32(lens, "cpu")   # (the same pages)
    q = randn(B, Hkv * G, T, d, seed=67)
    sees = bref.sees_of(bref.random_parents(B, T, seed=68))
    check_tree(c, c.cuda(), q, sees, fp32=(True,))


def test_tree_equals_a_chain():
    """A chain is what decode_paged computes."""
    c = ref.Cache(E4M3, 3, 2, 128, 64, 20, [1200, 77, 640], seed=11)
    dev = c.cuda()
    q = randn(3, 8, 6, 128, seed=12).cuda()
    parents = (torch.arange(6, dtype=torch.int32) - 1).repeat(3, 1)
    mask = bref.pack(bref.sees_of(parents)).cuda()
    a, la = dfa.decode_tree(dev, q, mask, out_fp32=True)
    b, lb = dfa.decode_paged(dev, q, out_fp32=True)
    # each side's weights 2^-22, its 2^x and sums 2^-21, its accumulation 60 * 2^-23,
    # relative to sum p |v|, which is at most the largest |v| (4 sigma of scale 1..8 cells)
    top = float(dev.v.float().nan_to_num().abs().max() * dev.v_scale.max())
    assert (a - b).abs().max() <= 2 * top * (2.0 ** -22 + 2.0 ** -20 + 60 * 2.0 ** -23)
    assert (la - lb).abs().max() <= 2.0 ** -16


def test_tree_strided_queries_and_default_outputs():
    c = ref.Cache(BF16, 2, 2, 64, 16, 4, [50, 33], seed=13)
    dev = c.cuda()
    T = 5
    sees = bref.sees_of(bref.random_parents(2, T, seed=14))
    packed = randn(2, T, 12, 64, seed=15).cuda()        # heads of a projection
    q = packed.transpose(1, 2)[:, 2:10]
    check_tree(c, dev, q, sees)
    o, lse = dfa.decode_tree(dev, q, bref.pack(sees).cuda())
    O, LSE, tO, tL = bref.attention(c, q.cpu(), sees)
    ref.check(o, O, tO, BF16)
    ref.check(lse, LSE, tL, torch.float32)
    dfa.stream_status(dev.status)


@pytest.mark.parametrize("dtype", [E4M3, BF16])
@pytest.mark.parametrize("G", [1, 16])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_tree_non_finite_nodes_stay_where_they_are_seen(dtype, G, bad):
    """A node's key or value that is not finite reaches the nodes that see it, in the
    features it has it in, and no other."""
    if dtype is E4M3 and bad == bad:
        pytest.skip("8-bit cells hold NaN alone")
    T, d, L = 12, 64, 300
    parents = bref.random_parents(2, T, seed=16, roots=0.3)
    sees = bref.sees_of(parents)
    for name, node in (("v", 2), ("k", 4), ("v", T - 1)):
        c = ref.Cache(dtype, 2, 1, d, 16, -(-L // 16), [L, T], seed=17)
        clean = bref.attention(c, randn(2, G, T, d, seed=18), sees)
        for b, n in ((0, L), (1, T)):
            j = n - T + node
            x = c.cells[name].float()
            x[int(c.table[b, j // 16]), 0, j % 16, 7] = bad
            c.cells[name] = x.to(dtype)
        dev = c.cuda()
        q = randn(2, G, T, d, seed=18)
        o, lse = dfa.decode_tree(dev, q.cuda(), bref.pack(sees).cuda(), out_fp32=True)
        o, lse = o.cpu().double(), lse.cpu().double()
        O, LSE, tO, tL = clean
        for b in range(2):
            for t in range(T):
                hit = bool(sees[b, t, node])
                if not hit or name == "v":
                    f = torch.ones(d, dtype=torch.bool)
                    f[7] = not hit
                    ref.check(o[b, :, t][:, f], O[b, :, t][:, f], tO[b, :, t][:, f] * 2 ** 5,
                              torch.float32, (name, b, t))
                    ref.check(lse[b, :, t], LSE[b, :, t], tL[b, :, t], torch.float32)
                if hit and name == "v":
                    assert not o[b, :, t, 7].isfinite().any()
                    if bad == bad:                       # one infinity: itself
                        assert (o[b, :, t, 7] == bad).all()
                if hit and name == "k" and bad != bad:
                    assert o[b, :, t].isnan().all()


@pytest.mark.parametrize("dtype", [E4M3, BF16])
@pytest.mark.parametrize("G", [1, 4, 16])
def test_tree_nan_nodes_with_bf16_outputs(dtype, G):
    T, d, L = 12, 128, 300
    sees = bref.sees_of(bref.random_parents(2, T, seed=70, roots=0.3))
    c = ref.Cache(dtype, 2, 1, d, 32, -(-L // 32), [L, T], seed=71)
    q = randn(2, G, T, d, seed=72)
    w = 2.0 ** -11 if dtype is E4M3 else 2.0 ** -16
    O, LSE, tO, tL = bref.attention(c, q, sees, weight=w)
    node = 3
    for b, n in ((0, L), (1, T)):
        j = n - T + node
        x = c.cells["v"].float()
        x[int(c.table[b, j // 32]), 0, j % 32, 100] = float("nan")
        c.cells["v"] = x.to(dtype)
    o, lse = dfa.decode_tree(c.cuda(), q.cuda(), bref.pack(sees).cuda())
    ref.check(lse, LSE, tL, torch.float32)
    for b in range(2):
        for t in range(T):
            hit = bool(sees[b, t, node])
            f = torch.ones(d, dtype=torch.bool)
            f[100] = not hit
            # (the node's own weight is then fp32's, the others' as before: no more than w)
            ref.check(o[b, :, t][:, f], O[b, :, t][:, f], tO[b, :, t][:, f], BF16, (b, t))
            assert not hit or o[b, :, t, 100].isnan().all()


@pytest.mark.parametrize("dtype", [E4M3, BF16])
@pytest.mark.parametrize("G", [2, 30])
@pytest.mark.parametrize("off", [2.0 ** 13, -2.0 ** 20])
def test_tree_far_scores_with_bf16_outputs(dtype, G, off):
    """As below, at offsets on either side of where scores are rounded first."""
    T, d = 3, 64
    c = ref.Cache(dtype, 1, 1, d, 64, 4, [200], seed=73)
    x = c.cells["k"].float()
    x[..., 1:] = torch.where(x[..., 1:] > 0, 0.25, -0.25) * (x[..., 1:] == x[..., 1:])
    x[..., 0] = 1.0
    c.cells["k"] = x.to(dtype)
    if c.scales:
        c.scales["k"][:] = 1.0
    q = torch.zeros(1, G, T, d)
    q[..., 1:9] = 0.5
    sees = bref.sees_of(bref.random_parents(1, T, seed=74))
    base = bref.attention(c, q.to(BF16), sees, scale=1.0)
    q[..., 0] = off
    o, lse = dfa.decode_tree(c.cuda(), q.to(BF16).cuda(), bref.pack(sees).cuda(), scale=1.0)
    step = 3 * 2.0 ** -23 * abs(off)
    vmax = float(rows_max(c))
    # two steps of the offset's size as below; fp16 weights, the output's rounding
    tol = vmax * (math.expm1(2 * step) + 2.0 ** -10 + 2.0 ** -8)
    assert (o.cpu().double() - base[0]).abs().max() <= tol
    assert (lse.cpu().double() - (base[1] + off)).abs().max() <= 2 * step + 2.0 ** -18


@pytest.mark.parametrize("dtype", [E4M3, BF16])
@pytest.mark.parametrize("far", [1e4, -1e4, 3e7, -3e7])
def test_tree_scores_far_from_zero(dtype, far):
    """A common offset of all scores, exact in fp32, changes nothing but the LSE: it is
    one feature of q times one of all keys."""
    T, d = 3, 64
    c = ref.Cache(dtype, 1, 1, d, 64, 4, [200], seed=19)
    off = 2.0 ** math.floor(math.log2(abs(far)))
    for name in ("k",):
        x = c.cells[name].float()
        x[..., 0] = 1.0 if dtype is BF16 else 1.0
        x[..., 1:] = torch.where(x[..., 1:] > 0, 0.25, -0.25) * (x[..., 1:] == x[..., 1:])
        c.cells[name] = x.to(dtype)
    if c.scales:
        c.scales["k"][:] = 1.0
    q = torch.zeros(1, 2, T, d)
    q[..., 1:9] = 0.5
    sees = bref.sees_of(bref.random_parents(1, T, seed=20))
    scale = 1.0
    base = bref.attention(c, q.to(BF16), sees, scale=scale)
    q[..., 0] = math.copysign(off, far)
    dev = c.cuda()
    o, lse = dfa.decode_tree(dev, q.to(BF16).cuda(), bref.pack(sees).cuda(), scale=scale,
                             out_fp32=True)
    # Scores are off + m / 8, rounded with the sum and once more times log2(e): two steps
    # of the offset's size, which the exponent has absolutely.
    step = 3 * 2.0 ** -23 * off
    ds = min(step, 20.0)
    spread = math.expm1(2 * ds) if ds < 1 else 2.0
    vmax = float(rows_max(c))
    assert (o.cpu().double() - base[0]).abs().max() <= vmax * spread + 2.0 ** -15 * vmax
    assert (lse.cpu().double() - (base[1] + math.copysign(off, far))).abs().max() <= (
        2 * step + 2.0 ** -18)


@pytest.mark.parametrize("dtype", [E4M3, BF16])
def test_tree_scores_of_any_size(dtype):
    """Finite scores of up to 1e38, all negative or not: the largest one's value comes
    out, to its last bit where it is alone."""
    T, d, L = 4, 64, 180
    for sign in (1.0, -1.0):
        c = ref.Cache(dtype, 1, 1, d, 16, 12, [L], seed=21)
        x = torch.zeros_like(c.cells["k"].float())
        order = torch.randperm(L, generator=torch.Generator().manual_seed(1))
        for j in range(L):
            # bf16: all different; 8 bits: few values, of which the largest is one key's
            x[int(c.table[0, j // 16]), 0, j % 16, 0] = sign * (
                1.0 + float(order[j]) / 256 if dtype is BF16 else 1.0 + (order[j] > 0))
        c.cells["k"] = x.to(dtype)
        if c.scales:
            c.scales["k"][:] = 1.0
        q = torch.zeros(1, 1, T, d)
        q[..., 0] = 1e37
        sees = torch.ones(1, T, T, dtype=torch.bool)
        K = bref.rows(c, "k", 0, L)[0, :, 0]
        dev = c.cuda()
        o, lse = dfa.decode_tree(dev, q.to(BF16).cuda(), bref.pack(sees).cuda(), scale=1.0,
                                 out_fp32=True)
        top = K == K.max()
        want = bref.rows(c, "v", 0, L)[0][top].mean(0)
        V = bref.rows(c, "v", 0, L)[0].abs().max()
        assert (o[0, 0].cpu().double() - want).abs().max() <= 2.0 ** -14 * V
        assert lse.isfinite().all()


@pytest.mark.parametrize("loud", [-90.0, -50.0, 50.0, 100.0])
@pytest.mark.parametrize("T", [3, 40])
def test_tree_extreme_value_scales(loud, T):
    """A page whose value scale is far from the others': its weight in the result follows
    the values, the sum of probabilities does not."""
    d, L = 64, 700
    c = ref.Cache(E4M3, 2, 2, d, 64, 11, [L, 640], seed=22)
    for b in range(2):
        c.scales["v"][int(c.table[b, 3])] *= 2.0 ** loud
    q = randn(2, 8, T, d, seed=23)
    sees = bref.sees_of(bref.random_parents(2, T, seed=24))
    check_tree(c, c.cuda(), q, sees)


@pytest.mark.parametrize("G", [2, 40])
@pytest.mark.parametrize("below", [8.0, 14.0, 16.0])
def test_tree_many_small_weights_behind_a_large_one(G, below):
    """One key e^below times the others' weights, in front of them, whose values it does not
    share: what small weights add up to is there."""
    T, d, L = 2, 64, 6000
    c = ref.Cache(E4M3, 1, 1, d, 64, -(-L // 64), [L], seed=75)
    for name in "kv":
        c.scales[name][:] = 1.0
    k, v = torch.zeros_like(c.cells["k"].float()), torch.ones_like(c.cells["v"].float())
    k[int(c.table[0, 0]), 0, 5, 0] = below
    v[int(c.table[0, 0]), 0, 5] = -1.0
    c.cells["k"], c.cells["v"] = k.to(E4M3), v.to(E4M3)
    q = torch.zeros(1, G, T, d)
    q[..., 0] = 1.0
    sees = torch.ones(1, T, T, dtype=torch.bool)
    big, rest = math.exp(below), L - 1.0
    want = (rest - big) / (rest + big)
    for fp32 in (False, True):
        o, lse = dfa.decode_tree(c.cuda(), q.to(BF16).cuda(), bref.pack(sees).cuda(), scale=1.0,
                                 out_fp32=fp32)
        # weights to half a step of fp16's 11 bits, or of its subnormals where the largest is
        # 2^4 (with two terms 2^8) or more; sums cut off at 2^-23 a tile and term
        sub = rest * 2.0 ** -25 / (2.0 ** 8 if fp32 else 2.0 ** 4) * big / (rest + big)
        tol = (2.0 ** -22 if fp32 else 2.0 ** -11) + sub + 4 * 47 * 2.0 ** -23
        tol += 0 if fp32 else 2.0 ** -8 * abs(want)
        assert (o.cpu().double() - want).abs().max() <= tol, fp32
        assert (lse.cpu().double() - math.log(rest + big)).abs().max() <= 1e-5


def test_tree_zero_pages_and_scales_of_the_callers():
    """Pages of zeros with the smallest scale; scales that are no powers of two."""
    c = ref.Cache(E4M3, 1, 1, 128, 16, 10, [150], seed=25)
    for name in "kv":
        pg = int(c.table[0, 2])
        x = c.cells[name].float()
        x[pg] = 0.0
        c.cells[name] = x.to(E4M3)
        c.scales[name][pg] = 2.0 ** -100
        c.scales[name][int(c.table[0, 4])] *= 1.37
    q = randn(1, 4, 6, 128, seed=26)
    check_tree(c, c.cuda(), q, bref.sees_of(bref.random_parents(1, 6, seed=27)))


def test_tree_reports_lengths_and_pages():
    for lens, n, code in (([20, 200], None, 6), ([20, -1], None, 6), ([20, 3], None, 6),
                          ([20, 60], [4, 5], 6), ([20, 60], [4, -1], 6)):
        c = ref.Cache(BF16, 2, 1, 64, 16, 4, [20, 60], seed=28)
        c.lens = i32(lens, "cpu")
        dev = c.cuda()
        q = randn(2, 2, 4, 64, seed=29)
        sees = bref.sees_of(bref.random_parents(2, 4, seed=30))
        o, lse = dfa.decode_tree(dev, q.cuda(), bref.pack(sees).cuda(), q_lens=i32(n))
        with pytest.raises(dfa.DfaError) as e:
            dfa.stream_status(dev.status)
        assert e.value.code == code
        c.lens = i32([20, 60], "cpu")
        O, LSE, tO, tL = bref.attention(c, q, sees)
        ref.check(o[0], O[0], tO[0], BF16)             # the others' are right
    for page in (-1, 10 ** 6):
        c = ref.Cache(E4M3, 2, 1, 64, 16, 4, [20, 60], seed=28)
        c.table[1, 2] = page
        dev = c.cuda()
        o, lse = dfa.decode_tree(dev, q.cuda(), bref.pack(sees).cuda())
        with pytest.raises(dfa.DfaError) as e:
            dfa.stream_status(dev.status)
        assert e.value.code == 6
        O, LSE, tO, tL = bref.attention(
            ref.Cache(E4M3, 2, 1, 64, 16, 4, [20, 60], seed=28), q, sees)
        ref.check(o[0], O[0], tO[0], BF16)


def test_tree_captured_and_replayed_as_sequences_grow():
    c = ref.Cache(E4M3, 2, 2, 128, 64, 40, [2500, 2000], seed=31)
    full = c.lens.clone()
    c.lens = i32([300, 10], "cpu")
    dev = c.cuda()
    T = 7
    q = randn(2, 8, T, 128, seed=32)
    sees = bref.sees_of(bref.random_parents(2, T, seed=33))
    parents = torch.zeros(2, T, dtype=torch.int32, device="cuda")
    ws = dfa.tree_workspace(dev, 8, T)
    qd = q.cuda()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        mask, pos = dfa.tree_plan(dev, parents, ws=ws)
        o, lse = dfa.decode_tree(dev, qd, mask, ws=ws)
    par = bref.random_parents(2, T, seed=33)
    parents.copy_(par)
    for lens in ([300, 10], [2500, 777], full.tolist()):
        dev.seq_lens.copy_(i32(lens))
        g.replay()
        dfa.stream_status(ws)
        c.lens = i32(lens, "cpu")
        O, LSE, tO, tL = bref.attention(c, q, sees)
        ref.check(o, O, tO, BF16, lens)
        ref.check(lse, LSE, tL, torch.float32, lens)
        assert torch.equal(pos.cpu().long(), i32(lens, "cpu")[:, None] - T + sees.sum(-1) - 1)


@pytest.mark.parametrize("dtype", [E4M3, BF16])
@pytest.mark.parametrize("G,T,d", [(2, 3, 64), (5, 16, 128)])
def test_tree_sequences_of_no_rows_to_several_tiles(dtype, G, T, d):
    """More sequences than blocks, so that blocks go from one short segment to the next;
    sequences without a node between them."""
    B, page, width = 240, 32, 16
    g = torch.Generator().manual_seed(d)
    lens = [int(x) for x in torch.randint(0, 400, (B,), generator=g)]
    lens[40:80] = [int(x) for x in torch.randint(1, 40, (40,), generator=g)]
    n = [min(L, int(x)) for L, x in zip(lens, torch.randint(0, T + 1, (B,), generator=g))]
    n[100:120] = [0] * 20
    c = ref.Cache(dtype, 1, 1, d, page, width, [512], seed=d)
    c.B, c.table, c.lens = B, c.table.repeat(B, 1), i32(lens, "cpu")   # (the same pages)
    q = randn(B, G, T, d, seed=60)
    sees = bref.sees_of(bref.random_parents(B, T, seed=61))
    check_tree(c, c.cuda(), q, sees, n, fp32=(G == 5,))


def test_tree_graphs_that_share_a_workspace():
    """One workspace, made for the larger of two calls, in two graphs replayed in turn."""
    calls, graphs = [], []
    for dtype, G, T, L in ((E4M3, 4, 30, 4000), (BF16, 1, 3, 900)):
        c = ref.Cache(dtype, 2, 2, 128, 64, 64, [L, L // 3], seed=L)
        sees = bref.sees_of(bref.random_parents(2, T, seed=T))
        calls.append((c.cuda(), randn(2, 2 * G, T, 128, seed=62).cuda(), bref.pack(sees).cuda()))
    want = [dfa.decode_tree(*a) for a in calls]
    ws = dfa.tree_workspace(calls[0][0], 8, 30)
    for a in calls:
        graphs.append((torch.cuda.CUDAGraph(), []))
        with torch.cuda.graph(graphs[-1][0]):
            graphs[-1][1].extend(dfa.decode_tree(*a, ws=ws))
    for _ in range(3):
        for (g, got), (o, lse) in zip(graphs, want):
            got[0].zero_()
            g.replay()
            assert torch.equal(got[0], o) and torch.equal(got[1], lse)
    dfa.stream_status(ws)


def test_tree_on_two_streams_at_once():
    c = ref.Cache(BF16, 4, 4, 128, 32, 100, [3000, 2000, 1000, 17], seed=34)
    dev = c.cuda()
    T = 9
    sees = bref.sees_of(bref.random_parents(4, T, seed=35))
    mask = bref.pack(sees).cuda()
    qs = [randn(4, 8, T, 128, seed=36 + i).cuda() for i in range(2)]
    want = [dfa.decode_tree(dev, q, mask) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    for _ in range(20):
        got = [dfa.decode_tree(dev, q, mask, stream=s) for q, s in zip(qs, streams)]
    torch.cuda.synchronize()
    for (a, la), (b, lb) in zip(got, want):
        assert torch.equal(a, b) and torch.equal(la, lb)      # the same bits, whoever runs beside
    dfa.stream_status(dev.status)


# ---------------------------------------------------------------------------
# positions of appended rows
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [E4M3, BF16])
@pytest.mark.parametrize("layout,rot", [("half", 64), ("interleaved", 32)])
def test_append_at_positions(dtype, layout, rot):
    """Rows rotated where the caller says and stored where they belong: the same cells as
    keys rotated apart and stored as they are (bf16: to the bit; 8 bits: once rounded)."""
    B, H, Hq, T, d, page = 3, 2, 4, 21, 64, 16
    lens, new = [50, 21, 40], [21, 20, 0]
    c = ref.Cache(dtype, B, H, d, page, 4, lens, seed=40)
    dev = c.cuda()
    k, v, q = (randn(B, h, T, d, seed=41 + h) for h in (H, H, Hq))
    pos = torch.randint(-5, 10 ** 6, (B, T), generator=torch.Generator().manual_seed(44),
                        dtype=torch.int32)
    out = torch.full((B, Hq, T, d), 7.0, dtype=BF16, device="cuda")
    ws = dfa.paged_workspace(dev)
    spec = dfa.rope_spec(d, layout=layout, rot_dim=rot)
    dfa.cache_append(dev, k.cuda(), v.cuda(), rope=spec, new_lens=i32(new), q=q.cuda(), q_out=out,
                     ws=ws, positions=pos.cuda())
    dfa.stream_status(ws)
    for b in range(B):
        n, L = new[b], lens[b]
        want = ref.rope(q[b, :, :n], pos[b, :n], layout, rot)
        ref.check(out[b, :, :n], want, ref.rope_tol(q[b, :, :n], rot, BF16, layout), BF16)
        assert (out[b, :, n:] == 7).all()
        want = ref.rope(k[b, :, :n], pos[b, :n], layout, rot)
        tol = ref.rope_tol(k[b, :, :n], rot, BF16, layout)
        j = torch.arange(L - n, L)
        pg = c.table[b, j // page].long()
        for name, w, t in (("k", want, tol), ("v", v[b, :, :n].double(), 0 * tol)):
            got = getattr(dev, name).float().cpu()[pg, :, j % page].double().transpose(0, 1)
            s = torch.ones(H, n, 1, dtype=torch.float64)
            if dtype is E4M3:
                s = getattr(dev, name + "_scale").cpu()[pg].t()[..., None].double()
            # half a step, or of the subnormals
            bad = (got * s - w).abs() > t + ref.HALF_STEP[dtype] * (w.abs() + t) + (
                s * 2.0 ** -10 if dtype is E4M3 else 0)
            assert not bad.any(), (name, b)


# ---------------------------------------------------------------------------
# kept rows
# ---------------------------------------------------------------------------
def check_compact(c, kept, kept_lens, q_lens, T=None, pass_lens=True):
    dev = c.cuda()
    ws = dfa.paged_workspace(dev)
    dfa.cache_compact(dev, kept.cuda(), i32(kept_lens) if pass_lens else None,
                      q_lens=None if q_lens is None else i32(q_lens), T=T, ws=ws)
    dfa.stream_status(ws)
    n = [T] * c.B if q_lens is None else q_lens
    want = bref.compact(c, kept, kept_lens, n)
    for name in "kv":
        cells, scales = want[name]
        got = getattr(dev, name).cpu()
        if scales is not None:
            assert torch.equal(getattr(dev, name + "_scale").cpu(), scales)
        same = (got.float() == cells) | (got.float().isnan() & cells.isnan())
        for b in range(c.B):                 # behind the last kept row: no meaning
            for j in range(int(c.lens[b]) - n[b] + kept_lens[b], c.table.shape[1] * c.page):
                same[int(c.table[b, j // c.page]), :, j % c.page] = True
        assert same.all(), (name, (~same).nonzero()[:5].tolist())
    return dev


def some(n, a, seed):
    return torch.randperm(n, generator=torch.Generator().manual_seed(seed))[:a].sort().values


@pytest.mark.parametrize("dtype", [E4M3, BF16])
@pytest.mark.parametrize("page,d", [(16, 64), (16, 128), (32, 64), (64, 128), (128, 64),
                                    (128, 128)])
def test_compact(dtype, page, d):
    """Paths of a tree and thinned contexts: from none to all of the rows, over one page and
    many, from any row of a page on."""
    lens = [300, 40, 130, 257, 16, 1, 200, 300]
    n = [300, 7, 130, 20, 16, 1, 64, 299]
    a = [150, 3, 130, 0, 5, 1, 1, 298]
    c = ref.Cache(dtype, 8, 2, d, page, -(-300 // page), lens, seed=page)
    kept = torch.zeros(8, 300, dtype=torch.int32)
    for b in range(8):
        kept[b, :a[b]] = some(n[b], a[b], b)
    check_compact(c, kept, a, n)


@pytest.mark.parametrize("dtype,page,d", [(E4M3, 16, 128), (E4M3, 128, 64), (BF16, 64, 128),
                                          (BF16, 32, 64)])
def test_compact_long(dtype, page, d):
    """Several batches of rows, the first of which stay; scales that go up and down."""
    lens, n, a = [2900, 1500], [2877, 1500], [2000, 1499]
    c = ref.Cache(dtype, 2, 1, d, page, -(-2900 // page), lens, seed=63)
    if dtype is E4M3:
        g = torch.Generator().manual_seed(64)
        for name in "kv":
            c.scales[name] *= 2.0 ** torch.randint(-4, 5, c.scales[name].shape, generator=g)
    kept = torch.zeros(2, 2000, dtype=torch.int32)
    kept[0, :40] = torch.arange(40)
    kept[0, 40:2000] = 40 + some(n[0] - 40, 1960, 65)
    kept[1, :1499] = some(1500, 1499, 66)
    check_compact(c, kept, a, n)


def test_compact_needs_no_counts():
    c = ref.Cache(BF16, 2, 1, 64, 16, 4, [50, 33], seed=50)
    kept = torch.tensor([[0, 2, 5], [1, 3, 7]], dtype=torch.int32)
    check_compact(c, kept, [3, 3], None, T=8, pass_lens=False)


def test_compact_pages_of_different_scales():
    """Rows from a loud page raise a quiet one's scale, the rows that stay with it."""
    for loud in (-20, -3, 3, 9, 30):
        c = ref.Cache(E4M3, 1, 2, 64, 16, 6, [90], seed=51)
        for p in range(6):
            for name in "kv":
                c.scales[name][int(c.table[0, p])] *= 2.0 ** (loud * (p % 3))
        kept = torch.zeros(1, 60, dtype=torch.int32)
        kept[0, :25] = some(85, 25, 52)
        check_compact(c, kept, [25], [85])


def test_compact_reports_bad_lists():
    for lists, a, n in (([3, 3, 4], 3, 8), ([4, 3, 5], 3, 8), ([-1, 2, 3], 3, 8),
                        ([0, 1, 8], 3, 8), ([0, 1, 2], 4, 8), ([0, 1, 2], -1, 8),
                        ([0, 1, 2], 3, 2), ([0, 1, 2], 3, 60), ([0, 1, 2], 3, -1)):
        for dtype in (BF16, E4M3):
            c = ref.Cache(dtype, 2, 1, 64, 16, 4, [40, 40], seed=53)
            dev = c.cuda()
            before = {m: getattr(dev, m).clone() for m in "kv"}
            kept = torch.tensor([[1, 5, 6], lists], dtype=torch.int32)
            dfa.cache_compact(dev, kept.cuda(), i32([3, a]), q_lens=i32([8, n]))
            with pytest.raises(dfa.DfaError) as e:
                dfa.stream_status(dev.status)
            assert e.value.code == 6
            for name in "kv":                # sequence 0 moved, sequence 1 did not
                now, was = getattr(dev, name), before[name]
                for p in c.table[1].tolist():
                    assert torch.equal(now[p].view(torch.uint8), was[p].view(torch.uint8))
                p = c.table[0].tolist()
                assert torch.equal(now[p[2], :, 0].view(torch.uint8),
                                   was[p[2], :, 1].view(torch.uint8))


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [E4M3, BF16])
def test_a_step_of_speculative_decoding(dtype):
    """Tree appended and attended to, the accepted path moved behind the context, rejected
    pages given back; then the next token sees what it would have seen had the path been
    appended alone."""
    B, Hkv, G, d, page, T = 3, 2, 2, 64, 16, 13
    ctx = [37, 0, 90]
    spec = dfa.rope_spec(d, layout="half")
    width = 10
    npages = B * width + 1
    kw, cells = {}, []
    for _ in range(2):
        cells.append(torch.zeros(npages, Hkv, page, d, device="cuda").to(dtype))
    if dtype is E4M3:
        kw = {n: torch.ones(npages, Hkv, device="cuda") for n in ("k_scale", "v_scale")}
    table = torch.zeros(B, width, dtype=torch.int32, device="cuda")
    lens = i32(ctx)
    pool = dfa.PagePool(table, lens, page, npages=npages)
    cache = dfa.PagedCache(*cells, table, lens, **kw)
    ws = dfa.tree_workspace(cache, Hkv * G, max(ctx))
    # the contexts
    k0, v0 = randn(B, Hkv, max(ctx), d, seed=60), randn(B, Hkv, max(ctx), d, seed=61)
    dfa.pages_reserve(pool, max(ctx), new_lens=i32(ctx))
    dfa.cache_append(cache, k0.cuda(), v0.cuda(), rope=spec, new_lens=i32(ctx), ws=ws)
    # the trees
    parents = bref.random_parents(B, T, seed=62, roots=0.0)
    sees = bref.sees_of(parents)
    n = [13, 13, 6]
    lens += i32(n)
    jobs, info = dfa.pages_reserve(pool, T, new_lens=i32(n))
    assert info.tolist()[0] == 0 and info.tolist()[2] == 0
    mask, pos = dfa.tree_plan(cache, parents.cuda(), q_lens=i32(n), ws=ws)
    k1, v1, q1 = (randn(B, h, T, d, seed=63 + i) for i, h in enumerate((Hkv, Hkv, Hkv * G)))
    q = dfa.cache_append(cache, k1.cuda(), v1.cuda(), rope=spec, new_lens=i32(n), q=q1.cuda(),
                         ws=ws, positions=pos)
    o, lse = dfa.decode_tree(cache, q, mask, q_lens=i32(n), ws=ws)
    dfa.stream_status(ws)
    # the path to one of the last nodes, by hand
    kept = torch.zeros(B, T, dtype=torch.int32)
    a = []
    for b in range(B):
        path = sees[b, n[b] - 1, :n[b]].nonzero()[:, 0]
        a.append(len(path))
        kept[b, :a[b]] = path
    dfa.cache_compact(cache, kept.cuda(), i32(a), q_lens=i32(n), T=T, ws=ws)
    lens.copy_(i32([c + x for c, x in zip(ctx, a)]))
    dfa.pages_trim(pool)
    assert pool.held.tolist() == [-(-(c + x) // page) for c, x in zip(ctx, a)]
    assert int(pool.refs.sum()) == int(pool.held.sum())
    # the same contexts and paths in a cache of their own, appended as chains
    other = dfa.PagedCache(*(torch.zeros_like(x) for x in cells),
                           torch.arange(B * width, dtype=torch.int32, device="cuda").view(B, -1),
                           i32(ctx), **{m: torch.ones_like(x) for m, x in kw.items()})
    dfa.cache_append(other, k0.cuda(), v0.cuda(), rope=spec, new_lens=i32(ctx))
    other.seq_lens.copy_(lens)
    kp, vp, qp = (torch.zeros(B, x.shape[1], max(a), d, dtype=BF16) for x in (k1, v1, q1))
    for b in range(B):
        for x, y in ((k1, kp), (v1, vp), (q1, qp)):
            y[b, :, :a[b]] = x[b][:, kept[b, :a[b]].long()]
    qc = dfa.cache_append(other, kp.cuda(), vp.cuda(), rope=spec, new_lens=i32(a), q=qp.cuda())
    oc, lc = dfa.decode_paged(other, qc, q_lens=i32(a))
    top = int(lens.max())
    got, want = dfa.cache_gather(cache, top), dfa.cache_gather(other, top)
    for b in range(B):
        L = int(lens[b])
        for x, y in zip(got, want):
            x, y = x[b, :, :L].float(), y[b, :, :L].float()
            # 8 bits: pages whose scales rose with rejected nodes round on coarser steps
            assert (x - y).abs().max() <= (0 if dtype is BF16 else 2 * 2.0 ** -3 * 5)
            if dtype is BF16:
                assert torch.equal(x, y)
    # the path's nodes saw what the chain's tokens see
    for b in range(B):
        x = o[b][:, kept[b, :a[b]].long().cuda()].float()
        y = oc[b, :, :a[b]].float()
        big = 2.0 ** -7 * (x.abs() + y.abs()) + 2.0 ** -9
        if dtype is BF16:
            assert ((x - y).abs() <= big).all()
    dfa.stream_status(ws)
    dfa.stream_status(pool.status)
