"""GPU parity of rotary positions and of the paged cache (append, gather,
decode) against plain fp64 forms: both pair layouts, part of the head, scaled
frequencies, strided rows, bf16 and e4m3 cells, every page size, ragged and
empty sequences, NaN wherever no sequence may look, refused arguments, graphs,
and the calls together as a serving loop uses them."""
import math

import pytest
import torch

import paged_ref as ref
from long_context_flashattention_gb300 import dfa

pytestmark = pytest.mark.gpu
BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn
BANDS = dict(scaling="bands", factor=8.0, orig_len=512.0, low=1.0, high=4.0, gain=1.25)
LINEAR = dict(scaling="linear", factor=4.0)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    dfa.lib()
    yield
    torch.cuda.synchronize()


def randn(*shape, seed=0, dtype=BF16):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def spec_of(d, layout, rot, kw):
    return dfa.rope_spec(d, layout=layout, rot_dim=rot, **kw)


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------
def check_rope(got, x, pos, layout, rot, inverse, kw):
    gain = kw.get("gain", 1.0)
    want = ref.rope(x, pos, layout, rot, inverse, **kw)
    ref.check(got, want, ref.rope_tol(x, rot, x.dtype, layout, gain), x.dtype, "rope")
    assert torch.equal(got.cpu()[..., rot:], x[..., rot:])


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("dtype", [BF16, torch.float32])
@pytest.mark.parametrize("B,H,L,d,rot,kw", [
    (1, 1, 1, 64, 64, {}),
    (2, 3, 37, 128, 128, {}),
    (1, 40, 5, 128, 64, LINEAR),
    (3, 8, 130, 64, 16, BANDS),
    (1, 5, 257, 128, 96, BANDS),
    (1, 2, 4099, 64, 48, LINEAR),
])
def test_rope_matches_fp64(layout, dtype, B, H, L, d, rot, kw):
    x = randn(B, H, L, d, seed=L, dtype=dtype)
    spec = spec_of(d, layout, rot, kw)
    for inverse in (False, True):
        got = dfa.rope(x.cuda(), spec, inverse=inverse)
        check_rope(got, x, torch.arange(L), layout, rot, inverse, kw)


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_rope_positions_far_and_negative(layout):
    """Any int32 position: the angle is reduced exactly."""
    pos = torch.tensor([[0, 1, 131071, 524287, 2 ** 24 + 1, 2 ** 31 - 1, -1, -2 ** 31]],
                       dtype=torch.int32)
    x = randn(1, 2, 8, 128, seed=3, dtype=torch.float32)
    got = dfa.rope(x.cuda(), dfa.rope_spec(128, layout=layout), positions=pos.cuda())
    want = ref.rope(x, pos[:, None], layout, 128)
    # a frequency is rounded three times in fp64 on each side (pow, the division
    # by 2 pi, the product): 2^31 positions times 6 half-steps of 2^-53
    tol = ref.rope_tol(x, 128, x.dtype, layout) + 2.0 ** 31 * 6 * 2.0 ** -53 * 2 * x.abs().max()
    ref.check(got, want, tol, x.dtype)


@pytest.mark.parametrize("dtype", [BF16, torch.float32])
@pytest.mark.parametrize("d,rot", [(64, 64), (128, 128), (128, 32)])
@pytest.mark.parametrize("H", [1, 2, 3, 4, 5, 6, 8, 9, 16, 17])
def test_rope_few_heads_at_positions_of_their_own(H, d, rot, dtype):
    """Lanes that heads do not take go to other tokens, whose positions differ; an
    odd number of tokens, input and output strided differently."""
    B, L = 3, 67
    x = randn(B, L, H, d, seed=H, dtype=dtype).transpose(1, 2)
    pos = torch.randint(-1000, 100000, (B, L), generator=torch.Generator().manual_seed(H),
                        dtype=torch.int32)
    out = torch.full((B, H + 1, L, d), 7.0, dtype=dtype, device="cuda")
    dfa.rope(x.cuda(), dfa.rope_spec(d, layout="half", rot_dim=rot, **BANDS), positions=pos.cuda(),
             out=out[:, :H])
    check_rope(out[:, :H], x, pos[:, None], "half", rot, False, BANDS)
    assert (out[:, H] == 7).all()


@pytest.mark.parametrize("kind,P,stripe", [("striped", 8, 1), ("striped", 4, 16),
                                           ("balanced", 4, 1), ("contiguous", 4, 1)])
def test_rope_at_a_workers_positions(orc, kind, P, stripe):
    N, p = 1024, P - 1
    x = randn(1, 3, N // P, 128, seed=5)
    m = dfa.partition_map(N, P, p, kind, stripe)
    got = dfa.rope(x.cuda(), dfa.rope_spec(128, layout="half"), pos_map=m)
    pos = torch.from_numpy(orc.partition_pos(kind, N, P, p, stripe))
    check_rope(got, x, pos, "half", 128, False, {})


def test_rope_equals_permute_rope_on_natural_order():
    x = randn(2, 4, 512, 128, seed=6)
    a = dfa.permute_rope(x.cuda(), 1, "contiguous").float().cpu()
    b = dfa.rope(x.cuda(), dfa.rope_spec(128)).float().cpu()
    # Both round an fp32 value that is within rope_tol of the exact one (the
    # permute's angle is an fp64 remainder in [-pi, pi] rounded to fp32, half a
    # step pi 2^-25 as here): the two values are 2 rope_tol apart (all that is
    # left where x cos and y sin cancel), and rounding adds half a step, 2^-8, of
    # each.
    tol = 2 * ref.rope_tol(x, 128, BF16, "interleaved") + 2.0 ** -8 * (a.abs() + b.abs())
    bad = (a - b).abs() > tol
    assert not bad.any(), int(bad.sum())


@pytest.mark.parametrize("layout,rot", [("half", 128), ("half", 64), ("interleaved", 32)])
def test_rope_in_place_on_a_packed_projection(layout, rot):
    """Query and key heads of one [B, L, H, d] buffer, strided in and out; the
    value heads behind them are not touched."""
    B, L, Hq, Hkv, d = 2, 19, 6, 2, 128
    qkv = randn(B, L, Hq + 2 * Hkv, d, seed=7)
    dev = qkv.cuda()
    qk = dev.transpose(1, 2)[:, :Hq + Hkv]
    got = dfa.rope(qk, dfa.rope_spec(d, layout=layout, rot_dim=rot), out=qk)
    assert got is qk
    x = qkv.transpose(1, 2)[:, :Hq + Hkv]
    check_rope(got, x, torch.arange(L), layout, rot, False, {})
    assert torch.equal(dev[:, :, Hq + Hkv:].cpu(), qkv[:, :, Hq + Hkv:])


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_rope_inverse_is_the_gradient(layout):
    """<rope(x + h e) - rope(x - h e), w> / 2h over random directions equals
    <e, inverse(w)>: the map is linear, so the difference is exact up to fp32."""
    d, rot, L, kw = 64, 32, 33, BANDS
    spec = spec_of(d, layout, rot, kw)
    x, e, w = (randn(1, 2, L, d, seed=s, dtype=torch.float32).cuda() for s in (8, 9, 10))
    h = 0.5
    num = ((dfa.rope(x + h * e, spec) - dfa.rope(x - h * e, spec)).double() * w.double()).sum()
    ana = (e.double() * dfa.rope(w, spec, inverse=True).double()).sum()
    # each of 2 L d terms carries at most a few 1e-6 (|x| up to 5, 1 / 2h = 1)
    assert abs(float(num / (2 * h) - ana)) <= 2 * L * d * 5 * 5 * 1e-6


def test_rope_broadcast_input_and_empty():
    x = randn(1, 1, 9, 64, seed=11).cuda().expand(3, 4, 9, 64)
    spec = dfa.rope_spec(64, layout="half")
    check_rope(dfa.rope(x, spec), x.cpu(), torch.arange(9), "half", 64, False, {})
    e = torch.empty(2, 3, 0, 64, dtype=BF16, device="cuda")
    assert dfa.rope(e, spec).shape == e.shape


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------
def run_append(c, T, new, layout=None, rot=None, kw={}, Hq=0, seed=20, k=None, v=None):
    """Append on the GPU and check every cell of the cache, the scales and q_out."""
    B, H, d, page = c.B, c.Hkv, c.d, c.page
    k = randn(B, T, H, d, seed=seed) if k is None else k
    v = randn(B, T, H, d, seed=seed + 1) if v is None else v
    q = randn(B, T, Hq, d, seed=seed + 2) if Hq else None
    news = [T] * B if new is None else new
    for b in range(B):  # rows that are not the sequence's must not be read
        k[b, news[b]:] = v[b, news[b]:] = float("nan")
    dev = c.cuda()
    spec = spec_of(d, layout, rot, kw) if layout else None
    new_lens = None if new is None else torch.tensor(new, dtype=torch.int32, device="cuda")
    q_out = torch.full((B, Hq, T, d), 7.0, dtype=BF16, device="cuda") if Hq else None
    ws = dfa.paged_workspace(dev)
    for _ in range(2):  # the same rows again give the same cells
        r = dfa.cache_append(dev, k.cuda().transpose(1, 2), v.cuda().transpose(1, 2), rope=spec,
                             new_lens=new_lens, q=q.cuda().transpose(1, 2) if Hq else None,
                             q_out=q_out, ws=ws)
        dfa.stream_status(ws)
        assert r is q_out
        check_append(c, dev, k, v, news, layout, rot, kw)
    for b in range(B if Hq else 0):
        pos = torch.arange(int(c.lens[b]) - news[b], int(c.lens[b]))
        got = q_out[b].cpu()
        check_rope(got[:, :news[b]], q[b, :news[b]].transpose(0, 1), pos, layout, rot, False, kw)
        assert (got[:, news[b]:] == 7.0).all()
    return dev


def check_append(c, dev, k, v, news, layout, rot, kw):
    page, E = c.page, c.dtype
    gain = kw.get("gain", 1.0)
    for name, x in (("k", k), ("v", v)):
        want = c.cells[name].double()
        tol = torch.zeros_like(want)
        scales = c.scales[name].double().clone() if c.scales else None
        got = getattr(dev, name).cpu()
        for b in range(c.B):
            n, L = news[b], int(c.lens[b])
            rows = x[b, :n].transpose(0, 1)
            vals, t = rows.double(), torch.zeros(rows.shape, dtype=torch.float64)
            if name == "k" and layout:
                pos = torch.arange(L - n, L)
                vals = ref.rope(rows, pos, layout, rot, **kw)
                t = ref.rope_tol(rows, rot, BF16, layout, gain)
            for p in range((L - n) // page, -(-L // page)):
                lo, hi = max(L - n, p * page), min(L, (p + 1) * page)
                if lo >= hi:
                    continue
                pg, at = int(c.table[b, p]), slice(lo - p * page, hi - p * page)
                part, tp = vals[:, lo - (L - n):hi - (L - n)], t[:, lo - (L - n):hi - (L - n)]
                if E is BF16:
                    want[pg, :, at], tol[pg, :, at] = part, tp
                    continue
                for h in range(c.Hkv):
                    fin = part[h][part[h].isfinite()].abs()
                    s = ref.pow2_scale(float(fin.max()) if fin.numel() else 0.0)
                    old = float(scales[pg, h])
                    if lo > p * page:
                        s = max(s, old)
                        want[pg, h, :at.start] *= old / s
                        if s > old:  # requantised: half a step, or of the subnormals
                            w = want[pg, h, :at.start]
                            tol[pg, h, :at.start] = 2.0 ** -10
                    scales[pg, h] = s
                    cells = part[h] / s
                    want[pg, h, at] = torch.where(cells.isfinite(), cells,
                                                  torch.tensor(float("nan"), dtype=torch.float64))
                    tol[pg, h, at] = tp[h] / s + 2.0 ** -10
        if scales is not None:
            assert torch.equal(getattr(dev, name + "_scale").cpu().double(), scales)
        ref.check(got, want, tol, E, name)
        if name == "v" and E is BF16:
            assert torch.equal(got.view(torch.int16)[~got.isnan()],
                               want.to(BF16).view(torch.int16)[~got.isnan()])


@pytest.mark.parametrize("dtype", [E4M3, BF16])
@pytest.mark.parametrize("page,d", [(16, 64), (16, 128), (32, 128), (64, 64), (64, 128),
                                    (128, 64), (128, 128)])
def test_append_one_token(dtype, page, d):
    """One token into fresh pages, into the middle and onto the last row of one."""
    lens = [1, page // 2, page, page + 1, 2 * page]
    c = ref.Cache(dtype, 5, 2, d, page, 2, lens, seed=page + d)
    run_append(c, 1, None, "half", d, {}, Hq=6)


@pytest.mark.parametrize("dtype", [E4M3, BF16])
@pytest.mark.parametrize("layout,rot,kw", [("interleaved", 32, {}), ("half", 64, BANDS),
                                           (None, None, {})])
def test_append_ragged(dtype, layout, rot, kw):
    """Zero to 150 new rows a sequence, pages that begin, fill and end anywhere."""
    new = [0, 1, 15, 16, 17, 150, 33]
    lens = [40, 1, 15, 48, 100, 150, 34]
    c = ref.Cache(dtype, 7, 3, 64, 32, 5, lens, seed=22)
    run_append(c, 150, new, layout, rot, kw, Hq=6 if layout else 0)


def test_append_raises_a_pages_scale():
    """Ever louder rows into one page: the rows that are there are requantised,
    and every power of two between is met."""
    for step in range(0, 14, 3):
        c = ref.Cache(E4M3, 1, 2, 64, 16, 1, [9], seed=step)
        v = randn(1, 1, 2, 64, seed=step) * 2.0 ** step
        run_append(c, 1, None, v=v)


def test_append_extremes():
    """All zeros, the smallest and largest magnitudes, values on the scale's
    border (448 is 1.75 * 2^8), infinities and NaN."""
    for i, x in enumerate([0.0, 2.0 ** -120, 2.0 ** -108, 1.75, 1.765625, 448.0, 3.0e38, 3.5e-4]):
        c = ref.Cache(E4M3, 1, 1, 64, 16, 1, [2], seed=i)
        v = randn(1, 2, 1, 64, seed=i).clamp(-1, 1) * min(x, 1e38)
        v[0, 1, 0, 5] = x
        run_append(c, 2, None, v=v)
    c = ref.Cache(E4M3, 1, 1, 64, 16, 1, [3], seed=9)
    v = randn(1, 3, 1, 64, seed=9)
    v[0, 0, 0, 3], v[0, 1, 0, 4], v[0, 2, 0, 5] = float("inf"), float("nan"), -float("inf")
    dev = run_append(c, 3, None, v=v)
    cells = dev.v[int(c.table[0, 0]), 0].float()
    assert cells[0, 3].isnan() and cells[1, 4].isnan() and cells[2, 5].isnan()
    assert cells[:3].isnan().sum() == 3


def test_append_pages_of_one_tensor():
    """K and V as the halves of one [npages, 2, Hkv, page, d] tensor."""
    c = ref.Cache(E4M3, 2, 2, 128, 16, 3, [20, 41], seed=30)
    both = torch.stack((c.cells["k"].float(), c.cells["v"].float()), 1).to(E4M3).cuda()
    dev = dfa.PagedCache(both[:, 0], both[:, 1], c.table.cuda(), c.lens.cuda(),
                         k_scale=c.scales["k"].cuda(), v_scale=c.scales["v"].cuda())
    k, v = randn(2, 20, 2, 128, seed=31), randn(2, 20, 2, 128, seed=32)
    dfa.cache_append(dev, k.cuda().transpose(1, 2), v.cuda().transpose(1, 2))
    check_append(c, dev, k, v, [20, 20], None, None, {})
    q = randn(2, 4, 1, 128, seed=33)
    c.cells["k"], c.cells["v"] = both[:, 0].cpu(), both[:, 1].cpu()
    c.scales = {"k": dev.k_scale.cpu(), "v": dev.v_scale.cpu()}
    check_decode(c, dev, q)


def test_append_q_in_place():
    c = ref.Cache(E4M3, 2, 2, 64, 16, 2, [5, 17], seed=34)
    dev = c.cuda()
    k, v, q = (randn(2, h, 3, 64, seed=35 + h) for h in (2, 2, 4))
    buf = q.cuda()
    new = torch.tensor([3, 2], dtype=torch.int32, device="cuda")
    spec = dfa.rope_spec(64, layout="half", rot_dim=32)
    out = dfa.cache_append(dev, k.cuda(), v.cuda(), rope=spec, new_lens=new, q=buf, q_out=buf)
    assert out is buf
    check_rope(buf[0].cpu(), q[0], torch.tensor([2, 3, 4]), "half", 32, False, {})
    check_rope(buf[1, :, :2].cpu(), q[1, :, :2], torch.tensor([15, 16]), "half", 32, False, {})
    assert torch.equal(buf[1, :, 2].cpu(), q[1, :, 2])


# ---------------------------------------------------------------------------
# gather
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [E4M3, BF16])
@pytest.mark.parametrize("page,d,pos0,L", [(16, 64, 0, 100), (16, 128, 7, 40), (64, 128, 63, 2),
                                           (128, 64, 0, 256), (32, 64, 90, 64), (32, 64, 500, 5)])
def test_gather_is_exact(dtype, page, d, pos0, L):
    lens = [0, 1, 63, 100]
    c = ref.Cache(dtype, 4, 2, d, page, -(-128 // page), lens, seed=40)
    dev = c.cuda()
    ws = dfa.paged_workspace(dev)
    outs = [torch.full((4, 2, L, d), 7.0, dtype=BF16, device="cuda") for _ in range(2)]
    got = dfa.cache_gather(dev, L, pos0=pos0, k_out=outs[0], v_out=outs[1], ws=ws)
    dfa.stream_status(ws)
    for name, o in zip("kv", got):
        want = torch.full((4, 2, L, d), 7.0, dtype=torch.float64)
        for b in range(4):
            n = min(lens[b], pos0 + L)
            if n > pos0:
                want[b, :, :n - pos0] = c.rows(name, b, n)[:, pos0:]
        assert torch.equal(o.cpu().double(), want)


# ---------------------------------------------------------------------------
# decode
# ---------------------------------------------------------------------------
def check_decode(c, dev, q, q_lens=None, causal=True, scale=None):
    B, Hq, T, d = q.shape
    O, LSE, tO, tL = ref.attention(c, q, q_lens, causal, scale)
    ql = None if q_lens is None else torch.tensor(q_lens, dtype=torch.int32, device="cuda")
    ws = dfa.paged_workspace(dev, Hq, T)
    for fp32 in (False, True):
        dt = torch.float32 if fp32 else BF16
        out = torch.full((B, Hq, T, d), 7.0, dtype=dt, device="cuda")
        lse = torch.full((B, Hq, T), 7.0, device="cuda")
        dfa.decode_paged(dev, q.cuda(), q_lens=ql, causal=causal, scale=scale, out_fp32=fp32,
                         out=out, lse=lse, ws=ws)
        dfa.stream_status(ws)
        for b in range(B):
            n = T if q_lens is None else q_lens[b]
            assert (out[b, :, n:] == 7.0).all() and (lse[b, :, n:] == 7.0).all()
            ref.check(out[b, :, :n], O[b, :, :n], tO[b, :, :n], dt, ("O", b))
            ref.check(lse[b, :, :n], LSE[b, :, :n], tL[b, :, :n], torch.float32, ("LSE", b))


@pytest.mark.parametrize("dtype", [E4M3, BF16])
@pytest.mark.parametrize("B,Hq,Hkv,T,d,page,lens,q_lens,causal", [
    (1, 1, 1, 1, 64, 16, [1], None, True),
    (1, 4, 1, 1, 128, 16, [15], None, True),
    (3, 8, 2, 1, 128, 64, [0, 64, 333], None, True),     # a sequence without rows: refused rows
    (2, 8, 8, 1, 64, 32, [700, 31], None, True),
    (4, 8, 2, 3, 128, 16, [3, 16, 17, 130], None, True),  # 12 query rows a head
    (4, 8, 2, 4, 64, 128, [4, 200, 129, 255], [4, 0, 1, 3], True),
    (2, 8, 1, 5, 128, 32, [100, 37], [5, 2], True),      # 40 query rows a head
    (2, 6, 2, 2, 64, 64, [65, 64], None, False),
    (1, 16, 1, 1, 128, 128, [513], None, False),
    (1, 3, 1, 7, 64, 16, [7], None, True),               # every row sees a different prefix
])
def test_decode_matches_fp64(dtype, B, Hq, Hkv, T, d, page, lens, q_lens, causal):
    if lens[0] == 0 and q_lens is None:
        q_lens = [0] + [T] * (B - 1)
    c = ref.Cache(dtype, B, Hkv, d, page, -(-max(lens) // page) + 1, lens, seed=50 + d + page)
    check_decode(c, c.cuda(), randn(B, Hq, T, d, seed=51), q_lens, causal)


@pytest.mark.parametrize("dtype", [E4M3, BF16])
def test_decode_empty_sequence_with_queries_is_refused_on_the_device(dtype):
    """More query tokens than rows: reported, the outputs of others are right."""
    c = ref.Cache(dtype, 2, 1, 64, 16, 4, [0, 50], seed=52)
    dev, q = c.cuda(), randn(2, 2, 1, 64, seed=53)
    ws = dfa.paged_workspace(dev, 2, 1)
    o, lse = dfa.decode_paged(dev, q.cuda(), ws=ws)
    with pytest.raises(dfa.DfaError) as e:
        dfa.stream_status(ws)
    assert e.value.code == 6
    O, LSE, tO, tL = ref.attention(c, q, [0, 1])
    ref.check(o[1], O[1], tO[1], BF16)
    ref.check(lse[1], LSE[1], tL[1], torch.float32)


@pytest.mark.parametrize("dtype", [E4M3, BF16])
def test_decode_strided_queries_and_scale(dtype):
    c = ref.Cache(dtype, 2, 2, 128, 16, 8, [100, 128], seed=54)
    qkv = randn(2, 3, 10, 128, seed=55)
    q = qkv.transpose(1, 2)[:, 2:8]
    dev = c.cuda()
    O, LSE, tO, tL = ref.attention(c, q, scale=0.3)
    o, lse = dfa.decode_paged(dev, qkv.cuda().transpose(1, 2)[:, 2:8], scale=0.3)
    ref.check(o, O, tO, BF16)
    ref.check(lse, LSE, tL, torch.float32)


@pytest.mark.parametrize("dtype", [E4M3, BF16])
def test_decode_large_and_small_magnitudes(dtype):
    """Queries and cells far from one; scores that reach tens of thousands, so
    that one key takes all the weight."""
    for i, gain in enumerate((1e-3, 40.0, 2e3)):
        c = ref.Cache(dtype, 1, 2, 128, 32, 8, [250], seed=56 + i, loud=gain)
        q = (randn(1, 4, 1, 128, seed=57).float() * 16).to(BF16)
        check_decode(c, c.cuda(), q)


def test_decode_value_scales_far_apart():
    """Pages whose value scales differ by 2^60 either way: the weights are held
    relative to the largest contribution."""
    c = ref.Cache(E4M3, 1, 1, 64, 16, 16, [256], seed=58)
    order = c.table[0].long()
    c.scales["v"][order, 0] = torch.exp2(torch.tensor([0., 60, -60, 3, -3, 30, -30, 59] * 2))
    check_decode(c, c.cuda(), randn(1, 2, 1, 64, seed=59))


@pytest.mark.parametrize("T", [1, 9])
@pytest.mark.parametrize("exps", [[115], [-100], [0, 115], [115, 0], [-100, 115], [115, -100, 0],
                                  [-100, 0], [0, -100], [41, 39, -41], [-126, 3]])
def test_decode_value_scales_at_the_ends_of_their_range(exps, T):
    """Pages of zeros (the smallest scale) and of values near the type's largest,
    alone and together: neither the weights nor the sum of probabilities leave
    fp32's range."""
    for split in (16, 40):
        c = ref.Cache(E4M3, 1, 1, 128, 16, split, [16 * split - 3], seed=158)
        order = c.table[0].long()
        e = torch.tensor([float(exps[i % len(exps)]) for i in range(split)])
        c.scales["v"][order, 0] = torch.exp2(e)
        check_decode(c, c.cuda(), randn(1, 2, T, 128, seed=159))


@pytest.mark.parametrize("d", [64, 128])
def test_decode_results_at_the_end_of_fp32(d):
    """Outputs next to fp32's smallest normal numbers: the quietest page has the
    loudest scores, by a little more than 2^8, so that what the weighted sum is
    relative to lies more than 2^126 below what the sum of probabilities is."""
    c = ref.Cache(E4M3, 1, 1, d, 16, 8, [128], seed=185)
    order = c.table[0].long()
    k = torch.zeros(c.npages, 1, 16, d)
    k[..., 0] = -96.0
    k[order[0], ..., 0], k[order[4], ..., 0] = 0.0, 7.0
    c.cells["k"] = k.to(E4M3)
    c.scales["k"][:] = 1.0
    c.scales["v"][:] = 2.0 ** -118
    c.scales["v"][order[4]] = 2.0 ** -126
    q = torch.zeros(1, 2, 1, d, dtype=BF16)
    q[..., 0] = 1.0
    check_decode(c, c.cuda(), q, scale=1.0)


def test_decode_of_appended_values_near_the_largest():
    dev, q = None, randn(1, 2, 1, 64, seed=160)
    x = torch.randn(1, 1, 40, 64, generator=torch.Generator().manual_seed(161))
    for gain in (1e38, 1e-38):
        k, v = randn(1, 1, 40, 64, seed=162), (x * gain / 4.2).to(BF16)
        c = ref.Cache(E4M3, 1, 1, 64, 16, 3, [40], seed=163)
        dev = c.cuda()
        dfa.cache_append(dev, k.cuda(), v.cuda())
        for name, got in (("k", dev.k), ("v", dev.v)):
            c.cells[name] = got.cpu()
        c.scales = {"k": dev.k_scale.cpu(), "v": dev.v_scale.cpu()}
        check_decode(c, dev, q)


@pytest.mark.parametrize("d,Hq", [(64, 1), (128, 12)])
def test_decode_extreme_scales_joined_from_many_blocks(d, Hq):
    """A long sequence cut into more partial results than one warp joins; whole
    stretches of it quiet, loud or in between."""
    n = 700
    c = ref.Cache(E4M3, 1, 1, d, 16, n, [16 * n - 5], seed=164)
    e = torch.tensor([(-100.0, 0.0, 115.0, 60.0, -40.0)[i // 140] for i in range(n)])
    c.scales["v"][c.table[0].long(), 0] = torch.exp2(e)
    check_decode(c, c.cuda(), randn(1, Hq, 1, d, seed=165))


@pytest.mark.parametrize("dtype", [E4M3, BF16])
@pytest.mark.parametrize("Hq,T,q_lens,causal", [(32, 32, None, True), (2, 512, [300, 512], True),
                                                (4, 3, [0, 2], False), (17, 1, None, False)])
def test_decode_most_rows_and_unmasked_ragged(dtype, Hq, T, q_lens, causal):
    """1024 query rows of a head, more tokens than a page; and ragged queries that
    see every key."""
    c = ref.Cache(dtype, 2, 1, 64, 16, 40, [300, 530], seed=166)
    check_decode(c, c.cuda(), randn(2, Hq, T, 64, seed=167), q_lens, causal)


@pytest.mark.parametrize("dtype", [E4M3, BF16])
def test_decode_nan_where_a_row_does_not_look(dtype):
    """Drafted tokens: the last token's K and V are NaN, which only that token
    sees; and NaN in a visible key makes a row NaN."""
    c = ref.Cache(dtype, 1, 1, 64, 16, 3, [37], seed=60)
    for name in "kv":
        x = c.cells[name].float()
        x[int(c.table[0, 36 // 16]), :, 36 % 16] = float("nan")
        c.cells[name] = x.to(c.dtype)
    q = randn(1, 2, 3, 64, seed=61)
    o, lse = dfa.decode_paged(c.cuda(), q.cuda())
    assert o[:, :, 2].isnan().all() and lse[:, :, 2].isnan().all()
    O, LSE, tO, tL = ref.attention(c, q)
    ref.check(o[:, :, :2], O[:, :, :2], tO[:, :, :2], BF16)
    ref.check(lse[:, :, :2], LSE[:, :, :2], tL[:, :, :2], torch.float32)


@pytest.mark.parametrize("dtype", [E4M3, BF16])
def test_decode_infinite_value_of_a_drafted_token(dtype):
    """An infinite value (NaN in 8 bits) that some rows see and others do not."""
    c = ref.Cache(dtype, 1, 2, 128, 16, 3, [40], seed=62)
    x = c.cells["v"].float()
    x[int(c.table[0, 38 // 16]), 0, 38 % 16, 5] = float("nan" if dtype is E4M3 else "inf")
    c.cells["v"] = x.to(c.dtype)
    q = randn(1, 8, 4, 128, seed=63)
    o, lse = dfa.decode_paged(c.cuda(), q.cuda())
    O, LSE, tO, tL = ref.attention(c, q)
    hit = torch.zeros(O.shape, dtype=torch.bool)
    hit[0, :4, 2:, 5] = True
    assert not o.cpu()[hit].isfinite().any()
    got = o.cpu().double()
    ref.check(torch.where(hit, 0.0, got), torch.where(hit, 0.0, O), torch.where(hit, 0.0, tO), BF16)
    ref.check(lse, LSE, tL, torch.float32)


def test_decode_ragged_batch_of_many():
    """More sequences than blocks, most of them short."""
    g = torch.Generator().manual_seed(64)
    lens = torch.randint(1, 70, (300,), generator=g).tolist()
    lens[7] = 900
    c = ref.Cache(E4M3, 300, 1, 64, 16, 57, lens, seed=65)
    check_decode(c, c.cuda(), randn(300, 2, 1, 64, seed=66))


@pytest.mark.parametrize("dtype", [E4M3, BF16])
@pytest.mark.parametrize("T", [1, 3])
def test_decode_ragged_batch_of_short_sequences(dtype, T):
    """Tables of a few tiles, whose segments are not cut: many more of them than
    blocks, idle sequences between, at the end and at the beginning."""
    g = torch.Generator().manual_seed(168)
    lens = torch.randint(T, 140, (400,), generator=g).tolist()
    q_lens = torch.randint(0, T + 1, (400,), generator=g).tolist()
    for b in (0, 1, 50, 51, 52, 399):
        lens[b] = q_lens[b] = 0
    c = ref.Cache(dtype, 400, 2, 64, 16, 9, lens, seed=169)
    check_decode(c, c.cuda(), randn(400, 8, T, 64, seed=170), q_lens)


def test_decode_many_query_heads_of_one_cache_head():
    c = ref.Cache(E4M3, 2, 1, 64, 32, 4, [100, 128], seed=67)
    check_decode(c, c.cuda(), randn(2, 48, 2, 64, seed=68))


@pytest.mark.parametrize("dtype", [E4M3, BF16])
@pytest.mark.parametrize("B,lens", [(1, [20000]), (32, [9 + i for i in range(31)] + [20000])])
def test_decode_one_long_sequence(dtype, B, lens):
    """One sequence cut over most of the grid: hundreds of partial results a row."""
    c = ref.Cache(dtype, B, 2, 64, 128, 157, lens, seed=86, extra=0)
    check_decode(c, c.cuda(), randn(B, 6, 1, 64, seed=87))


@pytest.mark.parametrize("dtype", [E4M3, BF16])
def test_decode_long_sequences_of_several_row_groups(dtype):
    """40 query rows of a head: three groups, each cut over its own blocks."""
    c = ref.Cache(dtype, 2, 1, 64, 32, 330, [9000, 10500], seed=183)
    check_decode(c, c.cuda(), randn(2, 10, 4, 64, seed=184), [4, 3])


def test_decode_mostly_idle_batch():
    """A padded batch: slots without queries, some of them without rows, between the
    others and at both ends; their outputs are left as they were."""
    g = torch.Generator().manual_seed(88)
    lens = torch.randint(0, 200, (400,), generator=g).tolist()
    q_lens = [min(2, n) if i % 7 == 3 else 0 for i, n in enumerate(lens)]
    c = ref.Cache(E4M3, 400, 1, 64, 16, 13, lens, seed=89)
    check_decode(c, c.cuda(), randn(400, 2, 2, 64, seed=90), q_lens)
    check_decode(c, c.cuda(), randn(400, 2, 2, 64, seed=90), [0] * 400)


def test_workspace_of_other_shapes_and_captured_without_one():
    """One workspace, sized for the largest call, serves calls of every shape in
    turn; and a call without one can be captured."""
    c = ref.Cache(E4M3, 2, 2, 128, 32, 8, [200, 131], seed=91)
    dev = c.cuda()
    ws = dfa.paged_workspace(dev, 8, 4)
    for T in (4, 1, 3, 1):
        q = randn(2, 8, T, 128, seed=92 + T)
        o, lse = dfa.decode_paged(dev, q.cuda(), ws=ws)
        dfa.cache_gather(dev, 7, ws=ws)
        dfa.stream_status(ws)
        O, LSE, tO, tL = ref.attention(c, q)
        ref.check(o, O, tO, BF16)
        ref.check(lse, LSE, tL, torch.float32)
    g, qg = torch.cuda.CUDAGraph(), q.cuda()
    with torch.cuda.graph(g):
        o, lse = dfa.decode_paged(dev, qg)
        r = dfa.rope(qg, dfa.rope_spec(128, layout="half"))
        k, v = dfa.cache_gather(dev, 200)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    ref.check(o, O, tO, BF16)
    check_rope(r, q, torch.arange(1), "half", 128, False, {})
    assert torch.equal(k[0].cpu().double(), c.rows("k", 0, 200))


def test_binding_refuses_on_the_gpu():
    """What only tensors on the device can show."""
    c = ref.Cache(E4M3, 2, 2, 64, 16, 2, [5, 17], seed=93)
    dev = c.cuda()
    x = randn(2, 2, 3, 64, seed=94).cuda()
    spec = dfa.rope_spec(64)
    pos = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    bad = [
        lambda: dfa.rope(x.half(), spec), lambda: dfa.rope(x[0], spec),
        lambda: dfa.rope(x, spec, positions=pos.long()),
        lambda: dfa.rope(x, spec, positions=pos[:, :2]),
        lambda: dfa.rope(x, spec, positions=pos, pos_map=dfa.pos_map(1, (3, 0))),
        lambda: dfa.rope(x.transpose(2, 3), spec), lambda: dfa.rope(x, spec, out=x[:1]),
        lambda: dfa.rope(x, spec, out=x.float()),
        lambda: dfa.cache_append(dev, x.float(), x), lambda: dfa.cache_append(dev, x, x[:1]),
        lambda: dfa.cache_append(dev, x, x, q_out=x),
        lambda: dfa.cache_append(dev, x, x, new_lens=torch.ones(2, device="cuda")),
        lambda: dfa.cache_append(dev, x, x, ws=torch.zeros(256, device="cuda")),
        lambda: dfa.cache_gather(dev, 4, k_out=x), lambda: dfa.decode_paged(dev, x[0]),
        lambda: dfa.decode_paged(dev, x[:1]), lambda: dfa.decode_paged(dev, x.float()),
        lambda: dfa.decode_paged(dev, x, out=x.float()),
        lambda: dfa.decode_paged(dev, x, lse=torch.zeros(2, 2, 2, device="cuda")),
        lambda: dfa.decode_paged(dev, x, q_lens=torch.ones(3, dtype=torch.int32, device="cuda")),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    for f in (lambda: dfa.rope(x, spec, out=x.as_strided((2, 2, 3, 64), (384, 0, 64, 1))),
              lambda: dfa.decode_paged(dev, x[:, :1]),                # 1 head over 2
              lambda: dfa.decode_paged(dev, x, ws=torch.zeros(256, dtype=torch.uint8,
                                                              device="cuda")),
              lambda: dfa.cache_append(dev, x, x, q=x, q_out=torch.empty_like(x))):
        with pytest.raises(dfa.DfaError):
            f()


def test_shared_pages_are_read_by_both():
    """Two sequences with a common prefix in the same pages."""
    c = ref.Cache(E4M3, 2, 1, 64, 16, 4, [50, 50], seed=69)
    c.table[1, :2] = c.table[0, :2]
    check_decode(c, c.cuda(), randn(2, 2, 1, 64, seed=70))


def test_long_cache_offsets_past_32_bits():
    """Pages whose first element lies beyond 2^32 elements."""
    page, H, d = 128, 8, 128
    npages = 2 ** 32 // (page * H * d) + 40
    k = torch.zeros(npages, H, page, d, dtype=E4M3, device="cuda")
    v = torch.zeros(npages, H, page, d, dtype=E4M3, device="cuda")
    ks, vs = (torch.ones(npages, H, device="cuda") for _ in range(2))
    table = torch.tensor([[npages - 1, npages - 30]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([200], dtype=torch.int32, device="cuda")
    dev = dfa.PagedCache(k, v, table, lens, k_scale=ks, v_scale=vs)
    kn, vn = (randn(1, H, 200, d, seed=s) for s in (71, 72))
    dfa.cache_append(dev, kn.cuda(), vn.cuda())
    gk, gv = dfa.cache_gather(dev, 200)
    c = ref.Cache(E4M3, 1, H, d, page, 2, [200], seed=73, extra=0)
    at = table[0].long()
    c.table = torch.tensor([[0, 1]], dtype=torch.int32)
    c.cells = {"k": k[at].cpu(), "v": v[at].cpu()}
    c.scales = {"k": ks[at].cpu(), "v": vs[at].cpu()}
    assert torch.equal(gk.cpu().double()[0], c.rows("k", 0, 200))
    assert torch.equal(gv.cpu().double()[0], c.rows("v", 0, 200))
    q = randn(1, 8, 1, d, seed=74)
    O, LSE, tO, tL = ref.attention(c, q)
    o, lse = dfa.decode_paged(dev, q.cuda())
    ref.check(o, O, tO, BF16)
    ref.check(lse, LSE, tL, torch.float32)


def test_bad_pages_and_lengths_are_reported_and_skipped():
    """The device checks every length and page: nothing is read or written
    through a bad one, the status word says so, other sequences are right."""
    c = ref.Cache(E4M3, 4, 2, 64, 16, 3, [40, 40, 40, 40], seed=75)
    dev = c.cuda()
    before = {n: getattr(dev, n).clone() for n in ("k", "v", "k_scale", "v_scale")}
    dev.block_table[1, 2] = c.npages          # the page that new rows go to
    dev.block_table[2, 0] = -7                # a page that is only read
    dev.seq_lens[3] = 49                      # longer than the table
    k, v, q = (randn(4, h, 2, 64, seed=76 + h) for h in (2, 2, 4))
    ws = dfa.paged_workspace(dev, 4, 2)

    def reported():
        with pytest.raises(dfa.DfaError) as e:
            dfa.stream_status(ws)
        assert e.value.code == 6
        dfa.stream_status(ws)  # read and cleared

    dfa.cache_append(dev, k.cuda(), v.cuda(), ws=ws)
    reported()
    touched = {int(c.table[b, 2]) for b in (0, 2)}
    same = [i for i in range(c.npages) if i not in touched]
    for n, t in before.items():
        assert torch.equal(getattr(dev, n)[same].view(torch.uint8), t[same].view(torch.uint8))
    o, lse = dfa.decode_paged(dev, q.cuda(), ws=ws)
    reported()
    dfa.cache_gather(dev, 48, ws=ws)
    reported()
    c.cells = {"k": dev.k.cpu(), "v": dev.v.cpu()}
    c.scales = {"k": dev.k_scale.cpu(), "v": dev.v_scale.cpu()}
    one = ref.Cache(E4M3, 1, 2, 64, 16, 3, [40], seed=75)
    one.table, one.cells, one.scales = c.table[:1], c.cells, c.scales
    O, LSE, tO, tL = ref.attention(one, q[:1])
    ref.check(o[:1], O, tO, BF16)
    new = torch.tensor([3, -1, 2, 2], dtype=torch.int32, device="cuda")  # above T, negative
    dfa.decode_paged(dev, q.cuda(), q_lens=new, ws=ws)
    reported()


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
def test_streams_and_workspaces_of_two_calls_at_once():
    """Two calls on two streams, each with its own workspace; and a call whose
    outputs the binding allocates for the given stream."""
    c1 = ref.Cache(E4M3, 2, 2, 128, 16, 40, [600, 77], seed=80)
    c2 = ref.Cache(BF16, 3, 1, 64, 64, 5, [300, 1, 64], seed=81)
    q1, q2 = randn(2, 8, 1, 128, seed=82), randn(3, 4, 2, 64, seed=83)
    d1, d2, g1, g2 = c1.cuda(), c2.cuda(), q1.cuda(), q2.cuda()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    n = torch.tensor([2, 1, 2], dtype=torch.int32, device="cuda")
    s2.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        o1, l1 = dfa.decode_paged(d1, g1, stream=s1)
        o2, l2 = dfa.decode_paged(d2, g2, q_lens=n, stream=s2)
    torch.cuda.synchronize()
    for c, q, o, lse, ql in ((c1, q1, o1, l1, [1, 1]), (c2, q2, o2, l2, [2, 1, 2])):
        O, LSE, tO, tL = ref.attention(c, q, ql)
        for b, n in enumerate(ql):
            ref.check(o[b, :, :n], O[b, :, :n], tO[b, :, :n], BF16)
            ref.check(lse[b, :, :n], LSE[b, :, :n], tL[b, :, :n], torch.float32)


@pytest.mark.parametrize("before", ["nothing", "copy", "memset", "join", "decode", "copies"])
def test_captured_behind(before):
    """A decode of few blocks captured as the first node of a graph, behind copies,
    behind a join of two streams, and behind another decode on one workspace; what
    came before it is seen."""
    c = ref.Cache(E4M3, 1, 2, 128, 16, 40, [600], seed=180)
    q, q0 = randn(1, 8, 1, 128, seed=181), randn(1, 8, 1, 128, seed=182)
    dev, src = c.cuda(), q.cuda()
    q_dev = q0.cuda()
    staging = torch.empty_like(q_dev)
    scratch = torch.ones(1 << 20, dtype=torch.uint8, device="cuda")
    ws = dfa.paged_workspace(dev, 8)
    out, lse = torch.empty_like(q_dev), torch.empty(1, 8, 1, device="cuda")
    o2, l2 = torch.empty_like(q_dev), torch.empty(1, 8, 1, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()

    def step():
        main = torch.cuda.current_stream()
        if before == "copy":
            q_dev.copy_(src)
        elif before == "copies":
            staging.copy_(src)
            q_dev.copy_(staging)
        elif before == "memset":
            q_dev.copy_(src)
            scratch.zero_()
        elif before == "join":
            side.wait_stream(main)
            with torch.cuda.stream(side):
                q_dev.copy_(src)
                q_dev.mul_(1)
            scratch.add_(1)
            main.wait_stream(side)
        elif before == "decode":
            dfa.decode_paged(dev, q_dev, out=o2, lse=l2, ws=ws)
            q_dev.copy_(src)
        dfa.decode_paged(dev, q_dev, out=out, lse=lse, ws=ws)

    if before == "nothing":
        q_dev.copy_(src)
    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    O, LSE, tO, tL = ref.attention(c, q)
    for _ in range(50):
        if before != "nothing":
            q_dev.copy_(q0)
        out.fill_(7.0)
        g.replay()
        ref.check(out, O, tO, BF16)
        ref.check(lse, LSE, tL, torch.float32)
    dfa.stream_status(ws)


def test_same_call_twice_gives_the_same_bits():
    c = ref.Cache(E4M3, 3, 2, 128, 16, 64, [1000, 3, 500], seed=84)
    dev, q = c.cuda(), randn(3, 8, 2, 128, seed=85).cuda()
    a = dfa.decode_paged(dev, q, out_fp32=True)
    for _ in range(5):
        b = dfa.decode_paged(dev, q, out_fp32=True)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype", [E4M3, BF16])
def test_serving_loop(dtype):
    """A prompt appended in two chunks (the second attends to the first through
    the gather and a chunk pair), then decoding steps replayed as one captured
    graph whose lengths advance on the device; every result against attention
    over the cached rows."""
    B, Hq, Hkv, d, page, width = 2, 8, 2, 128, 16, 20
    spec = dfa.rope_spec(d, layout="half", rot_dim=64)
    c = ref.Cache(dtype, B, Hkv, d, page, width, [0, 0], seed=90)
    dev = c.cuda()
    ws = dfa.paged_workspace(dev, Hq, 1)

    def refresh():
        c.lens = dev.seq_lens.cpu()
        c.cells = {"k": dev.k.cpu(), "v": dev.v.cpu()}
        if dtype is E4M3:
            c.scales = {"k": dev.k_scale.cpu(), "v": dev.v_scale.cpu()}

    at = 0
    for i, T in enumerate((150, 45)):
        q, k, v = (randn(B, h, T, d, seed=91 + 3 * i + j).cuda()
                   for j, h in enumerate((Hq, Hkv, Hkv)))
        dev.seq_lens += T
        q = dfa.cache_append(dev, k, v, rope=spec, q=q, ws=ws)
        L = at + T
        K, V = dfa.cache_gather(dev, L, ws=ws)
        o, lse = dfa.chunk_fwd(q, K, V, dfa.pos_map(1, (T, 0), (at, 0)),
                               dfa.pos_map(1, (L, 0), (0, 0)))
        dfa.stream_status(ws)
        refresh()
        rows = [0, T // 2, T - 1]
        for b in range(B):
            for t in rows:
                n = at + t + 1
                for h in (0, Hq - 1):
                    kk, vv = c.rows("k", b, n)[h // 4], c.rows("v", b, n)[h // 4]
                    s = (kk @ q[b, h, t].cpu().double()) / math.sqrt(d)
                    assert abs(float(lse[b, h, t]) - float(torch.logsumexp(s, 0))) <= 2e-3
                    assert (o[b, h, t].cpu().double() - torch.softmax(s, 0) @ vv).abs().max() <= 1e-2
        at = L
    # decoding: inputs are copied into place, one graph does a step
    q, k, v = (torch.zeros(B, h, 1, d, dtype=BF16, device="cuda") for h in (Hq, Hkv, Hkv))
    one = torch.ones(B, dtype=torch.int32, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(B, Hq, 1, device="cuda")
    qr = torch.empty_like(q)

    def step():
        dev.seq_lens.add_(one)
        dfa.cache_append(dev, k, v, rope=spec, q=q, q_out=qr, ws=ws)
        dfa.decode_paged(dev, qr, out=out, lse=lse, ws=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    lens = dev.seq_lens.clone()
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    dev.seq_lens.copy_(lens)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    dev.seq_lens.copy_(lens)
    for i in range(20):
        for j, t in enumerate((q, k, v)):
            t.copy_(randn(*t.shape, seed=200 + 3 * i + j))
        g.replay()
        if i in (0, 12, 19):
            dfa.stream_status(ws)
            refresh()
            assert c.lens.tolist() == [at + i + 1] * B
            O, LSE, tO, tL = ref.attention(c, qr.cpu())
            ref.check(out, O, tO, BF16)
            ref.check(lse, LSE, tL, torch.float32)
            check_rope(qr.cpu(), q.cpu(), torch.tensor([at + i]), "half", 64, False, {})
