"""Trees over a paged cache to the accuracy that the header gives each path: weights to 2^-25
(bf16 cells with an fp32 output, up to 64 rows a head), 2^-17 and 2^-22 (8 bits; 2^-11 with a
bf16 output), and sums of many tiles."""
import math

import pytest
import torch

from long_context_flashattention_gb300 import dfa

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


def queries(rows):
    """Scores of the second key, all different: bf16 values in (1/8, 2]."""
    return torch.linspace(0.13, 2.0, rows).to(BF16)


def weight_error(cells, rows):
    if cells is E4M3:
        return 2.0 ** -22
    return 2.0 ** -25 if rows <= 64 else 2.0 ** -17


def two_keys_bound(cells, rows):
    """Of O = w / (1 + w), w = e^-q, beside the weights' own rounding, relative, in 2^-24: the
    score 4 (log2 e and one operation rounded, an exponent below 2.9); 2^x 4; its sum 1; products
    cut off, 2 each for three terms; the joins of rows and groups 2, the division 1 and its
    product 1; for 8 bits two powers of two more, 4 each, and a product."""
    return (4 + 4 + 1 + 6 + 4 + (9 if cells is E4M3 else 0)) * 2.0 ** -24 + weight_error(
        cells, rows)


def test_the_bound_tells_terms_apart():
    """With a term less the weights alone are off by more than the bound (without a GPU)."""
    def left(w, dtype, terms):
        rest = w.clone()
        for _ in range(terms):
            rest = rest - rest.to(dtype).double()
        return (rest / w).abs().max()
    for rows in (17, 60, 64):
        w = torch.exp(-queries(rows).double())
        assert left(w, BF16, 3) <= weight_error(BF16, rows)
        # (w / (1 + w) has 1 / (1 + w) of the weight's error, at least half)
        assert left(w, BF16, 2) / (1 + w.max()) > two_keys_bound(BF16, rows)
        assert left(w * 256, torch.float16, 2) <= weight_error(E4M3, rows)
        assert left(w * 256, torch.float16, 1) / (1 + w.max()) > two_keys_bound(E4M3, rows)
    w = torch.exp(-queries(128).double())
    assert left(w, BF16, 2) <= weight_error(BF16, 128)
    assert left(w, BF16, 1) / 2 > two_keys_bound(BF16, 128)


def cache_of(cells, k0, v, Hkv, page, B=1):
    """Rows of which feature 0 of the key is k0 and all features of the value are v."""
    n = -(-k0.numel() // page)
    out = []
    for x, features in ((k0, 1), (v, 64)):
        t = torch.zeros(n * page, 64, device="cuda")
        t[:x.numel(), :features] = x[:, None]
        t = t.view(n, 1, page, 64).to(cells).expand(n, Hkv, page, 64)
        out.append(t.contiguous())
    kw = {}
    if cells is E4M3:
        kw = {s: torch.ones(n, Hkv, device="cuda") for s in ("k_scale", "v_scale")}
    table = torch.arange(n, device="cuda", dtype=torch.int32).repeat(B, 1)
    lens = torch.full((B,), k0.numel(), device="cuda", dtype=torch.int32)
    return dfa.PagedCache(*out, table, lens, **kw)


def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.gpu
@pytest.mark.parametrize("cells", [BF16, E4M3])
@pytest.mark.parametrize("T", [17, 60, 64, 128])
def test_weights_of_two_keys(cells, T):
    """A context of two keys, of scores 0 and -q and values 0 and 1; nodes that see nothing of
    their tree, whose keys would count a great deal."""
    need_gpu()
    q0 = queries(T)
    k0, v = torch.full((2 + T,), 8.0), torch.full((2 + T,), -100.0)
    k0[0], v[0], k0[1], v[1] = 0.0, 0.0, -1.0, 1.0
    c = cache_of(cells, k0.cuda(), v.cuda(), 2, 16)
    q = torch.zeros(1, 2, T, 64, dtype=BF16)
    q[0, :, :, 0] = q0
    mask = torch.zeros(1, T, -(-T // 32), dtype=torch.int32, device="cuda")
    o, lse = dfa.decode_tree(c, q.cuda(), mask, scale=1.0, out_fp32=True)
    dfa.stream_status(c.status)
    w = torch.exp(-q0.double())
    want = (w / (1 + w))[:, None]
    assert ((o[0].cpu().double() - want).abs() / want).max() <= two_keys_bound(cells, T)
    # (log2 to a step of it, at most 1, and the product)
    assert (lse[0].cpu().double() - torch.log1p(w)).abs().max() <= 2.0 ** -21


@pytest.mark.gpu
@pytest.mark.parametrize("cells", [BF16, E4M3])
@pytest.mark.parametrize("T", [16, 100])
def test_sums_of_thousands_of_tiles(cells, T):
    """4096 tiles to a block: the numerator (O times the sum that the LSE has) is off by what
    32 tiles' products cut off, 2^-23 each, and not by what all of them would."""
    need_gpu()
    L, B, Hkv = 1 << 19, 19, 8
    q0 = queries(T)
    k0, v = torch.full((L + T,), -1.0), torch.ones(L + T)
    k0[0], v[0] = 0.0, 0.0
    c = cache_of(cells, k0.cuda(), v.cuda(), Hkv, 128, B)
    q = torch.zeros(B, Hkv, T, 64, dtype=BF16)
    q[..., 0] = q0
    mask = torch.zeros(B, T, -(-T // 32), dtype=torch.int32, device="cuda")
    o, lse = dfa.decode_tree(c, q.cuda(), mask, scale=1.0, out_fp32=True)
    dfa.stream_status(c.status)
    want = (L - 1) * torch.exp(-q0.double())
    got = o.cpu().double() * torch.exp(lse.cpu().double())[..., None]
    # 8 products of 16 keys a tile, 128 sums set apart and added in fp32, the LSE to 2^-23 of
    # its 13, a few operations, and the weights
    bound = (32 * 8 * 2 + 128 + 2 * 13 + 40) * 2.0 ** -24 + weight_error(cells, T)
    err = (got - want[:, None]).abs() / want[:, None]
    assert err.max() <= bound, (float(err.max()), bound)
    assert math.isfinite(float(err.max()))


@pytest.mark.gpu
@pytest.mark.parametrize("cells", [BF16, E4M3])
@pytest.mark.parametrize("T", [16, 100])
def test_bf16_outputs_of_thousands_of_tiles(cells, T):
    """8192 tiles to a block of values 1 and 1.125, in such numbers that their mean lies above
    the border between two bf16 numbers by more than it may be off, for the products of 256
    tiles, but not by what all of them would cut off."""
    need_gpu()
    L, B, Hkv, page = 1 << 20, 19, 8, 128
    n = L // page
    # weights; 4 products of 16 keys a tile (8 with two terms); the sum's 8192 steps of 2^-24 at
    # worst; the shares of high values, rounded to a key
    off = (2.0 ** -11 if cells is E4M3 else 2.0 ** -17) + 256 * 8 * 2.0 ** -23 + (
        8192 * 2.0 ** -24) + 2.0 ** -16
    mean = (1 + 8.5 * 2.0 ** -7) * (1 + off)
    assert mean < 1 + 9 * 2.0 ** -7
    g = torch.Generator(device="cuda").manual_seed(1)

    def values(m):
        perm = torch.randperm(m, generator=g, device="cuda")
        return torch.where(perm < math.ceil((mean - 1) * 8 * m), 1.125, 1.0)
    # a page's first key has a larger weight than the others, which are then below 1, with
    # as many bits as their type has; high values are as many among those as among all
    k0 = torch.full((n, page), -1.0, device="cuda")
    v = values(L).view(n, page)
    k0[:, 0], v[:, 0] = 0.0, values(n)
    c = cache_of(cells, k0.flatten(), v.flatten(), Hkv, page, B)
    q = torch.zeros(B, Hkv, T, 64, dtype=BF16)
    q[..., 0] = queries(T)
    # (nodes that see one another, so that all rows count)
    mask = torch.full((B, T, -(-T // 32)), -1, dtype=torch.int32, device="cuda")
    o, _ = dfa.decode_tree(c, q.cuda(), mask, scale=1.0)
    dfa.stream_status(c.status)
    assert (o.float() == 1 + 9 * 2.0 ** -7).all(), float(o.float().min())
