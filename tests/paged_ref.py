"""Plain fp64 forms of the rotary positions and of the paged cache, on the CPU,
and the caches and tolerances that their tests share.  They share no code with
the kernels."""
import math

import torch

E4M3 = torch.float8_e4m3fn
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24, E4M3: 2.0 ** -4}


def frequencies(rot, base=10000.0, scaling="none", factor=1.0, orig_len=0.0, low=0.0, high=0.0,
                **_):
    f = []
    for t in range(rot // 2):
        x = base ** (-2.0 * t / rot)
        if scaling == "linear":
            x /= factor
        elif scaling == "bands":
            r = orig_len * x / (2 * math.pi)
            u = min(1.0, max(0.0, (r - low) / (high - low)))
            x = (1 - u) * x / factor + u * x
        f.append(x)
    return torch.tensor(f, dtype=torch.float64)


def rope(x, pos, layout, rot, inverse=False, gain=1.0, **kw):
    """x [..., n, d] (any dtype), pos [..., n] broadcasting; fp64."""
    x = x.double()
    a = pos.double()[..., None] * frequencies(rot, **kw)
    a = -a if inverse else a
    c, s = gain * torch.cos(a), gain * torch.sin(a)
    out = x.clone()
    lo = slice(0, rot // 2) if layout == "half" else slice(0, rot, 2)
    hi = slice(rot // 2, rot) if layout == "half" else slice(1, rot, 2)
    out[..., lo] = x[..., lo] * c - x[..., hi] * s
    out[..., hi] = x[..., lo] * s + x[..., hi] * c
    return out


def rope_tol(x, rot, dtype, layout, gain=1.0):
    """Half a step of the output's type (applied to |ref| by the caller), and the
    fp32 arithmetic: the angle's cos and sin are off by at most 2.5e-7 (the 32-bit
    phase as fp32, half a step of half a turn = pi 2^-25, and sincospif's 2
    steps of 2^-24), and three fp32 operations add 3 * 2^-24, all times the
    pair's |x| + |y|."""
    a = x.double().abs()
    pair = torch.zeros_like(a)
    lo = slice(0, rot // 2) if layout == "half" else slice(0, rot, 2)
    hi = slice(rot // 2, rot) if layout == "half" else slice(1, rot, 2)
    pair[..., lo] = pair[..., hi] = a[..., lo] + a[..., hi]
    return gain * pair * (2.5e-7 + 3 * 2.0 ** -24)


def pow2_scale(amax):
    """Smallest power of two s >= 2^-100 with amax <= 448 s."""
    s = 2.0 ** -100
    while amax > 448 * s:
        s *= 2
    return s


class Cache:
    """A cache on the CPU: pages in random order; cells of pages and rows that no
    sequence owns hold NaN."""

    def __init__(self, dtype, B, Hkv, d, page, max_pages, lens, seed=0, loud=None, extra=2):
        g = torch.Generator().manual_seed(seed)
        self.dtype, self.page, self.Hkv, self.d, self.B = dtype, page, Hkv, d, B
        self.npages = B * max_pages + extra
        self.table = torch.randperm(self.npages, generator=g)[:B * max_pages].to(
            torch.int32).view(B, max_pages)
        self.lens = torch.tensor(lens, dtype=torch.int32)
        shape = (self.npages, Hkv, page, d)
        self.cells, self.scales = {}, {}
        for name in "kv":
            x = torch.randn(shape, generator=g)
            if loud is not None:
                x = x * loud
            if dtype is E4M3:
                amax = x.abs().amax((2, 3))
                s = torch.tensor([[pow2_scale(float(a)) for a in r] for r in amax])
                # scales of different pages far apart, as a loud token makes them
                s = s * torch.exp2(torch.randint(0, 4, s.shape, generator=g).float())
                self.scales[name] = s.float()
                x = x / self.scales[name][..., None, None]
            x = x.to(dtype)
            owned = torch.zeros(self.npages, page, dtype=torch.bool)
            for b in range(B):
                for j in range(int(self.lens[b])):
                    owned[self.table[b, j // page], j % page] = True
            x = torch.where(owned[:, None, :, None], x.float(), torch.tensor(float("nan")))
            self.cells[name] = x.to(dtype)

    def scale(self, name, pg, h):
        return float(self.scales[name][pg, h]) if self.scales else 1.0

    def rows(self, name, b, n):
        """Rows [0, n) of sequence b, [Hkv, n, d] fp64."""
        out = torch.zeros(self.Hkv, n, self.d, dtype=torch.float64)
        for j in range(n):
            pg = int(self.table[b, j // self.page])
            x = self.cells[name][pg, :, j % self.page].double()
            for h in range(self.Hkv):
                out[h, j] = x[h] * self.scale(name, pg, h)
        return out

    def cuda(self):
        from long_context_flashattention_gb300 import dfa
        t = [self.cells["k"].cuda(), self.cells["v"].cuda(), self.table.cuda(), self.lens.cuda()]
        kw = {n + "_scale": s.cuda() for n, s in self.scales.items()}
        return dfa.PagedCache(*t, **kw)


def attention(cache, q, q_lens=None, causal=True, scale=None):
    """O, LSE (fp64) of q [B,Hq,T,d] and per element the bounds on the kernel's
    deviation; rows from q_lens on are NaN."""
    B, Hq, T, d = q.shape
    scale = 1 / math.sqrt(d) if scale is None else scale
    O = torch.full((B, Hq, T, d), float("nan"), dtype=torch.float64)
    LSE = torch.full((B, Hq, T), float("nan"), dtype=torch.float64)
    tO, tL = torch.zeros_like(O), torch.zeros_like(LSE)
    G = Hq // cache.Hkv
    for b in range(B):
        n = T if q_lens is None else int(q_lens[b])
        L = int(cache.lens[b])
        K, V = cache.rows("k", b, L), cache.rows("v", b, L)
        for t in range(n):
            seen = max(0, min(L, L - n + t + 1)) if causal else L
            for h in range(Hq):
                if seen == 0:
                    O[b, h, t], LSE[b, h, t] = 0.0, -math.inf
                    continue
                k, v = K[h // G, :seen], V[h // G, :seen]
                x = q[b, h, t].double()
                s = scale * (k @ x)
                LSE[b, h, t] = torch.logsumexp(s, 0)
                p = torch.softmax(s, 0)
                O[b, h, t] = p @ v
                # a score: d products summed in fp32, then scaled
                ds = (d + 4) * 2.0 ** -24 * scale * float((k.abs() @ x.abs()).max())
                # the sum of exponentials (2^-22 each) in fp32
                dl = ds + (seen + 16) * 2.0 ** -24 + 2.0 ** -21
                tL[b, h, t] = dl + 2.0 ** -23 * abs(float(LSE[b, h, t]))
                # probabilities in fp16 (half a step 2^-11, subnormals 2^-25 of the
                # largest weight) or as two bf16 terms (2^-16)
                w = p @ v.abs()
                tO[b, h, t] = w * (2.0 ** -11 + 2 * dl + (seen + 16) * 2.0 ** -24) + (
                    2.0 ** -24 * float(p.max()) * v.abs().sum(0))
    return O, LSE, tO, tL


def check(got, ref, tol, dtype, what=""):
    """|got - ref| <= tol + half a step of the output's type, element by element."""
    got = got.double().cpu()
    bad = ~((got - ref).abs() <= tol + HALF_STEP[dtype] * (ref.abs() + tol))
    same = (got == ref) | (got.isnan() & ref.isnan())
    bad &= ~same
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:4].tolist(),
                           got[bad][:4].tolist(), ref[bad][:4].tolist())
