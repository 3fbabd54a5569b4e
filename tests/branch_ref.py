"""Plain forms of trees of drafted tokens, kept rows and page pools, on the CPU, attention
in fp64.  They share no code with the kernels."""
import math

import torch

from paged_ref import E4M3


def random_parents(B, T, seed=0, roots=0.1):
    g = torch.Generator().manual_seed(seed)
    out = torch.empty(B, T, dtype=torch.int32)
    for b in range(B):
        for t in range(T):
            r = torch.rand(2, generator=g).tolist()
            out[b, t] = -1 if t == 0 or r[0] < roots else max(0, t - 1 - int(r[1] * 5))
    return out


def sees_of(parents):
    """[B, T, T] truth values: t sees u, its ancestor or itself."""
    B, T = parents.shape
    out = torch.zeros(B, T, T, dtype=torch.bool)
    for b in range(B):
        for t in range(T):
            p = int(parents[b, t])
            if p >= 0:
                out[b, t] = out[b, p]
            out[b, t, t] = True
    return out


def pack(sees):
    """Truth values [..., T] as int32 words."""
    T = sees.shape[-1]
    W = -(-T // 32)
    out = torch.zeros(*sees.shape[:-1], W, dtype=torch.int64)
    for u in range(T):
        out[..., u // 32] += sees[..., u].long() << (u % 32)
    return torch.where(out >= 2 ** 31, out - 2 ** 32, out).to(torch.int32)


def rows(cache, name, b, n):
    """Rows [0, n) of sequence b of a paged_ref.Cache, [Hkv, n, d] fp64."""
    j = torch.arange(n)
    pg = cache.table[b, j // cache.page].long()
    x = cache.cells[name].float()[pg, :, j % cache.page].double()     # [n, Hkv, d]
    if cache.scales:
        x = x * cache.scales[name][pg].double()[..., None]
    return x.transpose(0, 1)


def attention(cache, q, sees, q_lens=None, scale=None, weight=2.0 ** -11):
    """O, LSE (fp64) of q [B,Hq,T,d] under sees [B,T,T], and per element the bounds on the
    kernel's deviation (before the output's own rounding); rows from q_lens on are NaN.
      ds   a score: d products summed in fp32 by the matrix unit, which may cut off
           (2^-23 each) instead of rounding, and its scaling;
      dl   that, 2^x to two steps, and the sum of L terms in fp32;
      O    the weights' rounding (`weight` of each; half a step of fp16's subnormals is
           2^-25 where the largest weight is 2^11 or more, at least 2^-24 without that),
           twice dl (weights and sum), and the products' sum, cut off at 2^-23 per tile
           and term (4 for 128 keys) and 16 tiles for the joins."""
    B, Hq, T, d = q.shape
    scale = 1 / math.sqrt(d) if scale is None else scale
    O = torch.full((B, Hq, T, d), float("nan"), dtype=torch.float64)
    LSE = torch.full((B, Hq, T), float("nan"), dtype=torch.float64)
    tO, tL = torch.zeros_like(O), torch.zeros_like(LSE)
    G = Hq // cache.Hkv
    for b in range(B):
        n = T if q_lens is None else int(q_lens[b])
        L = int(cache.lens[b])
        if n == 0:
            continue
        K, V = rows(cache, "k", b, L), rows(cache, "v", b, L)
        seen = torch.ones(n, L, dtype=torch.bool)
        seen[:, L - n:] = sees[b, :n, :n]
        for h in range(cache.Hkv):
            x = q[b, h * G:(h + 1) * G, :n].double()                 # [G, n, d]
            # what nobody sees may hold anything
            for t in range(n):
                at = seen[t].nonzero()[:, 0]
                hs = slice(h * G, (h + 1) * G)
                if at.numel() == 0:
                    O[b, hs, t], LSE[b, hs, t] = 0.0, -math.inf
                    continue
                k, v = K[h, at], V[h, at]
                s = scale * (x[:, t] @ k.T)                          # [G, keys]
                lse = torch.logsumexp(s, -1)
                p = torch.softmax(s, -1)
                LSE[b, hs, t], O[b, hs, t] = lse, p @ v
                ds = (d + 4) * 2.0 ** -23 * scale * (x[:, t].abs() @ k.abs().T).amax(-1)
                dl = ds + (at.numel() + 16) * 2.0 ** -24 + 2.0 ** -21
                tL[b, hs, t] = dl + 2.0 ** -23 * lse.abs()
                acc = (4 * -(-L // 128) + 16) * 2.0 ** -23
                tO[b, hs, t] = (p @ v.abs()) * (weight + 2 * dl + acc)[:, None] + (
                    2.0 ** -24 * p.amax(-1)[:, None] * v.abs().sum(0))
    return O, LSE, tO, tL


def compact(cache, kept, kept_lens, q_lens):
    """cache_compact on a paged_ref.Cache, cells as codes in fp32: {name: (cells, scales)}."""
    page, out = cache.page, {}
    for name in "kv":
        cells = cache.cells[name].float().clone()
        scales = cache.scales[name].clone() if cache.scales else None
        for b in range(cache.B):
            first, a = int(cache.lens[b]) - int(q_lens[b]), int(kept_lens[b])
            src = [first + int(kept[b, i]) for i in range(a)]
            dst = [first + i for i in range(a)]
            place = lambda j: (int(cache.table[b, j // page]), j % page)  # noqa: E731
            was = [cells[place(j)[0], :, place(j)[1]].clone() for j in src]
            old = None if scales is None else [scales[place(j)[0]].clone() for j in src]
            begin = None if scales is None else scales.clone()
            for p in sorted({j // page for j in dst}):
                i = [i for i, j in enumerate(dst) if j // page == p]
                to, r0 = int(cache.table[b, p]), dst[i[0]] % page
                if scales is not None:
                    top = torch.stack([old[k] for k in i]).amax(0)
                    if r0 > 0:
                        top = torch.maximum(top, begin[to])
                        f = (begin[to] / top)[:, None, None]
                        # (cells of pages that nobody owns are NaN)
                        cells[to, :, :r0] = (cells[to, :, :r0] * f).to(E4M3).float()
                    scales[to] = top
                for k in i:
                    x = was[k]
                    if scales is not None:
                        x = (x * (old[k] / scales[to])[:, None]).to(E4M3).float()
                    cells[to, :, dst[k] % page] = x
        out[name] = cells, scales
    return out


class Pool:
    """A page pool, sequence by sequence and page by page."""

    def __init__(self, B, max_pages, npages, page):
        self.B, self.max_pages, self.npages, self.page = B, max_pages, npages, page
        self.pages = [[] for _ in range(B)]
        self.lens = [0] * B

    def refs(self):
        n = [0] * self.npages
        for p in self.pages:
            for i in p:
                n[i] += 1
        return n

    def fork(self, src):
        pages, lens = [list(p) for p in self.pages], list(self.lens)
        for b, s in enumerate(src):
            if s == -1:
                self.pages[b], self.lens[b] = [], 0
            elif 0 <= s < self.B:
                self.pages[b], self.lens[b] = list(pages[s]), lens[s]

    def reserve(self, new, max_jobs=1 << 30):
        """(jobs, pages taken, refused)"""
        refs, page = self.refs(), self.page
        writers = {}
        for b in range(self.B):
            if new[b] > 0:
                for e in range((self.lens[b] - new[b]) // page,
                               min(len(self.pages[b]), -(-self.lens[b] // page))):
                    writers.setdefault(self.pages[b][e], []).append(b)
        takes = []
        for b in range(self.B):
            need = -(-self.lens[b] // page)
            if new[b] > 0:
                for e in range((self.lens[b] - new[b]) // page, min(len(self.pages[b]), need)):
                    i = self.pages[b][e]
                    alone = len(writers[i]) == refs[i] and writers[i][-1] == b
                    if refs[i] > 1 and not alone:
                        takes.append((b, e, i))
            takes += [(b, e, None) for e in range(len(self.pages[b]), need)]
        free = [i for i, n in enumerate(refs) if n == 0]
        njobs = sum(t[2] is not None for t in takes)
        if len(takes) > len(free) or njobs > max_jobs:
            return [], len(takes), 1
        jobs = []
        for (b, e, i), to in zip(takes, free):
            if i is None:
                self.pages[b].append(to)
            else:
                self.pages[b][e] = to
                jobs.append([i, to])
        return jobs, len(takes), 0

    def trim(self):
        for b in range(self.B):
            del self.pages[b][-(-self.lens[b] // self.page):]
