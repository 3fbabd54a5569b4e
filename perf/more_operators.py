"""Cases for the operators around drafted tokens and shared pages of a paged
key/value cache: the plan of a tree of drafted tokens (who sees whom, at which
position), attention of such a tree over the cache, the rows of a cache that are
kept moved together, and the pages behind the sequences: forked, made writable,
copied and given back.

`own` false: each operator in plain torch operations, in fp32, rounded once at
the end.  `own` true: the calls of this package.

The cache: pages of `page` tokens, [npages, Hkv, page, d] for K and for V, in
bf16 or in e4m3 with one fp32 scale (a power of two) per page and head, a stored
value being code * scale.  Row j of sequence b lies in page
block_table[b, j // page] at row j % page; seq_lens[b] counts the drafted rows too.

A tree of n drafted tokens takes the last n rows of its sequence, a node's parent
before it.  mask[b, t] has bit u (of word u // 32) where node t sees node u: its
ancestors and itself.  All nodes see every row before the tree.

A pool counts for every page the sequences that hold it (refs); sequence b holds
the first held[b] entries of its row of the table.  Pages are taken lowest number
first, by sequence, then by place in the sequence.
"""
import math

import torch

own = False

E4M3 = torch.float8_e4m3fn
DTYPES = {"bf16": torch.bfloat16, "e4m3": E4M3}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one request with eight drafted tokens, a short context: latency
        dict(name="tree_one", op="tree", cache="e4m3", B=1, Hq=32, Hkv=8, T=8, d=128, page=64,
             maxlen=1000, ragged=False, fp32=False),
        # a full batch of ragged contexts, trees of up to 16 tokens
        dict(name="tree_batch", op="tree", cache="bf16", B=64, Hq=32, Hkv=8, T=16, d=128, page=16,
             maxlen=8192, ragged=True, fp32=False),
        # large trees of an odd size over longer contexts in 8 bits
        dict(name="tree_wide", op="tree", cache="e4m3", B=8, Hq=32, Hkv=8, T=60, d=128, page=32,
             maxlen=16384, ragged=False, fp32=False),
        # one request at 128K, results in fp32 to be merged with others
        dict(name="tree_128k", op="tree", cache="bf16", B=1, Hq=32, Hkv=8, T=32, d=64, page=128,
             maxlen=131072, ragged=False, fp32=True),
        # the trees of one step of a batch
        dict(name="plan_step", op="plan", B=64, T=60, ragged=True),
        # deep trees of the most tokens
        dict(name="plan_deep", op="plan", B=256, T=1024, ragged=False),
        # the accepted path of each tree moved behind the context, in 8 bits
        dict(name="compact_path", op="compact", cache="e4m3", B=32, Hkv=4, T=32, d=64, page=32,
             maxlen=128, what="path"),
        # half of the tokens of long contexts thrown out
        dict(name="compact_half", op="compact", cache="bf16", B=16, Hkv=8, T=8191, d=128, page=64,
             maxlen=8192, what="half"),
        # a step of beam search of two requests
        dict(name="beam_step", op="beam", requests=2, beams=4, Hkv=8, d=128, page=16, maxlen=1000),
        # of 64 requests
        dict(name="beam_batch", op="beam", requests=64, beams=4, Hkv=8, d=128, page=64,
             maxlen=4096),
        # room for 32 drafted tokens of a batch, and back what was rejected
        dict(name="slots_step", op="slots", B=64, T=32, page=16, maxlen=2048),
        # for a chunk of prompt of each of many sequences
        dict(name="slots_chunk", op="slots", B=512, T=500, page=16, maxlen=2048),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("tree", "tree", "tree", "plan", "compact", "beam", "slots"))
    d = rng.choice((64, 128, 128))
    page = rng.choice((16, 32, 64, 128))
    cache = rng.choice(("e4m3", "bf16"))
    Hkv = rng.choice((1, 2, 4, 8, 8, 16))
    if op == "plan":
        return dict(op=op, B=_log(rng, 1, 256), T=_log(rng, 1, 1024), ragged=rng.random() < 0.5)
    if op == "beam":
        requests, beams = _log(rng, 1, 64), rng.choice((2, 3, 4, 5, 8))
        cells = requests * Hkv * d
        return dict(op=op, requests=requests, beams=beams, Hkv=Hkv, d=d, page=page,
                    maxlen=_log(rng, 1, max(1, min(16384, (1 << 28) // cells - 3 * beams * page))))
    if op == "slots":
        B = _log(rng, 1, 512)
        T = _log(rng, 1, 500)
        return dict(op=op, B=B, T=T, page=page, maxlen=T + _log(rng, 1, 1500))
    if op == "compact":
        what = rng.choice(("path", "half"))
        B = _log(rng, 1, 64)
        if cache == "e4m3" or what == "path":
            T = _log(rng, 1, 128)
            maxlen = T + _log(rng, 1, 128)
        else:
            maxlen = _log(rng, 2, max(2, min(16384, (1 << 27) // (B * Hkv * d))))
            T = rng.randint(max(1, maxlen // 2), maxlen)
        return dict(op=op, cache=cache, B=B, Hkv=Hkv, T=T, d=d, page=page, maxlen=maxlen,
                    what=what)
    G = rng.choice((1, 2, 4, 8))
    B, T = _log(rng, 1, 64), _log(rng, 1, 128)
    most = min(131072, (1 << 29) // (B * Hkv * d), (1 << 28) // (B * Hkv * G * T))
    return dict(op=op, cache=cache, B=B, Hq=Hkv * G, Hkv=Hkv, T=T, d=d, page=page,
                maxlen=max(T, _log(rng, 1, max(1, most))), ragged=rng.random() < 0.5,
                fp32=rng.random() < 0.25)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _randn(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _ints(g, lo, hi, *shape):
    """Whole numbers in [lo, hi]."""
    return torch.randint(lo, hi + 1, shape, generator=g, device="cuda", dtype=torch.int32)


def _lengths(g, B, lo, hi):
    """Ragged lengths in [lo, hi], the longest always among them."""
    n = _ints(g, lo, hi, B)
    n[B // 2] = hi
    return n


def _cache(g, c, lens):
    """A filled cache whose pages lie in random order, among pages of nobody;
    keys with a few loud channels, as rotated keys have them, and heads and pages
    of different loudness."""
    B, H, d, page = c["B"], c["Hkv"], c["d"], c["page"]
    width = -(-c["maxlen"] // page)
    npages = B * width + 3
    table = torch.randperm(npages, generator=g, device="cuda")[:B * width].to(torch.int32)
    loud = 1.0 + 7.0 * (torch.rand(H, 1, d, generator=g, device="cuda") < 0.05).float()
    by_head = torch.exp(_randn(g, 2, H, 1, 1, dtype=torch.float32))
    s = dict(block_table=table.view(B, width), seq_lens=lens, k_scale=None, v_scale=None)
    for name, gain in (("k", loud * by_head[0]), ("v", by_head[1])):
        x = torch.randn(npages, H, page, d, generator=g, device="cuda") * gain
        if c["cache"] == "e4m3":
            scale = torch.exp2(torch.ceil(torch.log2(x.abs().amax((2, 3)) / 448.0)))
            s[name + "_scale"] = scale
            x = x / scale[:, :, None, None]
        s[name] = x.to(DTYPES[c["cache"]])
    return s


def _parents(g, B, T):
    """Trees as a drafter leaves them: the last accepted token is node 0, most nodes
    hang from one of the few before them, some begin at the context again."""
    t = torch.arange(T, device="cuda")
    back = torch.empty(B, T, device="cuda").exponential_(0.4, generator=g).long() + 1
    parent = (t - back).clamp(min=0)
    root = torch.rand(B, T, generator=g, device="cuda") < 0.03
    return torch.where(root | (t == 0), torch.full_like(parent, -1), parent).to(torch.int32)


def _closure(parents):
    """[B, T, T]: does node t see node u?  Each step doubles how far up it is known."""
    B, T = parents.shape
    sees = torch.eye(T, device="cuda", dtype=torch.bool).repeat(B, 1, 1)
    up = parents.long()
    for _ in range(max(1, (T - 1).bit_length())):
        there = up >= 0
        at = up.clamp(min=0)
        above = torch.gather(sees, 1, at[:, :, None].expand(B, T, T))
        sees = sees | (above & there[:, :, None])
        up = torch.where(there, torch.gather(up, 1, at), up)
    return sees


def _packed(sees):
    """Truth values [..., T] as int32 words, bit u of word u // 32."""
    T = sees.shape[-1]
    sees = torch.nn.functional.pad(sees, (0, -T % 32)).unflatten(-1, (-1, 32))
    w = (sees.long() << torch.arange(32, device="cuda")).sum(-1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)


def _unpacked(mask, T):
    bits = (mask.long()[..., None] >> torch.arange(32, device="cuda")) & 1
    return bits.flatten(-2)[..., :T].bool()


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=c)
    if c["op"] == "beam":
        return s | _prepare_beam(g, c)
    if c["op"] == "slots":
        return s | _prepare_slots(g, c)
    B, T = c["B"], c["T"]
    if c["op"] == "plan":
        s["q_lens"] = _lengths(g, B, 0, T) if c["ragged"] else None
        s["parents"] = _parents(g, B, T)
        cell = dict(B=B, Hkv=1, d=64, page=128, maxlen=128, cache="bf16")
        s |= _cache(g, cell, _ints(g, T, 131072, B))
        s["block_table"] = s["block_table"].expand(B, 1024).contiguous()
        s["mask"] = torch.zeros(B, T, -(-T // 32), device="cuda", dtype=torch.int32)
        s["positions"] = torch.zeros(B, T, device="cuda", dtype=torch.int32)
        return s
    n = _lengths(g, B, 0, T) if c["op"] == "compact" or c["ragged"] else None
    s["q_lens"] = n
    least = torch.full((B,), T, device="cuda", dtype=torch.int32) if n is None else n
    s |= _cache(g, c, torch.maximum(_lengths(g, B, 1, c["maxlen"]), least))
    if c["op"] == "compact":
        t = torch.arange(T, device="cuda")
        if c["what"] == "path":    # a node and its ancestors
            sees = _closure(_parents(g, B, T))
            node = (torch.rand(B, generator=g, device="cuda") * n).long()
            keep = sees[torch.arange(B, device="cuda"), node]
        else:                      # the first ones, the last ones, some in between
            keep = torch.rand(B, T, generator=g, device="cuda") < 0.5
            keep = keep | (t < 4) | (t >= n[:, None] - 64)
        keep = keep & (t < n[:, None])
        s["kept"] = torch.argsort((~keep).to(torch.int8), dim=1, stable=True).to(torch.int32)
        s["kept_lens"] = keep.sum(1).to(torch.int32)
        return s
    s["mask"] = _packed(_closure(_parents(g, B, T)))
    # heads of a packed projection [B, T, H, d]
    s["q"] = _randn(g, B, T, c["Hq"], c["d"]).transpose(1, 2)
    dtype = torch.float32 if c["fp32"] else torch.bfloat16
    s["o"] = torch.zeros(B, c["Hq"], T, c["d"], device="cuda", dtype=dtype)
    s["lse"] = torch.zeros(B, c["Hq"], T, device="cuda")
    return s


def _prepare_beam(g, c):
    """Beams of a request share the full pages of its context and have a last page
    each; every step the beams go on from some of them."""
    R, W, page = c["requests"], c["beams"], c["page"]
    B = R * W
    lens = _lengths(g, R, 1, c["maxlen"]).long()
    held = -(-lens // page)
    width = -(-c["maxlen"] // page)
    e = torch.arange(width, device="cuda")
    npages = R * width + 3 * B + 5
    order = torch.randperm(npages, generator=g, device="cuda")
    shared = order[:R * width].view(R, 1, width)
    tails = order[R * width:R * width + B].view(R, W, 1)
    last = (e == held[:, None] - 1)[:, None]
    table = torch.where(last, tails, shared.expand(R, W, width)).reshape(B, width)
    held = held.repeat_interleave(W)
    refs = torch.bincount(table[e < held[:, None]], minlength=npages).to(torch.int32)
    src = torch.arange(R, device="cuda")[:, None] * W + _ints(g, 0, W - 1, R, W)
    s = dict(block_table=table.to(torch.int32), held=held.to(torch.int32), refs=refs,
             seq_lens=lens.repeat_interleave(W).to(torch.int32),
             src=src.flatten().to(torch.int32), k_scale=None, v_scale=None)
    for name in "kv":
        s[name] = torch.randn(npages, c["Hkv"], page, c["d"], generator=g, device="cuda",
                              dtype=torch.bfloat16)
    s["jobs"] = torch.zeros(2 * B, 2, device="cuda", dtype=torch.int32)
    return s


def _prepare_slots(g, c):
    """Sequences with pages of their own, in a pool with as many free ones again."""
    B, T, page = c["B"], c["T"], c["page"]
    base = _lengths(g, B, 0, c["maxlen"] - T)
    longer = base + T
    kept = base + _ints(g, 0, T, B)
    width = -(-c["maxlen"] // page)
    npages = 2 * B * width + 5
    table = torch.randperm(npages, generator=g, device="cuda")[:B * width].view(B, width)
    held = -(-base // page)
    mine = torch.arange(width, device="cuda") < held[:, None]
    refs = torch.bincount(table[mine], minlength=npages).to(torch.int32)
    return dict(block_table=table.to(torch.int32), held=held.to(torch.int32), refs=refs,
                seq_lens=base.clone(), longer=longer, kept=kept,
                jobs=torch.zeros(B * (T // page + 2), 2, device="cuda", dtype=torch.int32))


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _counts(s):
    n = s["q_lens"]
    return torch.full_like(s["seq_lens"], s["case"]["T"]) if n is None else n


def _plain_plan(s):
    n = _counts(s)
    t = torch.arange(s["case"]["T"], device="cuda")
    there = t < n[:, None]
    sees = _closure(s["parents"])
    depth = sees.sum(-1) - 1
    at = ((s["seq_lens"] - n)[:, None] + depth).to(torch.int32)
    s["mask"] = torch.where(there[..., None], _packed(sees), s["mask"])
    s["positions"] = torch.where(there, at, s["positions"])
    return s["mask"], s["positions"]


def _dense(s, name, L):
    """Cached rows [0, L) as fp32 [B, Hkv, L, d], zero behind a sequence's end."""
    ids = s["block_table"].long()
    x = s[name][ids].float()                                     # [B, pages, H, page, d]
    if s[name + "_scale"] is not None:
        x = x * s[name + "_scale"][ids][..., None, None]
    x = x.transpose(1, 2).flatten(2, 3)[:, :, :L]
    there = torch.arange(L, device="cuda") < s["seq_lens"][:, None]
    return torch.where(there[:, None, :, None], x, torch.zeros_like(x))


def _plain_tree(s):
    c = s["case"]
    B, Hkv, T, d, L = c["B"], c["Hkv"], c["T"], c["d"], c["maxlen"]
    n = _counts(s)
    valid = torch.arange(T, device="cuda") < n[:, None]
    # the key's node: below 0 before the tree, n and above behind the end
    node = torch.arange(L, device="cuda") - (s["seq_lens"] - n)[:, None]
    at = node.clamp(0, T - 1)[:, None].expand(B, T, L)
    seen = torch.gather(_unpacked(s["mask"], T), 2, at) & (node < n[:, None])[:, None]
    seen = seen | (node < 0)[:, None]
    k, v = _dense(s, "k", L), _dense(s, "v", L)
    q = s["q"].float().reshape(B, Hkv, -1, d)
    x = torch.matmul(q, k.transpose(2, 3)).view(B, Hkv, -1, T, L) * (1.0 / math.sqrt(d))
    x = torch.where(seen[:, None, None], x, torch.full_like(x, float("-inf")))
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == float("-inf"), torch.zeros_like(m), m))
    z = p.sum(-1, keepdim=True)
    p = p / torch.where(z == 0, torch.ones_like(z), z)
    o = torch.matmul(p.view(B, Hkv, -1, L), v).view(B, -1, T, d)
    lse = (m + torch.log(z)).view(B, -1, T)
    there = valid[:, None, :]
    s["o"] = torch.where(there[..., None], o.to(s["o"].dtype), s["o"])
    s["lse"] = torch.where(there, lse, s["lse"])
    return s["o"], s["lse"]


def _plain_compact(s):
    c, page, table = s["case"], s["case"]["page"], s["block_table"].long()
    first = (s["seq_lens"] - s["q_lens"]).long()
    b, i = (torch.arange(c["T"], device="cuda") < s["kept_lens"][:, None]).nonzero(as_tuple=True)
    src, dst = first[b] + s["kept"][b, i], first[b] + i
    sp, sr, dp, dr = table[b, src // page], src % page, table[b, dst // page], dst % page
    for name in "kv":
        pages, scales = s[name], s[name + "_scale"]
        rows = pages[sp, :, sr]
        if scales is None:
            pages[dp, :, dr] = rows
            continue
        scale = scales[sp]                                       # [rows, H]
        new = torch.zeros_like(scales).index_reduce_(0, dp, scale, "amax")
        # pages whose first rows stay
        kb = ((first % page > 0) & (s["kept_lens"] > 0)).nonzero()[:, 0]
        kp, kr = table[kb, first[kb] // page], first[kb] % page
        new[kp] = torch.maximum(new[kp], scales[kp])
        was = pages[kp].float()
        stay = (torch.arange(page, device="cuda") < kr[:, None])[:, None, :, None]
        pages[kp] = torch.where(stay, was * (scales[kp] / new[kp])[..., None, None], was).to(E4M3)
        pages[dp, :, dr] = (rows.float() * (scale / new[dp])[..., None]).to(E4M3)
        scales.copy_(torch.where(new > 0, new, scales))
    return _compact_outputs(s)


def _compact_outputs(s):
    """What the cells stand for."""
    return {n: s[n] if s[n + "_scale"] is None else s[n].float() * s[n + "_scale"][..., None, None]
            for n in "kv"}


def _plain_fork(s):
    src, table = s["src"].long(), s["block_table"]
    e = torch.arange(table.shape[1], device="cuda")
    old, held = e < s["held"][:, None], s["held"][src]
    new = e < held[:, None]
    rows = table[src]
    n = s["refs"].shape[0]
    s["refs"] += (torch.bincount(rows[new].long(), minlength=n) -
                  torch.bincount(table[old].long(), minlength=n)).to(torch.int32)
    table.copy_(torch.where(new, rows, table))
    s["held"].copy_(held)
    s["seq_lens"].copy_(s["seq_lens"][src])


def _plain_reserve(s, T):
    """Pages for the last T rows of every sequence: those that are missing, and copies
    of those that others hold too (the last sequence that writes such a page keeps it
    where nobody but writers holds it)."""
    table, held, refs, page = s["block_table"], s["held"], s["refs"], s["case"]["page"]
    B, width = table.shape
    npages = refs.shape[0]
    e = torch.arange(width, device="cuda")
    lens = s["seq_lens"]
    need = -(-lens // page)
    missing = (e >= held[:, None]) & (e < need[:, None])
    written = (e >= ((lens - T) // page)[:, None]) & (e < torch.minimum(need, held)[:, None])
    ids = table.long()
    written = written & (refs[ids.clamp(0, npages - 1)] > 1)
    wb, we = written.nonzero(as_tuple=True)
    wp = ids[wb, we]
    writers = torch.bincount(wp, minlength=npages)
    last = torch.full((npages,), -1, device="cuda").index_reduce_(0, wp, wb, "amax")
    keeps = (writers[wp] == refs[wp]) & (last[wp] == wb)
    copied = torch.zeros_like(written)
    copied[wb, we] = ~keeps
    takes = missing | copied
    b, at = takes.nonzero(as_tuple=True)
    free = (refs == 0).nonzero()[:, 0]
    if b.numel() > free.numel():
        raise RuntimeError("the pool has too few free pages")
    to = free[:b.numel()]
    jobs = copied[b, at]
    pairs = torch.stack((ids[b, at], to), 1)[jobs]
    s["jobs"][:pairs.shape[0]] = pairs.to(torch.int32)
    refs -= torch.bincount(pairs[:, 0], minlength=npages).to(torch.int32)
    refs[to] = 1
    table[b, at] = to.to(torch.int32)
    held.copy_(torch.maximum(held, need))
    return pairs


def _plain_trim(s):
    table, held, page = s["block_table"], s["held"], s["case"]["page"]
    e = torch.arange(table.shape[1], device="cuda")
    need = torch.minimum(held, -(-s["seq_lens"] // page))
    gone = (e >= need[:, None]) & (e < held[:, None])
    s["refs"] -= torch.bincount(table[gone].long(), minlength=s["refs"].shape[0]).to(torch.int32)
    held.copy_(need)


def _pool_outputs(s, *names):
    return {n: s[n] for n in ("block_table", "held", "refs", "seq_lens", "jobs") + names}


def _plain_beam(s):
    _plain_fork(s)
    pairs = _plain_reserve(s, 1)
    for name in "kv":
        s[name][pairs[:, 1]] = s[name][pairs[:, 0]]
    return _pool_outputs(s, "k", "v")


def _plain_slots(s):
    s["seq_lens"].copy_(s["longer"])
    _plain_reserve(s, s["case"]["T"])
    s["seq_lens"].copy_(s["kept"])
    _plain_trim(s)
    return _pool_outputs(s)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _handles(s, dfa):
    """What a program keeps between calls: the cache's and the pool's handle and a
    workspace."""
    if "handles" not in s:
        c = s["case"]
        cache = pool = ws = None
        if "k" in s:
            cache = dfa.PagedCache(s["k"], s["v"], s["block_table"], s["seq_lens"],
                                   k_scale=s["k_scale"], v_scale=s["v_scale"])
            ws = (dfa.tree_workspace(cache, c["Hq"], c["T"]) if c["op"] == "tree" else
                  dfa.paged_workspace(cache))
        if "refs" in s:
            pool = dfa.PagePool(s["block_table"], s["seq_lens"], c["page"], held=s["held"],
                                refs=s["refs"])
        s["handles"] = cache, pool, ws
    return s["handles"]


def _own(s):
    from long_context_flashattention_gb300 import dfa
    c = s["case"]
    cache, pool, ws = _handles(s, dfa)
    if c["op"] == "tree":
        return dfa.decode_tree(cache, s["q"], s["mask"], q_lens=s["q_lens"], out_fp32=c["fp32"],
                               out=s["o"], lse=s["lse"], ws=ws)
    if c["op"] == "plan":
        return dfa.tree_plan(cache, s["parents"], q_lens=s["q_lens"], mask=s["mask"],
                             positions=s["positions"], ws=ws)
    if c["op"] == "compact":
        dfa.cache_compact(cache, s["kept"], s["kept_lens"], q_lens=s["q_lens"], ws=ws)
        return _compact_outputs(s)
    if c["op"] == "beam":
        dfa.pages_fork(pool, s["src"])
        jobs, info = dfa.pages_reserve(pool, 1, jobs=s["jobs"])
        dfa.cache_copy(cache, jobs, info, ws=ws)
        return _pool_outputs(s, "k", "v")
    s["seq_lens"].copy_(s["longer"])
    dfa.pages_reserve(pool, c["T"], jobs=s["jobs"])
    s["seq_lens"].copy_(s["kept"])
    dfa.pages_trim(pool)
    return _pool_outputs(s)


def run(state):
    if own:
        return _own(state)
    plain = dict(tree=_plain_tree, plan=_plain_plan, compact=_plain_compact, beam=_plain_beam,
                 slots=_plain_slots)
    return plain[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# work
# ---------------------------------------------------------------------------
def work(case):
    """Expected over the random lengths and trees."""
    c = case
    if c["op"] == "plan":
        n = c["B"] * c["T"] * (0.5 if c["ragged"] else 1)
        return dict(bytes=n * (8 + 4 * -(-c["T"] // 32)), flops=n * math.log2(2 * c["T"]))
    if c["op"] == "slots":
        pages = c["B"] * (c["T"] / c["page"] + 1)
        return dict(bytes=12 * pages + 24 * c["B"], flops=pages)
    cell = 1 if c.get("cache") == "e4m3" else 2
    row = 2 * c["Hkv"] * c["d"] * cell
    if c["op"] == "beam":
        B, W = c["requests"] * c["beams"], c["beams"]
        copies = c["requests"] * W * (1 - 1 / W) ** W
        return dict(bytes=2 * copies * row * c["page"] + 8 * B * c["maxlen"] / 2 / c["page"],
                    flops=B)
    if c["op"] == "compact":
        moved = c["B"] * min(c["T"], 8 if c["what"] == "path" else c["T"] / 2) / 2
        return dict(bytes=2 * moved * row, flops=moved * row / cell)
    rows = (c["B"] + 1) * c["maxlen"] / 2
    new = c["T"] * (0.5 if c["ragged"] else 1)
    out = (2 + (4 if c["fp32"] else 2)) * c["B"] * new * c["Hq"] * c["d"]
    return dict(bytes=rows * row + out, flops=4 * rows * new * c["Hq"] * c["d"])


# ---------------------------------------------------------------------------
# exact values, in 64 bits, sequence by sequence
# ---------------------------------------------------------------------------
def _exact_rows(s, name, b, n):
    """Cached rows [0, n) of sequence b: [Hkv, n, d]."""
    ids = s["block_table"][b, :-(-n // s["case"]["page"])].tolist()
    x = torch.cat([s[name][i].double() * (1.0 if s[name + "_scale"] is None else
                                          s[name + "_scale"][i].double()[:, None, None])
                   for i in ids], 1)
    return x[:, :n]


def _exact_tree(s):
    c = s["case"]
    o, lse = s["o"].double(), s["lse"].double()
    words = s["mask"].tolist()
    for b, (L, n) in enumerate(zip(s["seq_lens"].tolist(), _counts(s).tolist())):
        if n == 0:
            continue
        k, v = _exact_rows(s, "k", b, L), _exact_rows(s, "v", b, L)
        hidden = torch.tensor([[(words[b][t][u // 32] >> (u % 32)) & 1 == 0 for u in range(n)]
                               for t in range(n)], device="cuda")
        q = s["q"][b, :, :n].double().unflatten(0, (c["Hkv"], -1))
        x = torch.einsum("hgtd,hld->hgtl", q, k) / c["d"] ** 0.5
        x[..., L - n:].masked_fill_(hidden, -math.inf)
        lse[b, :, :n] = torch.logsumexp(x, -1).flatten(0, 1)
        o[b, :, :n] = torch.einsum("hgtl,hld->hgtd", torch.softmax(x, -1), v).flatten(0, 1)
    return o, lse


def _exact_compact(s):
    c, page = s["case"], s["case"]["page"]
    table = s["block_table"].tolist()
    out = {}
    for name in "kv":
        cells, scales = s[name].double(), s[name + "_scale"]
        if scales is not None:
            cells = cells * scales.double()[..., None, None]
        new = cells.clone()
        for b, (L, n, a) in enumerate(zip(s["seq_lens"].tolist(), s["q_lens"].tolist(),
                                          s["kept_lens"].tolist())):
            first, kept = L - n, s["kept"][b, :a].tolist()
            for p in range(first // page, -(-(first + a) // page)):
                lo, hi = max(first, p * page), min(first + a, (p + 1) * page)
                src = [first + kept[j - first] for j in range(lo, hi)]
                if not src:
                    continue
                pg = torch.tensor([table[b][j // page] for j in src], device="cuda")
                at = torch.tensor([j % page for j in src], device="cuda")
                to = table[b][p]
                new[to, :, lo - p * page:hi - p * page] = cells[pg, :, at].transpose(0, 1)
                if scales is not None:
                    # what is behind the last row keeps its codes, under the page's new scale
                    top = scales[pg].amax(0)
                    if lo > p * page:
                        top = torch.maximum(top, scales[to])
                    new[to, :, hi - p * page:] *= (top / scales[to]).double()[:, None, None]
        out[name] = new
    return out


def _exact_beam(s):
    """The beams one after the other; the whole numbers have no such values."""
    page = s["case"]["page"]
    src, lens = s["src"].tolist(), s["seq_lens"].tolist()
    refs = s["refs"].tolist()
    last = [s["block_table"][b, -(-n // page) - 1].item() for b, n in enumerate(lens)]
    new_last = [last[p] for p in src]
    for p in last:
        refs[p] -= 1
    for p in new_last:
        refs[p] += 1
    # (the other pages change hands too, but stay in use)
    free = iter([p for p, r in enumerate(refs) if r == 0])
    out = dict.fromkeys(("block_table", "held", "refs", "seq_lens", "jobs"))
    k, v = s["k"].double(), s["v"].double()
    for b, p in enumerate(new_last):
        if refs[p] > 1:
            to = next(free)
            k[to], v[to] = s["k"][p].double(), s["v"][p].double()
            refs[p] -= 1
    return out | dict(k=k, v=v)


def exact(case, seed):
    if case["op"] in ("plan", "slots"):
        return None                      # whole numbers
    s = prepare(case, seed)
    return dict(tree=_exact_tree, compact=_exact_compact, beam=_exact_beam)[case["op"]](s)
