"""Cases for the serving operators around a paged key/value cache: rotary
positions, the append of new keys and values (rotated and quantised on the
way), the gather of cached rows into contiguous bf16, and decoding attention
that reads the pages.

`own` false: each operator in plain torch operations, in fp32 (angles in fp64),
rounded once at the end.  `own` true: the calls of this package.

The cache: pages of `page` tokens, [npages, Hkv, page, d] for K and for V, in
bf16 or in e4m3 with one fp32 scale per page and head.  A scale is a power of
two, the smallest s with max|x| <= 448 s over the page's rows (2^-100 at
least), so a stored value is code * scale.  Row j of sequence b lies in page
block_table[b, j // page] at row j % page; seq_lens[b] counts the new rows too.
"""
import math

import torch

own = False

E4M3 = torch.float8_e4m3fn
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": E4M3}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one new token of 64 running requests, query and key heads of one
        # packed projection: nothing but latency
        dict(name="rope_token", op="rope", dtype="bf16", B=64, H=40, L=1, d=128, rot=128,
             layout="half", scaling="none", inverse=False, where="positions", packed=True),
        # a 32K prompt straight out of the projection ([B, L, H, d] storage),
        # half layout, frequencies stretched in bands for a longer context
        dict(name="rope_prefill", op="rope", dtype="bf16", B=1, H=32, L=32768, d=128, rot=128,
             layout="half", scaling="bands", inverse=False, where="natural", packed=True),
        # gradients of fp32 keys through the rotation of half of the head,
        # positions that restart with each packed document, an odd length
        dict(name="rope_grad", op="rope", dtype="fp32", B=2, H=8, L=16381, d=128, rot=64,
             layout="interleaved", scaling="linear", inverse=True, where="documents",
             packed=False),
        # one decoding step of 64 requests: rotate q and k, store k and v
        dict(name="append_token", op="append", cache="e4m3", B=64, Hq=32, Hkv=8, T=1, d=128,
             page=64, maxlen=8192, rot=128, layout="half", scaling="none", ragged=False),
        # a mixed batch: prompts' chunks of 0 to 1000 tokens on top of what is
        # there already, small pages, part of the head rotated
        dict(name="append_chunks", op="append", cache="e4m3", B=16, Hq=8, Hkv=4, T=1000, d=64,
             page=16, maxlen=4096, rot=32, layout="interleaved", scaling="none", ragged=True),
        # a 32K prompt stored in bf16
        dict(name="append_prompt", op="append", cache="bf16", B=1, Hq=32, Hkv=32, T=32768,
             d=128, page=128, maxlen=32768, rot=128, layout="half", scaling="bands",
             ragged=False),
        # a short context brought back for a chunk of prompt that attends to it
        dict(name="gather_chunk", op="gather", cache="e4m3", B=4, Hkv=8, d=64, page=16,
             maxlen=1021, pos0=0, L=1021),
        # two 64K contexts brought back from 8 bits
        dict(name="gather_64k", op="gather", cache="e4m3", B=2, Hkv=8, d=128, page=64,
             maxlen=65536, pos0=0, L=65536),
        # one request, a short context: latency
        dict(name="decode_one", op="decode", cache="e4m3", B=1, Hq=32, Hkv=8, T=1, d=128,
             page=64, maxlen=1000, ragged=False),
        # a full batch of ragged contexts
        dict(name="decode_batch", op="decode", cache="e4m3", B=64, Hq=32, Hkv=8, T=1, d=128,
             page=64, maxlen=8192, ragged=False),
        # one request at 128K without head sharing
        dict(name="decode_128k", op="decode", cache="e4m3", B=1, Hq=32, Hkv=32, T=1, d=128,
             page=128, maxlen=131072, ragged=False),
        # up to four drafted tokens a request, checked in one pass over bf16 pages
        dict(name="decode_draft", op="decode", cache="bf16", B=16, Hq=32, Hkv=8, T=4, d=128,
             page=16, maxlen=8192, ragged=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rope", "append", "gather", "decode", "decode"))
    d = rng.choice((64, 128, 128))
    rot = rng.choice((d, d, d // 2, d // 4))
    layout = rng.choice(("half", "interleaved"))
    scaling = rng.choice(("none", "linear", "bands"))
    page = rng.choice((16, 32, 64, 128))
    cache = rng.choice(("e4m3", "e4m3", "bf16"))
    Hkv = rng.choice((1, 2, 4, 8, 8, 32))
    if op == "rope":
        B, H = _log(rng, 1, 64), _log(rng, 1, 64)
        L = _log(rng, 1, max(1, min(65536, (1 << 27) // (B * H * d))))
        return dict(op=op, dtype=rng.choice(("bf16", "bf16", "fp32")), B=B, H=H, L=L, d=d,
                    rot=rot, layout=layout, scaling=scaling, inverse=rng.random() < 0.5,
                    where=rng.choice(("positions", "natural", "documents", "striped")),
                    packed=rng.random() < 0.5)
    G = rng.choice((1, 2, 4, 8)) if Hkv < 32 else 1
    if op == "append":
        B = _log(rng, 1, 128)
        T = _log(rng, 1, max(1, min(32768, (1 << 26) // (B * Hkv * G * d))))
        return dict(op=op, cache=cache, B=B, Hq=Hkv * G, Hkv=Hkv, T=T, d=d, page=page,
                    maxlen=T + _log(rng, 1, 2048), rot=rot, layout=layout, scaling=scaling,
                    ragged=rng.random() < 0.5)
    B = _log(rng, 1, 64)
    maxlen = _log(rng, 1, max(1, min(131072, (1 << 27) // (B * Hkv * d))))
    if op == "gather":
        pos0 = rng.randrange(maxlen) if rng.random() < 0.3 else 0
        return dict(op=op, cache=cache, B=B, Hkv=Hkv, d=d, page=page, maxlen=maxlen, pos0=pos0,
                    L=maxlen - pos0)
    return dict(op=op, cache=cache, B=B, Hq=Hkv * G, Hkv=Hkv, T=rng.choice((1, 1, 1, 2, 3, 5)),
                d=d, page=page, maxlen=maxlen, ragged=rng.random() < 0.5)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _randn(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _rows(g, B, H, L, d, dtype, packed):
    """[B, H, L, d], as a view of [B, L, H, d] where the rows come from a projection."""
    if packed:
        return _randn(g, B, L, H, d, dtype=dtype).transpose(1, 2)
    return _randn(g, B, H, L, d, dtype=dtype)


def _lengths(g, B, lo, hi):
    """Ragged lengths in [lo, hi], the longest always among them."""
    n = torch.randint(lo, hi + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    n[B // 2] = hi
    return n


def _cache(g, c, lens):
    """A filled cache whose pages lie in random order, among pages of nobody;
    keys with a few loud channels, as rotated keys have them, and heads of
    different loudness."""
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


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=c)
    if c["op"] == "rope":
        s["x"] = _rows(g, c["B"], c["H"], c["L"], c["d"], DTYPES[c["dtype"]], c["packed"])
        s["positions"] = None
        if c["where"] == "positions":    # each request at a position of its own
            first = torch.randint(0, 131072, (c["B"], 1), generator=g, device="cuda",
                                  dtype=torch.int32)
            s["positions"] = first + torch.arange(c["L"], device="cuda", dtype=torch.int32)
        elif c["where"] == "documents":  # restarting every few hundred tokens
            start = torch.rand(c["B"], c["L"], generator=g, device="cuda") < 0.003
            at = torch.arange(c["L"], device="cuda", dtype=torch.int32).expand(c["B"], -1)
            last = torch.where(start, at, torch.zeros_like(at)).cummax(1).values
            s["positions"] = (at - last).contiguous()
        return s
    if c["op"] == "gather":
        s |= _cache(g, c, _lengths(g, c["B"], 1, c["maxlen"]))
        s["k_out"], s["v_out"] = (torch.zeros(c["B"], c["Hkv"], c["L"], c["d"], device="cuda",
                                              dtype=torch.bfloat16) for _ in range(2))
        return s
    T = c["T"]
    new = _lengths(g, c["B"], 0, T) if c["ragged"] else None
    s["new_lens"] = new
    least = torch.full((c["B"],), T, device="cuda", dtype=torch.int32) if new is None else new
    s |= _cache(g, c, torch.maximum(_lengths(g, c["B"], 1, c["maxlen"]), least))
    s["q"] = _rows(g, c["B"], c["Hq"], T, c["d"], torch.bfloat16, True)
    if c["op"] == "append":
        s["k_new"] = _rows(g, c["B"], c["Hkv"], T, c["d"], torch.bfloat16, True)
        s["v_new"] = _rows(g, c["B"], c["Hkv"], T, c["d"], torch.bfloat16, True)
        s["q_out"] = torch.zeros(c["B"], c["Hq"], T, c["d"], device="cuda", dtype=torch.bfloat16)
    else:
        s["o"] = torch.zeros(c["B"], c["Hq"], T, c["d"], device="cuda", dtype=torch.bfloat16)
        s["lse"] = torch.zeros(c["B"], c["Hq"], T, device="cuda")
    return s


SCALING = {"none": {}, "linear": dict(factor=4.0),
           "bands": dict(factor=8.0, orig_len=8192, low=1.0, high=4.0, gain=1.1)}
BASE = 10000.0
STRIPES = 8  # "striped": the rows are worker 3's of 8 token stripes


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _angles(c, pos):
    """cos and sin (fp32, gain included) of positions [...] -> [..., rot/2]."""
    half = c["rot"] // 2
    kw = SCALING[c["scaling"]]
    f = BASE ** (-2.0 * torch.arange(half, device="cuda", dtype=torch.float64) / c["rot"])
    if c["scaling"] == "linear":
        f = f / kw["factor"]
    elif c["scaling"] == "bands":
        turns = kw["orig_len"] * f / (2 * math.pi)
        keep = ((turns - kw["low"]) / (kw["high"] - kw["low"])).clamp(0, 1)
        f = keep * f + (1 - keep) * f / kw["factor"]
    a = pos.double()[..., None] * f
    gain = kw.get("gain", 1.0)
    return (gain * torch.cos(a)).float(), (gain * torch.sin(a)).float()


def _rotate(c, x, cos, sin):
    """x fp32 [B, H, L, d]; cos, sin [B, 1, L, rot/2]."""
    rot = c["rot"]
    head, rest = x[..., :rot], x[..., rot:]
    if c["layout"] == "half":
        a, b = head[..., :rot // 2], head[..., rot // 2:]
        head = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    else:
        a, b = head[..., 0::2], head[..., 1::2]
        head = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    return torch.cat((head, rest), -1)


def _rope_positions(s):
    c = s["case"]
    if s["positions"] is not None:
        return s["positions"]
    at = torch.arange(c["L"], device="cuda")
    return (at * STRIPES + 3 if c["where"] == "striped" else at).expand(c["B"], -1)


def _plain_rope(s):
    c = s["case"]
    cos, sin = _angles(c, _rope_positions(s))
    if c["inverse"]:
        sin = -sin
    return _rotate(c, s["x"].float(), cos[:, None], sin[:, None]).to(s["x"].dtype)


def _store(s, name, x, slot, valid):
    """Put rows x fp32 [B, H, T, d] into the pages at slots [B, T] where valid."""
    c, page = s["case"], s["case"]["page"]
    pages = s[name]
    b, t = valid.nonzero(as_tuple=True)
    j = slot[b, t]
    to = s["block_table"][b, j // page].long()
    row = j % page
    if c["cache"] == "bf16":
        pages[to, :, row] = x[b, :, t].to(torch.bfloat16)
        return
    scales = s[name + "_scale"]
    vals = x[b, :, t]                                            # [n, H, d]
    need = torch.zeros_like(scales)
    need.index_reduce_(0, to, vals.abs().amax(-1), "amax")       # largest new value of a page
    m, e = torch.frexp(need)                                     # m in [0.5, 1)
    e = torch.where(need > 0, e - 9 + (m > 0.875).int(), torch.full_like(e, -100)).clamp(min=-100)
    need = torch.ldexp(torch.ones_like(scales), e)
    touched = torch.unique(to)
    first = torch.zeros(scales.shape[0], device="cuda", dtype=torch.bool)
    first[to[row == 0]] = True                                   # pages begun by these rows
    begin = torch.full((scales.shape[0],), page, device="cuda")  # first new row of a page
    begin.index_reduce_(0, to, row, "amin")
    old = scales[touched]
    new = torch.where(first[touched][:, None], need[touched], torch.maximum(old, need[touched]))
    was = pages[touched].float()                                 # [pages, H, page, d]
    before = torch.arange(page, device="cuda") < begin[touched][:, None]
    kept = torch.where(before[:, None, :, None], was * (old / new)[:, :, None, None], was)
    pages[touched] = kept.to(E4M3)
    scales[touched] = new
    pages[to, :, row] = (vals / scales[to][..., None]).to(E4M3)


def _new_rows(s):
    """(slots [B, T], valid [B, T]) of the new tokens."""
    c = s["case"]
    t = torch.arange(c["T"], device="cuda")
    n = torch.full_like(s["seq_lens"], c["T"]) if s["new_lens"] is None else s["new_lens"]
    return (s["seq_lens"] - n)[:, None] + t, t < n[:, None]


def _plain_append(s):
    c = s["case"]
    slot, valid = _new_rows(s)
    cos, sin = (a[:, None] for a in _angles(c, slot))
    _store(s, "k", _rotate(c, s["k_new"].float(), cos, sin), slot, valid)
    _store(s, "v", s["v_new"].float(), slot, valid)
    q = _rotate(c, s["q"].float(), cos, sin).to(torch.bfloat16)
    s["q_out"] = torch.where(valid[:, None, :, None], q, s["q_out"])
    return _append_outputs(s)


def _append_outputs(s):
    out = {n: s[n] for n in ("q_out", "k", "v")}
    return out | ({n: s[n] for n in ("k_scale", "v_scale")} if s["k_scale"] is not None else {})


def _dense(s, name, pos0, L):
    """Cached rows [pos0, pos0 + L) as fp32 [B, Hkv, L, d], zero behind a sequence's end."""
    page = s["case"]["page"]
    j = torch.arange(pos0, pos0 + L, device="cuda")
    p0, p1 = pos0 // page, -(-(pos0 + L) // page)
    ids = s["block_table"][:, p0:p1].long()
    x = s[name][ids].float()                                     # [B, pages, H, page, d]
    if s[name + "_scale"] is not None:
        x = x * s[name + "_scale"][ids][..., None, None]
    x = x.transpose(1, 2).flatten(2, 3)[:, :, pos0 - p0 * page:][:, :, :L]
    return torch.where((j < s["seq_lens"][:, None])[:, None, :, None], x, torch.zeros_like(x))


def _plain_gather(s):
    c = s["case"]
    j = torch.arange(c["pos0"], c["pos0"] + c["L"], device="cuda")
    there = (j < s["seq_lens"][:, None])[:, None, :, None]
    for name in ("k", "v"):
        x = _dense(s, name, c["pos0"], c["L"]).to(torch.bfloat16)
        s[name + "_out"] = torch.where(there, x, s[name + "_out"])
    return s["k_out"], s["v_out"]


def _plain_decode(s):
    c = s["case"]
    B, Hkv, T, d = c["B"], c["Hkv"], c["T"], c["d"]
    L = c["maxlen"]
    slot, valid = _new_rows(s)
    k, v = _dense(s, "k", 0, L), _dense(s, "v", 0, L)
    q = s["q"].float().reshape(B, Hkv, -1, d)
    x = torch.matmul(q, k.transpose(2, 3)).view(B, Hkv, -1, T, L) * (1.0 / math.sqrt(d))
    seen = torch.arange(L, device="cuda") <= slot[:, :, None]    # [B, T, L]
    x = torch.where(seen[:, None, None], x, torch.full_like(x, float("-inf")))
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m)
    n = p.sum(-1, keepdim=True)
    o = torch.matmul((p / n).view(B, Hkv, -1, L), v).view(B, -1, T, d)
    lse = (m + torch.log(n)).view(B, -1, T)
    there = valid[:, None, :]
    s["o"] = torch.where(there[..., None], o.to(torch.bfloat16), s["o"])
    s["lse"] = torch.where(there, lse, s["lse"])
    return s["o"], s["lse"]


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _kept(s, dfa):
    """What a program keeps between calls: the rotation, the cache's handle and a workspace."""
    if "kept" not in s:
        c = s["case"]
        rope = (dfa.rope_spec(c["d"], layout=c["layout"], rot_dim=c["rot"], theta_base=BASE,
                              scaling=c["scaling"], **SCALING[c["scaling"]])
                if "rot" in c else None)
        cache = ws = pmap = None
        if c["op"] == "rope":
            if c["where"] == "striped":
                pmap = dfa.partition_map(c["L"] * STRIPES, STRIPES, 3, "striped")
        else:
            cache = dfa.PagedCache(s["k"], s["v"], s["block_table"], s["seq_lens"],
                                   k_scale=s["k_scale"], v_scale=s["v_scale"])
            ws = dfa.paged_workspace(cache, c.get("Hq", c["Hkv"]), c.get("T", 1))
        s["kept"] = rope, cache, ws, pmap
    return s["kept"]


def _own(s):
    from long_context_flashattention_gb300 import dfa
    c = s["case"]
    rope, cache, ws, pmap = _kept(s, dfa)
    if c["op"] == "rope":
        return dfa.rope(s["x"], rope, positions=s["positions"], pos_map=pmap,
                        inverse=c["inverse"])
    if c["op"] == "append":
        dfa.cache_append(cache, s["k_new"], s["v_new"], rope=rope, new_lens=s["new_lens"],
                         q=s["q"], q_out=s["q_out"], ws=ws)
        return _append_outputs(s)
    if c["op"] == "gather":
        return dfa.cache_gather(cache, c["L"], pos0=c["pos0"], k_out=s["k_out"],
                                v_out=s["v_out"], ws=ws)
    return dfa.decode_paged(cache, s["q"], q_lens=s["new_lens"], out=s["o"], lse=s["lse"], ws=ws)


def run(state):
    if own:
        return _own(state)
    plain = dict(rope=_plain_rope, append=_plain_append, gather=_plain_gather,
                 decode=_plain_decode)
    return plain[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# work
# ---------------------------------------------------------------------------
def work(case):
    """Expected over the random lengths (uniform up to the longest)."""
    c = case
    if c["op"] == "rope":
        n = c["B"] * c["H"] * c["L"] * c["d"]
        size = 2 if c["dtype"] == "bf16" else 4
        return dict(bytes=2 * n * size, flops=3 * n * c["rot"] / c["d"])
    cell = 1 if c["cache"] == "e4m3" else 2
    if c["op"] == "append":
        rows = c["B"] * c["T"] * (0.5 if c["ragged"] else 1)
        n, nq = 2 * rows * c["Hkv"] * c["d"], rows * c["Hq"] * c["d"]
        return dict(bytes=n * (2 + cell) + 4 * nq, flops=3 * (n / 2 + nq) + n)
    rows = (c["B"] + 1) * c["maxlen"] / 2
    if c["op"] == "gather":
        rows *= c["L"] / c["maxlen"]
        n = 2 * rows * c["Hkv"] * c["d"]
        return dict(bytes=n * (cell + 2), flops=n)
    new = c["T"] * (0.5 if c["ragged"] else 1)
    return dict(bytes=2 * rows * c["Hkv"] * c["d"] * cell + 4 * c["B"] * new * c["Hq"] * c["d"],
                flops=4 * rows * new * c["Hq"] * c["d"])


# ---------------------------------------------------------------------------
# exact values, in 64 bits, sequence by sequence
# ---------------------------------------------------------------------------
def _turned(c, x, pos, sign=1.0):
    """Rows x [H, n, d] (fp64) at positions [n]: each feature pair as a complex
    number times gain * exp(i * angle)."""
    rot, kw = c["rot"], SCALING[c["scaling"]]
    freqs = []
    for i in range(rot // 2):
        f = BASE ** (-2.0 * i / rot)
        if c["scaling"] == "linear":
            f /= kw["factor"]
        elif c["scaling"] == "bands":
            wave = 2.0 * math.pi / f
            if wave > kw["orig_len"] / kw["low"]:
                f /= kw["factor"]
            elif wave > kw["orig_len"] / kw["high"]:
                u = (kw["orig_len"] / wave - kw["low"]) / (kw["high"] - kw["low"])
                f = (1 - u) * f / kw["factor"] + u * f
        freqs.append(f)
    a = sign * pos.double()[:, None] * torch.tensor(freqs, device=x.device, dtype=torch.float64)
    w = torch.polar(torch.full_like(a, kw.get("gain", 1.0)), a)
    pairs = (x[..., :rot].unflatten(-1, (2, rot // 2)).movedim(-2, -1) if c["layout"] == "half"
             else x[..., :rot].unflatten(-1, (rot // 2, 2)))
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * w)
    z = z.movedim(-1, -2).flatten(-2) if c["layout"] == "half" else z.flatten(-2)
    return torch.cat((z, x[..., rot:]), -1)


def _exact_rope(s):
    c = s["case"]
    sign = -1.0 if c["inverse"] else 1.0
    out = torch.empty(c["B"], c["H"], c["L"], c["d"], device="cuda", dtype=torch.float64)
    for b in range(c["B"]):
        if s["positions"] is not None:
            pos = s["positions"][b]
        else:
            pos = torch.arange(c["L"], device="cuda")
            pos = STRIPES * pos + 3 if c["where"] == "striped" else pos
        out[b] = _turned(c, s["x"][b].double(), pos, sign)
    return out


def _exact_append(s):
    c, page = s["case"], s["case"]["page"]
    out = {n: s[n].double() for n in ("q_out", "k", "v")}
    if c["cache"] == "e4m3":
        out |= {n: s[n].double() for n in ("k_scale", "v_scale")}
    lens = s["seq_lens"].tolist()
    news = [c["T"]] * c["B"] if s["new_lens"] is None else s["new_lens"].tolist()
    for b in range(c["B"]):
        n, first = news[b], lens[b] - news[b]
        if n == 0:
            continue
        pos = torch.arange(first, lens[b], device="cuda")
        out["q_out"][b, :, :n] = _turned(c, s["q"][b, :, :n].double(), pos)
        for name, x in (("k", _turned(c, s["k_new"][b, :, :n].double(), pos)),
                        ("v", s["v_new"][b, :, :n].double())):
            for p in range(first // page, (lens[b] - 1) // page + 1):
                lo, hi = max(first, p * page), min(lens[b], (p + 1) * page)
                to = int(s["block_table"][b, p])
                rows = x[:, lo - first:hi - first]
                if c["cache"] == "e4m3":
                    top = rows.abs().amax((1, 2)).tolist()
                    for h in range(c["Hkv"]):
                        e = -100
                        if top[h] > 0:
                            m, e = math.frexp(top[h])
                            e = max(-100, e - (9 if m <= 0.875 else 8))
                        scale, old = 2.0 ** e, float(out[name + "_scale"][to, h])
                        if lo > p * page:
                            scale = max(scale, old)
                            out[name][to, h, :lo - p * page] *= old / scale
                        out[name + "_scale"][to, h] = scale
                    rows = rows / out[name + "_scale"][to][:, None, None]
                out[name][to, :, lo - p * page:hi - p * page] = rows
    return out


def _exact_rows(s, name, b, n):
    """Cached rows [0, n) of sequence b: [Hkv, n, d]."""
    ids = s["block_table"][b, :-(-n // s["case"]["page"])].tolist()
    x = torch.cat([s[name][i].double() * (1.0 if s[name + "_scale"] is None else
                                          s[name + "_scale"][i].double()[:, None, None])
                   for i in ids], 1)
    return x[:, :n]


def _exact_gather(s):
    c = s["case"]
    out = [torch.zeros(c["B"], c["Hkv"], c["L"], c["d"], device="cuda", dtype=torch.float64)
           for _ in range(2)]
    for b, n in enumerate(s["seq_lens"].tolist()):
        n = min(n, c["pos0"] + c["L"])
        if n > c["pos0"]:
            for o, name in zip(out, "kv"):
                o[b, :, :n - c["pos0"]] = _exact_rows(s, name, b, n)[:, c["pos0"]:]
    return tuple(out)


def _exact_decode(s):
    c = s["case"]
    G = c["Hq"] // c["Hkv"]
    o, lse = s["o"].double(), s["lse"].double()
    news = [c["T"]] * c["B"] if s["new_lens"] is None else s["new_lens"].tolist()
    for b, n in enumerate(s["seq_lens"].tolist()):
        if news[b] == 0:
            continue
        k, v = _exact_rows(s, "k", b, n), _exact_rows(s, "v", b, n)
        for t in range(news[b]):
            upto = n - news[b] + t + 1
            q = s["q"][b, :, t].double().view(c["Hkv"], G, -1)
            x = torch.einsum("hgd,hnd->hgn", q, k[:, :upto]) / c["d"] ** 0.5
            lse[b, :, t] = torch.logsumexp(x, -1).flatten()
            o[b, :, t] = torch.einsum("hgn,hnd->hgd", torch.softmax(x, -1),
                                      v[:, :upto]).reshape(-1, c["d"])
    return o, lse


def exact(case, seed):
    if case["op"] == "append" and case["cache"] == "e4m3":
        pages = case["B"] * (case["T"] // case["page"] + 2)
        if pages * case["Hkv"] > 40000:  # scale by scale on the host: too long
            return None
    s = prepare(case, seed)
    return dict(rope=_exact_rope, append=_exact_append, gather=_exact_gather,
                decode=_exact_decode)[case["op"]](s)
