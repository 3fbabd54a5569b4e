"""Thin ctypes binding over libdfa (include/dfa.h).

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind the C ABI.  PyTorch supplies device memory and the current
stream.  There is no fallback: if libdfa.so is missing or a call fails, an
exception is raised.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import re

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
# DFA_DEBUG_BOUNDS=1 loads the bounds-checking build of the library instead
DEBUG_BOUNDS = os.environ.get("DFA_DEBUG_BOUNDS") == "1"
LIB_PATH = os.path.join(_PKG, "libdfa_bounds.so" if DEBUG_BOUNDS else "libdfa.so")
HEADER = os.path.join(os.path.dirname(_PKG), "include", "dfa.h")

PARTITIONS = {"contiguous": 0, "balanced": 1, "striped": 2}
OP_FWD, OP_BWD, OP_CHUNK_FWD, OP_CHUNK_BWD, OP_RING_FWD = 0, 1, 2, 3, 4
STATUS = {0: "DFA_OK", 1: "DFA_ERR_INVALID_ARG", 2: "DFA_ERR_UNSUPPORTED",
          3: "DFA_ERR_WORKSPACE", 4: "DFA_ERR_CUDA", 5: "DFA_ERR_TIMEOUT", 6: "DFA_ERR_BOUNDS"}


class DfaError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{STATUS.get(code, code)}: {msg}")
        self.code = code


class AttnDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32),
                ("N", ctypes.c_int64), ("d", ctypes.c_int32), ("causal", ctypes.c_int32),
                ("scale", ctypes.c_float), ("P", ctypes.c_int32), ("partition", ctypes.c_int32),
                ("stripe", ctypes.c_int32), ("o_fp32", ctypes.c_int32),
                ("ndocs", ctypes.c_int32), ("doc_bounds", ctypes.c_void_p)]


class PosMap(ctypes.Structure):
    _fields_ = [("nseg", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("len", ctypes.c_int64 * 2), ("base", ctypes.c_int64 * 2),
                ("blk", ctypes.c_int64), ("blk_stride", ctypes.c_int64)]


class ChunkPair(ctypes.Structure):
    _fields_ = [("q", PosMap), ("kv", PosMap)]


class RingWorker(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("kv_slots", ctypes.c_void_p), ("o", ctypes.c_void_p), ("lse", ctypes.c_void_p)]


class HostStep(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("dout", ctypes.c_void_p), ("o", ctypes.c_void_p), ("lse", ctypes.c_void_p),
                ("dq", ctypes.c_void_p), ("dk", ctypes.c_void_p), ("dv", ctypes.c_void_p)]


class SchedPair(ctypes.Structure):
    _fields_ = [("worker", ctypes.c_int32), ("step", ctypes.c_int32),
                ("kv_worker", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("tokens", ctypes.c_int64), ("first_item", ctypes.c_int64),
                ("n_items", ctypes.c_int64)]


class SchedItem(ctypes.Structure):
    _fields_ = [("worker", ctypes.c_int32), ("step", ctypes.c_int32), ("q_tile", ctypes.c_int32),
                ("kv_begin", ctypes.c_int32), ("kv_end", ctypes.c_int32),
                ("mask_class", ctypes.c_int32)]


class Schedule(ctypes.Structure):
    _fields_ = [("pair_tokens", ctypes.POINTER(ctypes.c_int64)),
                ("tile_counts", ctypes.POINTER(ctypes.c_int64)),
                ("total_pairs", ctypes.c_int64), ("eta_slots", ctypes.c_double),
                ("eta_flops", ctypes.c_double), ("pairs", ctypes.POINTER(SchedPair)),
                ("items", ctypes.POINTER(SchedItem)), ("capacity", ctypes.c_int64),
                ("n_items", ctypes.c_int64)]


TILE_SKIP, TILE_FULL, TILE_PARTIAL = 0, 1, 2


class RopeSpec(ctypes.Structure):
    _fields_ = [("layout", ctypes.c_int32), ("rot_dim", ctypes.c_int32),
                ("scaling", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("theta_base", ctypes.c_double), ("factor", ctypes.c_double),
                ("orig_len", ctypes.c_double), ("low", ctypes.c_double),
                ("high", ctypes.c_double), ("gain", ctypes.c_double)]


class PagedCacheDesc(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("page", ctypes.c_int32), ("Hkv", ctypes.c_int32),
                ("d", ctypes.c_int32), ("npages", ctypes.c_int64),
                ("page_stride", ctypes.c_int64), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("B", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("block_table", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p),
                ("status", ctypes.c_void_p)]


class PagePoolDesc(ctypes.Structure):
    _fields_ = [("page", ctypes.c_int32), ("B", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("npages", ctypes.c_int64),
                ("block_table", ctypes.c_void_p), ("held", ctypes.c_void_p),
                ("refs", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p),
                ("status", ctypes.c_void_p)]


ROPE_LAYOUTS = {"interleaved": 0, "half": 1}
ROPE_SCALINGS = {"none": 0, "linear": 1, "bands": 2}


_lib = None


def lib():
    """Load libdfa.so (building it first if the sources are newer)."""
    global _lib
    if _lib is None:
        from . import build as _build
        if not _build.up_to_date(debug_bounds=DEBUG_BOUNDS):
            _build.build(debug_bounds=DEBUG_BOUNDS)
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libdfa.so not found at {LIB_PATH}; run build()")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        D = ctypes.POINTER(AttnDesc)
        C = ctypes.POINTER(PagedCacheDesc)
        P = ctypes.POINTER(PagePoolDesc)
        sigs = {
            "dfa_attn_fwd": (i32, [D, vp, vp, vp, vp, vp, vp, sz, vp]),
            "dfa_attn_bwd": (i32, [D, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
            "dfa_attn_bwd_noalloc": (i32, [D, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]),
            "dfa_chunk_fwd": (i32, [D, ctypes.POINTER(ChunkPair), i64, i64, vp, vp, vp, vp, vp,
                                    vp, sz, vp]),
            "dfa_chunk_bwd": (i32, [D, ctypes.POINTER(ChunkPair), i64, i64, vp, vp, vp, vp, vp,
                                    vp, vp, vp, vp, vp, vp, sz, vp]),
            "dfa_lse_merge": (i32, [i64, i32, i32, vp, vp, vp, vp, i32, i32, vp]),
            "dfa_permute": (i32, [D, i32, vp, vp, i32, i64, i64, vp]),
            "dfa_permute_rope": (i32, [D, i32, vp, vp, i64, ctypes.c_float, vp]),
            "dfa_ring_fwd": (i32, [D, ctypes.POINTER(RingWorker), vp, sz, i32, vp, vp]),
            "dfa_attn_step_host_workspace_size": (sz, [D, i32]),
            "dfa_attn_step_host": (i32, [D, vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, vp, sz, vp,
                                         vp, vp]),
            "dfa_attn_steps_host": (i32, [D, i32, ctypes.POINTER(HostStep), i32, vp, sz, vp, vp,
                                          vp]),
            "dfa_decode_workspace_size": (sz, [D, i32, i64, i32]),
            "dfa_decode": (i32, [D, i32, i64, i64, vp, vp, vp, vp, vp, i32, vp, sz, vp]),
            "dfa_rope": (i32, [ctypes.POINTER(RopeSpec), i32, i32, i64, i32, i32, vp, vp, vp, vp,
                               ctypes.POINTER(PosMap), vp, i32, vp]),
            "dfa_cache_append": (i32, [C, ctypes.POINTER(RopeSpec), i32, vp, vp, vp, vp, vp, i32,
                                       vp, vp, vp, vp, vp, sz, vp]),
            "dfa_cache_gather": (i32, [C, i64, i64, vp, vp, vp, sz, vp]),
            "dfa_decode_paged_workspace_size": (sz, [D, i32]),
            "dfa_decode_paged": (i32, [D, C, i32, vp, vp, vp, vp, vp, vp, sz, vp]),
            "dfa_cache_append_at": (i32, [C, ctypes.POINTER(RopeSpec), i32, vp, vp, vp, vp, vp, vp,
                                          i32, vp, vp, vp, vp, vp, sz, vp]),
            "dfa_tree_plan": (i32, [C, i32, vp, vp, vp, vp, vp, sz, vp]),
            "dfa_decode_tree_workspace_size": (sz, [D, i32]),
            "dfa_decode_tree": (i32, [D, C, i32, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
            "dfa_cache_compact": (i32, [C, i32, vp, i32, vp, vp, vp, sz, vp]),
            "dfa_cache_copy": (i32, [C, vp, i32, vp, vp, sz, vp]),
            "dfa_pages_workspace_size": (sz, [P]),
            "dfa_pages_fork": (i32, [P, vp, vp, sz, vp]),
            "dfa_pages_reserve": (i32, [P, i32, vp, vp, i32, vp, vp, sz, vp]),
            "dfa_pages_trim": (i32, [P, vp, sz, vp]),
            "dfa_make_schedule": (i32, [D, i32, i32, ctypes.POINTER(Schedule)]),
            "dfa_partition_map": (i32, [D, i32, ctypes.POINTER(PosMap)]),
            "dfa_workspace_size": (sz, [D, i32]),
            "dfa_stream_status": (i32, [vp, vp]),
            "dfa_selftest_timeout": (i32, [vp, i64, vp]),
            "dfa_status_string": (ctypes.c_char_p, [i32]),
            "dfa_last_error": (ctypes.c_char_p, []),
            "dfa_version": (i32, []),
        }
        for name, (res, args) in sigs.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def header_symbols():
    """Names of the functions declared in include/dfa.h."""
    txt = open(HEADER).read()
    return sorted(set(re.findall(r"^\s*(?:const\s+)?[a-z_0-9]+\s*\*?\s*(dfa_[a-z_0-9]+)\s*\(",
                                 txt, re.M)))


def _check(code: int):
    if code != 0:
        raise DfaError(code, lib().dfa_last_error().decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def make_desc(B, Hq, Hkv, N, d, causal=True, scale=None, P=1, partition="contiguous",
              stripe=1, o_fp32=False, docs=None) -> AttnDesc:
    """docs: None, or an int64 CUDA tensor of ndocs + 1 cumulative document
    bounds in global positions (kept alive by the descriptor)."""
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    nd, ptr = 0, None
    if docs is not None:
        if not docs.is_cuda or docs.dtype != torch.int64 or docs.dim() != 1 or docs.numel() < 2:
            raise ValueError("docs must be a 1-D int64 CUDA tensor of >= 2 bounds")
        nd, ptr = docs.numel() - 1, docs.data_ptr()
    desc = AttnDesc(B, Hq, Hkv, N, d, int(causal), float(scale), P, PARTITIONS[partition],
                    stripe, int(o_fp32), nd, ptr)
    desc._docs = docs
    return desc


def desc_for(q, k, **kw) -> AttnDesc:
    B, Hq, N, d = q.shape
    return make_desc(B, Hq, k.shape[1], N, d, **kw)


def workspace_size(desc: AttnDesc, op: int) -> int:
    return int(lib().dfa_workspace_size(ctypes.byref(desc), op))


def new_workspace(desc: AttnDesc, op: int, device=None) -> torch.Tensor:
    n = workspace_size(desc, op)
    if n == 0:
        raise DfaError(1, "invalid descriptor for workspace sizing: " +
                       lib().dfa_last_error().decode())
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def _need_cuda(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("tensors must be contiguous CUDA tensors")


# ----------------------------------------------------------------------------
# whole-sequence attention
# ----------------------------------------------------------------------------
def attn_fwd(q, k, v, causal=True, scale=None, P=1, partition="contiguous", stripe=1,
             o_fp32=False, ws=None, out=None, lse=None, stream=None, docs=None):
    """Attention forward.  q [B,Hq,N,d], k/v [B,Hkv,N,d] bf16, rows in the
    worker-major order of the partition (natural order for contiguous).
    Returns (O, LSE)."""
    _need_cuda(q, k, v)
    desc = desc_for(q, k, causal=causal, scale=scale, P=P, partition=partition, stripe=stripe,
                    o_fp32=o_fp32, docs=docs)
    B, Hq, N, d = q.shape
    if out is None:
        out = torch.empty(B, Hq, N, d, dtype=torch.float32 if o_fp32 else torch.bfloat16,
                          device=q.device)
    if lse is None:
        lse = torch.empty(B, Hq, N, dtype=torch.float32, device=q.device)
    if ws is None:
        ws = new_workspace(desc, OP_FWD, q.device)
    _check(lib().dfa_attn_fwd(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(out),
                              _ptr(lse), _ptr(ws), ws.numel(), _stream(stream)))
    return out, lse


def attn_bwd(q, k, v, o, dout, lse, causal=True, scale=None, P=1, partition="contiguous",
             stripe=1, ws=None, dq=None, dk=None, dv=None, stream=None, docs=None):
    """Recomputation backward.  Returns (dQ, dK, dV) in bf16."""
    _need_cuda(q, k, v, o, dout, lse)
    desc = desc_for(q, k, causal=causal, scale=scale, P=P, partition=partition, stripe=stripe,
                    docs=docs)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    if ws is None:
        ws = new_workspace(desc, OP_BWD, q.device)
    _check(lib().dfa_attn_bwd(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(o),
                              _ptr(dout), _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(ws),
                              ws.numel(), _stream(stream)))
    return dq, dk, dv


def attn_bwd_noalloc(q, k, v, o, dout, lse, causal=True, scale=None, P=1,
                     partition="contiguous", stripe=1, dq=None, dk=None, dv=None, stream=None):
    """attn_bwd without a workspace: the library's fixed 64 MiB device scratch is
    used instead (for callers that cannot allocate; calls must not overlap)."""
    _need_cuda(q, k, v, o, dout, lse)
    desc = desc_for(q, k, causal=causal, scale=scale, P=P, partition=partition, stripe=stripe)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    _check(lib().dfa_attn_bwd_noalloc(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(o),
                                      _ptr(dout), _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv),
                                      _stream(stream)))
    return dq, dk, dv


# ----------------------------------------------------------------------------
# chunk pairs
# ----------------------------------------------------------------------------
def pos_map(nseg=1, len=(0, 0), base=(0, 0), blk=1, blk_stride=1) -> PosMap:
    m = PosMap()
    m.nseg = nseg
    m.len[0], m.len[1] = len
    m.base[0], m.base[1] = base
    m.blk = blk
    m.blk_stride = blk_stride
    return m


def partition_map(N, P, p, partition="contiguous", stripe=1) -> PosMap:
    desc = make_desc(1, 1, 1, N, 64, P=P, partition=partition, stripe=stripe)
    m = PosMap()
    _check(lib().dfa_partition_map(ctypes.byref(desc), p, ctypes.byref(m)))
    return m


def chunk_fwd(q, k, v, qmap: PosMap, kvmap: PosMap, causal=True, scale=None, ws=None,
              o_part=None, lse_part=None, stream=None, docs=None):
    """Partial (O fp32, LSE) of one chunk pair at the given global positions."""
    _need_cuda(q, k, v)
    B, Hq, Lq, d = q.shape
    Lk = k.shape[2]
    desc = make_desc(B, Hq, k.shape[1], max(Lq, Lk), d, causal=causal, scale=scale, docs=docs)
    pair = ChunkPair(qmap, kvmap)
    if o_part is None:
        o_part = torch.empty(B, Hq, Lq, d, dtype=torch.float32, device=q.device)
    if lse_part is None:
        lse_part = torch.empty(B, Hq, Lq, dtype=torch.float32, device=q.device)
    if ws is None:
        ws = new_workspace(desc, OP_CHUNK_FWD, q.device)
    _check(lib().dfa_chunk_fwd(ctypes.byref(desc), ctypes.byref(pair), Lq, Lk, _ptr(q), _ptr(k),
                               _ptr(v), _ptr(o_part), _ptr(lse_part), _ptr(ws), ws.numel(),
                               _stream(stream)))
    return o_part, lse_part


def chunk_bwd(q, k, v, o, dout, lse, qmap: PosMap, kvmap: PosMap, dq_acc, dk_acc, dv_acc,
              delta=None, causal=True, scale=None, ws=None, stream=None, docs=None):
    """Accumulate one chunk pair's gradient contribution (fp32 accumulators)."""
    _need_cuda(q, k, v, dout, lse, dq_acc, dk_acc, dv_acc)
    B, Hq, Lq, d = q.shape
    Lk = k.shape[2]
    desc = make_desc(B, Hq, k.shape[1], Lq, d, causal=causal, scale=scale, docs=docs)
    pair = ChunkPair(qmap, kvmap)
    if ws is None:
        ws = new_workspace(desc, OP_CHUNK_BWD, q.device)
    _check(lib().dfa_chunk_bwd(ctypes.byref(desc), ctypes.byref(pair), Lq, Lk, _ptr(q), _ptr(k),
                               _ptr(v), _ptr(o), _ptr(dout), _ptr(lse), _ptr(delta),
                               _ptr(dq_acc), _ptr(dk_acc), _ptr(dv_acc), _ptr(ws), ws.numel(),
                               _stream(stream)))


def lse_merge(o_parts, lse_parts, out_fp32=True, o_out=None, lse_out=None, accumulate=False,
              stream=None):
    """Merge k partials: o_parts [k, rows, d] fp32, lse_parts [k, rows] fp32."""
    _need_cuda(o_parts, lse_parts)
    k, rows, d = o_parts.shape
    if o_out is None:
        o_out = torch.empty(rows, d, dtype=torch.float32 if out_fp32 else torch.bfloat16,
                            device=o_parts.device)
    if lse_out is None:
        lse_out = torch.empty(rows, dtype=torch.float32, device=o_parts.device)
    _check(lib().dfa_lse_merge(rows, d, k, _ptr(o_parts), _ptr(lse_parts), _ptr(o_out),
                               _ptr(lse_out), int(out_fp32), int(accumulate), _stream(stream)))
    return o_out, lse_out


def permute(x, P, partition, inverse=False, stripe=1, out=None, stream=None):
    """Reorder the token axis (dim 2 of [B,H,N,d], or dim 2 of [B,H,N]) between
    natural order and the partition's worker-major order."""
    _need_cuda(x)
    if x.dim() == 4:
        B, H, N, d = x.shape
        row = d
    elif x.dim() == 3:
        B, H, N = x.shape
        row = 1
    else:
        raise ValueError("expected [B,H,N,d] or [B,H,N]")
    desc = make_desc(1, 1, 1, N, 64, P=P, partition=partition, stripe=stripe)
    out = torch.empty_like(x) if out is None else out
    _check(lib().dfa_permute(ctypes.byref(desc), int(inverse), _ptr(x), _ptr(out),
                             x.element_size(), row, B * H, _stream(stream)))
    return out


def permute_rope(x, P, partition, inverse=False, stripe=1, theta_base=10000.0, out=None,
                 stream=None):
    """dfa_permute of bf16 [B,H,N,d] query or key rows with the rotary embedding
    applied at each token's global position (inverse: the transposed rotation
    and the inverse permutation, for dQ / dK)."""
    _need_cuda(x)
    if x.dim() != 4 or x.dtype != torch.bfloat16:
        raise ValueError("expected bf16 [B,H,N,d]")
    B, H, N, d = x.shape
    desc = make_desc(1, 1, 1, N, d, P=P, partition=partition, stripe=stripe)
    out = torch.empty_like(x) if out is None else out
    _check(lib().dfa_permute_rope(ctypes.byref(desc), int(inverse), _ptr(x), _ptr(out), B * H,
                                  float(theta_base), _stream(stream)))
    return out


def decode(q, k, v, q_pos0=None, causal=True, scale=None, split_len=512, out_fp32=False,
           ws=None, out=None, lse=None, stream=None):
    """Split-KV decoding (dfa_decode): q [B,Hq,T,d] bf16 at positions q_pos0 + t
    (default: the last T positions of the cache) against k, v [B,Hkv,L,d]."""
    _need_cuda(q, k, v)
    B, Hq, T, d = q.shape
    Hkv, L = k.shape[1], k.shape[2]
    if q_pos0 is None:
        q_pos0 = L - T
    desc = make_desc(B, Hq, Hkv, L, d, causal=causal, scale=scale, o_fp32=out_fp32)
    if ws is None:
        n = int(lib().dfa_decode_workspace_size(ctypes.byref(desc), T, L, split_len))
        if n == 0:
            raise DfaError(1, "bad decode arguments")
        ws = torch.empty(n, dtype=torch.uint8, device=q.device)
    if out is None:
        out = torch.empty(B, Hq, T, d, dtype=torch.float32 if out_fp32 else torch.bfloat16,
                          device=q.device)
    if lse is None:
        lse = torch.empty(B, Hq, T, dtype=torch.float32, device=q.device)
    _check(lib().dfa_decode(ctypes.byref(desc), T, L, int(q_pos0), _ptr(q), _ptr(k), _ptr(v),
                            _ptr(out), _ptr(lse), split_len, _ptr(ws), ws.numel(),
                            _stream(stream)))
    return out, lse


_copy_streams = {}


def ring_fwd(q_chunks, k_chunks, v_chunks, partition, stripe=1, causal=True, scale=None,
             overlap=True, outs=None, slots=None, ws=None, stream=None, copy_stream=None):
    """The ring schedule on one GPU (dfa_ring_fwd): worker p holds chunk p of the
    partition (q [B,Hq,n,d], k/v [B,Hkv,n,d] bf16, worker-major chunks); returns
    [(o [B,Hq,n,d] fp32, lse [B,Hq,n] fp32)] per worker.  With overlap the K/V
    hand-over runs on a second stream (copy_stream, or one kept per device)."""
    P = len(q_chunks)
    _need_cuda(*q_chunks, *k_chunks, *v_chunks)
    B, Hq, n, d = q_chunks[0].shape
    Hkv = k_chunks[0].shape[1]
    dev = q_chunks[0].device
    desc = make_desc(B, Hq, Hkv, n * P, d, causal=causal, scale=scale, P=P,
                     partition=partition, stripe=stripe)
    if outs is None:
        outs = [(torch.empty(B, Hq, n, d, dtype=torch.float32, device=dev),
                 torch.empty(B, Hq, n, dtype=torch.float32, device=dev)) for _ in range(P)]
    if slots is None:
        slots = [torch.empty(4 * B * Hkv * n * d, dtype=torch.bfloat16, device=dev)
                 for _ in range(P)]
    if ws is None:
        ws = new_workspace(desc, OP_RING_FWD, dev)
    if overlap and copy_stream is None:
        copy_stream = _copy_streams.setdefault(dev, torch.cuda.Stream(dev))
    arr = (RingWorker * P)(*[RingWorker(q.data_ptr(), k.data_ptr(), v.data_ptr(), sl.data_ptr(),
                                        o.data_ptr(), l.data_ptr())
                             for q, k, v, sl, (o, l) in zip(q_chunks, k_chunks, v_chunks, slots,
                                                            outs)])
    _check(lib().dfa_ring_fwd(ctypes.byref(desc), arr, _ptr(ws), ws.numel(), int(overlap),
                              _stream(stream), _stream(copy_stream) if overlap else None))
    return outs


_up_streams, _down_streams = {}, {}


def step_host_workspace(desc: AttnDesc, kv_heads_per_group=0, device=None) -> torch.Tensor:
    n = int(lib().dfa_attn_step_host_workspace_size(ctypes.byref(desc), kv_heads_per_group))
    if n == 0:
        raise DfaError(1, "invalid arguments for workspace sizing: " +
                       lib().dfa_last_error().decode())
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def attn_step_host(q, k, v, dout, causal=True, scale=None, P=1, partition="contiguous",
                   stripe=1, docs=None, kv_heads_per_group=0, outs=None, ws=None, overlap=True,
                   stream=None, h2d_stream=None, d2h_stream=None):
    """One attention training step from host memory (dfa_attn_step_host): q/dout
    [B,Hq,N,d], k/v [B,Hkv,N,d] bf16 CPU tensors in natural order (pinned for
    the copies to overlap the compute).  Returns CPU tensors (o, lse, dq, dk,
    dv), pinned when allocated here; they hold the results once the compute
    stream has passed the call (e.g. after torch.cuda.synchronize()).  With
    overlap the uploads and downloads run on two extra streams (given, or kept
    per device)."""
    for t in (q, k, v, dout):
        if t.is_cuda or not t.is_contiguous() or t.dtype != torch.bfloat16:
            raise ValueError("q, k, v, dout must be contiguous bf16 host tensors")
    desc = desc_for(q, k, causal=causal, scale=scale, P=P, partition=partition, stripe=stripe,
                    docs=docs)
    B, Hq, N, d = q.shape
    Hkv = k.shape[1]
    dev = torch.device("cuda", torch.cuda.current_device())
    if outs is None:
        def pinned(*shape, dtype=torch.bfloat16):
            return torch.empty(*shape, dtype=dtype, pin_memory=True)
        outs = (pinned(B, Hq, N, d), pinned(B, Hq, N, dtype=torch.float32), pinned(B, Hq, N, d),
                pinned(B, Hkv, N, d), pinned(B, Hkv, N, d))
    for t in outs:
        if t.is_cuda or not t.is_contiguous():
            raise ValueError("outputs must be contiguous host tensors")
    if ws is None:
        ws = step_host_workspace(desc, kv_heads_per_group, dev)
    if overlap:
        h2d_stream = h2d_stream or _up_streams.setdefault(dev, torch.cuda.Stream(dev))
        d2h_stream = d2h_stream or _down_streams.setdefault(dev, torch.cuda.Stream(dev))
    o, lse, dq, dk, dv = outs
    _check(lib().dfa_attn_step_host(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(dout),
                                    _ptr(o), _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv),
                                    kv_heads_per_group, _ptr(ws), ws.numel(), _stream(stream),
                                    _stream(h2d_stream) if overlap else None,
                                    _stream(d2h_stream) if overlap else None))
    return outs


def attn_steps_host(steps, causal=True, scale=None, P=1, partition="contiguous", stripe=1,
                    docs=None, kv_heads_per_group=0, outs=None, ws=None, overlap=True,
                    stream=None, h2d_stream=None, d2h_stream=None):
    """Several steps from host memory in one call (dfa_attn_steps_host): steps
    is a list of (q, k, v, dout) bf16 host tensors of one shape; outs a list of
    (o, lse, dq, dk, dv) host tensors per step (allocated pinned when None).
    Returns outs."""
    if not steps:
        raise ValueError("need at least one step")
    q0, k0 = steps[0][0], steps[0][1]
    for st in steps:
        for t, ref in zip(st, steps[0]):
            if (t.is_cuda or not t.is_contiguous() or t.dtype != torch.bfloat16 or
                    t.shape != ref.shape):
                raise ValueError("steps must be contiguous bf16 host tensors of one shape")
    desc = desc_for(q0, k0, causal=causal, scale=scale, P=P, partition=partition, stripe=stripe,
                    docs=docs)
    B, Hq, N, d = q0.shape
    Hkv = k0.shape[1]
    dev = torch.device("cuda", torch.cuda.current_device())
    if outs is None:
        def pinned(*shape, dtype=torch.bfloat16):
            return torch.empty(*shape, dtype=dtype, pin_memory=True)
        outs = [(pinned(B, Hq, N, d), pinned(B, Hq, N, dtype=torch.float32), pinned(B, Hq, N, d),
                 pinned(B, Hkv, N, d), pinned(B, Hkv, N, d)) for _ in steps]
    if len(outs) != len(steps):
        raise ValueError("one output set per step")
    for o in outs:
        for t in o:
            if t.is_cuda or not t.is_contiguous():
                raise ValueError("outputs must be contiguous host tensors")
    if ws is None:
        ws = step_host_workspace(desc, kv_heads_per_group, dev)
    if overlap:
        h2d_stream = h2d_stream or _up_streams.setdefault(dev, torch.cuda.Stream(dev))
        d2h_stream = d2h_stream or _down_streams.setdefault(dev, torch.cuda.Stream(dev))
    arr = (HostStep * len(steps))(*[
        HostStep(q.data_ptr(), k.data_ptr(), v.data_ptr(), do.data_ptr(), o.data_ptr(),
                 l.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr())
        for (q, k, v, do), (o, l, dq, dk, dv) in zip(steps, outs)])
    _check(lib().dfa_attn_steps_host(ctypes.byref(desc), len(steps), arr, kv_heads_per_group,
                                     _ptr(ws), ws.numel(), _stream(stream),
                                     _stream(h2d_stream) if overlap else None,
                                     _stream(d2h_stream) if overlap else None))
    return outs


# ----------------------------------------------------------------------------
# rotary positions and the paged key/value cache
# ----------------------------------------------------------------------------
def rope_spec(d, layout="interleaved", rot_dim=None, theta_base=10000.0, scaling="none",
              factor=1.0, orig_len=0.0, low=0.0, high=0.0, gain=1.0) -> RopeSpec:
    """A rotary embedding (dfa_rope_spec) of the first rot_dim (default: all) of
    d features: layout "interleaved" (pairs 2t, 2t+1) or "half" (t, t +
    rot_dim/2); scaling "none", "linear" (factor) or "bands" (factor, orig_len,
    low, high); gain multiplies the rotated features."""
    return RopeSpec(ROPE_LAYOUTS[layout], d if rot_dim is None else rot_dim,
                    ROPE_SCALINGS[scaling], 0, theta_base, factor, orig_len, low, high, gain)


# The calls below are made once per layer and decoded token, so their Python
# part is kept short: descriptors and stride arrays are made once per value, and
# the stream and device are asked for without building objects.
_Strides = ctypes.c_int64 * 3


@functools.lru_cache(maxsize=4096)
def _strides(st):
    return _Strides(st[0], st[1], st[2]) if st[3] == 1 else None


def _rows(t, name, dtype, device, shape):
    """Pointer and strides of a [B,H,L,d] row tensor with contiguous features."""
    if t.dtype is not dtype or t.device != device or t.shape != shape:
        raise ValueError(f"{name} must be a {dtype} {list(shape)} tensor on {device}, not "
                         f"{t.dtype} {list(t.shape)} on {t.device}")
    st = _strides(t.stride())
    if st is None:
        raise ValueError(f"the features of {name} must be contiguous")
    return t.data_ptr(), st


def _int32(t, name, shape, device):
    if t is None:
        return None
    if t.dtype != torch.int32 or t.device != device or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 {list(shape)} tensor on {device}")
    return t.data_ptr()


def _raw_stream(device, stream):
    """The call's stream; its kernels run on the current device, so the tensors
    have to be there."""
    if device.type != "cuda" or device.index != torch._C._cuda_getDevice():
        raise ValueError(f"tensors must be on the current CUDA device, not on {device}")
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(device.index)


def _new(stream, shape, dtype, device):
    """Memory that the call's stream may use at once (and keeps until it is done)."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream())
    return t


def rope(x, spec: RopeSpec, positions=None, pos_map: PosMap | None = None, inverse=False,
         out=None, stream=None):
    """Rotate rows x [B,H,L,d] (bf16 or fp32; any strides with contiguous
    features) at positions [B,L] int32, or at those of pos_map, or at 0..L-1
    (dfa_rope).  inverse: the transposed rotation, for gradients.  out=x works in
    place; without out a contiguous tensor is returned."""
    dev, dtype, shape = x.device, x.dtype, x.shape
    raw = _raw_stream(dev, stream)
    if dtype is not torch.bfloat16 and dtype is not torch.float32 or len(shape) != 4:
        raise ValueError("x must be a bf16 or fp32 [B,H,L,d] tensor")
    if positions is not None and pos_map is not None:
        raise ValueError("give positions or pos_map, not both")
    xp, xs = _rows(x, "x", dtype, dev, shape)
    B, H, L, d = shape
    if out is None:
        out = _new(stream, shape, dtype, dev)
        op, os_ = out.data_ptr(), None
    else:
        op, os_ = (xp, xs) if out is x else _rows(out, "out", dtype, dev, shape)
    code = lib().dfa_rope(ctypes.byref(spec), B, H, L, d, dtype is torch.float32, xp, xs, op, os_,
                          None if pos_map is None else ctypes.byref(pos_map),
                          _int32(positions, "positions", (B, L), dev), inverse, raw)
    if code:
        _check(code)
    return out


class PagedCache:
    """A paged key/value cache (dfa_paged_cache) over the caller's tensors, which
    it keeps alive: k, v [npages,Hkv,page,d], bf16 or float8_e4m3fn (pages may be
    strided: k and v can be two halves of one tensor), with k_scale and v_scale
    [npages,Hkv] fp32 for 8 bits; block_table [B,max_pages] and seq_lens [B]
    int32.  Change their contents freely (cache.seq_lens += 1); a new table or
    batch is a new PagedCache: the calls go by the tensors it was made with.

    The device checks lengths and pages.  A call that was given no workspace reports
    them to cache.status, one with a workspace to that: stream_status(cache.status)
    or stream_status(ws) raises what was found."""

    def __init__(self, k, v, block_table, seq_lens, k_scale=None, v_scale=None):
        dev = k.device
        if k.dim() != 4 or k.dtype not in (torch.bfloat16, torch.float8_e4m3fn):
            raise ValueError("k must be a bf16 or float8_e4m3fn [npages,Hkv,page,d] tensor")
        if v.shape != k.shape or v.dtype != k.dtype or v.stride() != k.stride():
            raise ValueError("k and v must agree in shape, dtype and strides")
        npages, Hkv, page, d = k.shape
        # (the strides of dimensions of one element say nothing)
        inner = zip(k.shape[1:], k.stride()[1:], (page * d, d, 1))
        if any(n > 1 and st != want for n, st, want in inner) or (
                npages > 1 and k.stride(0) < Hkv * page * d):
            raise ValueError("the heads, rows and features of a page must be contiguous")
        if block_table.dim() != 2:
            raise ValueError("block_table must be [B, max_pages]")
        B, max_pages = block_table.shape
        e4m3 = k.dtype == torch.float8_e4m3fn
        if e4m3 != (k_scale is not None) or e4m3 != (v_scale is not None):
            raise ValueError("an 8-bit cache has k_scale and v_scale, a bf16 cache has none")
        for t in (k_scale, v_scale):
            if t is not None and (t.dtype != torch.float32 or t.shape != (npages, Hkv) or
                                  not t.is_contiguous()):
                raise ValueError("scales must be contiguous fp32 [npages, Hkv] tensors")
        for t in (v, block_table, seq_lens, k_scale, v_scale):
            if t is not None and t.device != dev:
                raise ValueError("the cache's tensors must be on one device")
        self.device, self.dtype = dev, k.dtype
        self.B, self.Hkv, self.page, self.d = B, Hkv, page, d
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.block_table, self.seq_lens = block_table, seq_lens
        self.desc = PagedCacheDesc(
            int(e4m3), page, Hkv, d, npages, k.stride(0) if npages > 1 else 0, k.data_ptr(),
            v.data_ptr(), k_scale.data_ptr() if e4m3 else None,
            v_scale.data_ptr() if e4m3 else None, B, max_pages,
            _int32(block_table, "block_table", (B, max_pages), dev),
            _int32(seq_lens, "seq_lens", (B,), dev))
        self._ref = ctypes.byref(self.desc)
        # for calls without a workspace, whose own nobody could read
        self.status = torch.zeros(256, dtype=torch.uint8, device=dev)
        self._own = PagedCacheDesc.from_buffer_copy(self.desc)
        self._own.status = self.status.data_ptr()
        self._own_ref = ctypes.byref(self._own)

    def __setattr__(self, name, value):
        if self.__dict__.get(name, value) is not value:
            raise AttributeError(f"{name} of a PagedCache stays: change its contents, or make a "
                                 "new PagedCache")
        super().__setattr__(name, value)

    def __delattr__(self, name):
        raise AttributeError(f"{name} of a PagedCache stays: change its contents")


def paged_workspace(cache: PagedCache, Hq=None, T=1) -> torch.Tensor:
    """A workspace for the calls on this cache: Hq query heads, T tokens a
    sequence at most.  It serves one call at a time, and the device's errors are then
    reported to it."""
    # more rows than decode_paged takes: the other calls need the status word only
    n = _paged_desc(cache.B, Hq or cache.Hkv, cache.Hkv, T, cache.d, True, 1.0, False)[1]
    return torch.zeros(n, dtype=torch.uint8, device=cache.device)


def _ws(ws, nbytes, cache, stream):
    """A call's workspace, and the cache as the call sees it: errors go to the caller's
    workspace, without one to the cache's status."""
    if ws is None:
        return _new(stream, (nbytes,), torch.uint8, cache.device), cache._own_ref
    if ws.dtype is not torch.uint8 or ws.device != cache.device or not ws.is_contiguous():
        raise ValueError(f"ws must be a contiguous uint8 tensor on {cache.device}")
    return ws, cache._ref


def _plain(t, name, dtype, device, shape):
    if (t.dtype is not dtype or t.device != device or t.shape != shape or
            not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {dtype} {list(shape)} tensor on {device}")
    return t.data_ptr()


@functools.lru_cache(maxsize=1024)
def _paged_desc(B, Hq, Hkv, T, d, causal, scale, fp32):
    """dfa_decode_paged's descriptor (by reference) and workspace bytes (256 at
    least: an invalid one is for the call to refuse)."""
    ref = ctypes.byref(AttnDesc(B, Hq, Hkv, 1, d, causal, scale, 1, 0, 1, fp32, 0, None))
    return ref, max(256, int(lib().dfa_decode_paged_workspace_size(ref, T)))


def cache_append(cache: PagedCache, k, v, rope: RopeSpec | None = None, new_lens=None, q=None,
                 q_out=None, ws=None, stream=None, positions=None):
    """Store the new rows k, v [B,Hkv,T,d] bf16 (any strides with contiguous
    features) of every sequence at the end of its cached rows, keys rotated by
    rope on the way (dfa_cache_append).  cache.seq_lens counts them already;
    new_lens [B] int32: how many of the T are a sequence's (default: all).  With
    q [B,Hq,T,d] its rows are rotated too, into q_out (default: a new contiguous
    tensor; rows from new_lens on are not written), which is returned.  positions
    [B,T] int32: where the rotation takes the rows to be, instead of where they are
    stored (dfa_cache_append_at; tree_plan makes those of a tree)."""
    dev = cache.device
    raw = _raw_stream(dev, stream)
    if k.dim() != 4 or q is not None and q.dim() != 4:
        raise ValueError("k, v and q must be [B,H,T,d]")
    T = k.shape[2]
    shape = (cache.B, cache.Hkv, T, cache.d)
    kp, ks = _rows(k, "k", torch.bfloat16, dev, shape)
    vp, vs = _rows(v, "v", torch.bfloat16, dev, shape)
    ws, ref = _ws(ws, 256, cache, stream)
    Hq, qp, qs, op, os_ = 0, None, None, None, None
    if q is not None:
        Hq = q.shape[1]
        shape = (cache.B, Hq, T, cache.d)
        qp, qs = _rows(q, "q", torch.bfloat16, dev, shape)
        if q_out is None:
            q_out = _new(stream, shape, torch.bfloat16, dev)
            op = q_out.data_ptr()
        else:
            op, os_ = _rows(q_out, "q_out", torch.bfloat16, dev, shape)
    elif q_out is not None:
        raise ValueError("q_out without q")
    spec = None if rope is None else ctypes.byref(rope)
    new = _int32(new_lens, "new_lens", (cache.B,), dev)
    if positions is None:
        code = lib().dfa_cache_append(ref, spec, T, new, kp, ks, vp, vs, Hq, qp, qs, op, os_,
                                      ws.data_ptr(), ws.numel(), raw)
    else:
        code = lib().dfa_cache_append_at(ref, spec, T, new,
                                         _int32(positions, "positions", (cache.B, T), dev), kp,
                                         ks, vp, vs, Hq, qp, qs, op, os_, ws.data_ptr(),
                                         ws.numel(), raw)
    if code:
        _check(code)
    return q_out


def cache_gather(cache: PagedCache, L, pos0=0, k_out=None, v_out=None, ws=None, stream=None):
    """Cached rows [pos0, pos0 + L) of every sequence as contiguous bf16
    [B,Hkv,L,d] (dfa_cache_gather): returns (k_out, v_out).  Rows behind a
    sequence's end are not written."""
    dev = cache.device
    raw = _raw_stream(dev, stream)
    shape = (cache.B, cache.Hkv, L, cache.d)
    if k_out is None:
        k_out = _new(stream, shape, torch.bfloat16, dev)
    if v_out is None:
        v_out = _new(stream, shape, torch.bfloat16, dev)
    ws, ref = _ws(ws, 256, cache, stream)
    code = lib().dfa_cache_gather(ref, pos0, L,
                                  _plain(k_out, "k_out", torch.bfloat16, dev, shape),
                                  _plain(v_out, "v_out", torch.bfloat16, dev, shape),
                                  ws.data_ptr(), ws.numel(), raw)
    if code:
        _check(code)
    return k_out, v_out


def decode_paged(cache: PagedCache, q, q_lens=None, causal=True, scale=None, out_fp32=False,
                 ws=None, out=None, lse=None, stream=None):
    """Attention of the last tokens of every sequence over its cached rows
    (dfa_decode_paged): q [B,Hq,T,d] bf16 (any strides with contiguous features),
    q_lens [B] int32 of the T tokens per sequence (default: all), the last of
    them at position seq_lens - 1.  Returns (O [B,Hq,T,d], LSE [B,Hq,T]); rows
    from q_lens on are not written."""
    dev = cache.device
    raw = _raw_stream(dev, stream)
    shape = q.shape
    if len(shape) != 4:
        raise ValueError("q must be [B,Hq,T,d]")
    B, Hq, T, d = shape
    qp, qs = _rows(q, "q", torch.bfloat16, dev, (cache.B, Hq, T, cache.d))
    o_dtype = torch.float32 if out_fp32 else torch.bfloat16
    if out is None:
        out = _new(stream, shape, o_dtype, dev)
    if lse is None:
        lse = _new(stream, (B, Hq, T), torch.float32, dev)
    desc, need = _paged_desc(B, Hq, cache.Hkv, T, d, bool(causal),
                             1.0 / math.sqrt(d) if scale is None else scale, bool(out_fp32))
    ws, ref = _ws(ws, need, cache, stream)
    code = lib().dfa_decode_paged(desc, ref, T, _int32(q_lens, "q_lens", (B,), dev), qp, qs,
                                  _plain(out, "out", o_dtype, dev, shape),
                                  _plain(lse, "lse", torch.float32, dev, (B, Hq, T)),
                                  ws.data_ptr(), ws.numel(), raw)
    if code:
        _check(code)
    return out, lse


# ----------------------------------------------------------------------------
# branching sequences: trees of drafted tokens, kept rows, shared pages
# ----------------------------------------------------------------------------
def _words(T):
    return (T + 31) // 32


def tree_plan(cache: PagedCache, parents, q_lens=None, mask=None, positions=None, ws=None,
              stream=None):
    """Plan of the trees of drafted tokens in the last q_lens [B] int32 (default: T) rows
    of every sequence (dfa_tree_plan).  parents [B,T] int32: the node that a node
    continues, one before it, or -1 for the context.  Returns (mask [B,T,ceil(T/32)]
    int32: bit u of row t where node t sees node u, its ancestors and itself; positions
    [B,T] int32: the context's length plus the node's depth).  Rows from q_lens on are not
    written."""
    dev = cache.device
    raw = _raw_stream(dev, stream)
    if parents.dim() != 2:
        raise ValueError("parents must be [B, T]")
    B, T = cache.B, parents.shape[1]
    par = _int32(parents, "parents", (B, T), dev)
    if mask is None:
        mask = _new(stream, (B, T, _words(T)), torch.int32, dev)
    if positions is None:
        positions = _new(stream, (B, T), torch.int32, dev)
    ws, ref = _ws(ws, 256, cache, stream)
    code = lib().dfa_tree_plan(ref, T, _int32(q_lens, "q_lens", (B,), dev), par,
                               _int32(mask, "mask", (B, T, _words(T)), dev),
                               _int32(positions, "positions", (B, T), dev), ws.data_ptr(),
                               ws.numel(), raw)
    if code:
        _check(code)
    return mask, positions


@functools.lru_cache(maxsize=1024)
def _tree_desc(B, Hq, Hkv, T, d, scale, fp32):
    """dfa_decode_tree's descriptor (by reference) and workspace bytes (256 at least:
    an invalid one is for the call to refuse)."""
    ref = ctypes.byref(AttnDesc(B, Hq, Hkv, 1, d, True, scale, 1, 0, 1, fp32, 0, None))
    return ref, max(256, int(lib().dfa_decode_tree_workspace_size(ref, T)))


def tree_workspace(cache: PagedCache, Hq=None, T=1) -> torch.Tensor:
    """A workspace for decode_tree (and the other calls on this cache but decode_paged,
    whose is paged_workspace): Hq query heads, T tokens a tree at most.  It serves one
    call at a time, and the device's errors are then reported to it."""
    Hq = Hq or cache.Hkv
    n = max(_tree_desc(cache.B, Hq, cache.Hkv, t, cache.d, 1.0, True)[1] for t in (1, T))
    return torch.zeros(n, dtype=torch.uint8, device=cache.device)


def decode_tree(cache: PagedCache, q, mask, q_lens=None, scale=None, out_fp32=False, ws=None,
                out=None, lse=None, stream=None):
    """Attention of a tree of drafted tokens over every sequence's cached rows
    (dfa_decode_tree): q [B,Hq,T,d] bf16 (any strides with contiguous features), q_lens
    [B] int32 of the T tokens per sequence (default: all), their keys and values in the
    sequence's last rows.  mask [B,T,ceil(T/32)] int32: which of those each of them sees
    (tree_plan); all see the rows before.  Returns (O [B,Hq,T,d], LSE [B,Hq,T]); rows from
    q_lens on are not written."""
    dev = cache.device
    raw = _raw_stream(dev, stream)
    shape = q.shape
    if len(shape) != 4:
        raise ValueError("q must be [B,Hq,T,d]")
    B, Hq, T, d = shape
    qp, qs = _rows(q, "q", torch.bfloat16, dev, (cache.B, Hq, T, cache.d))
    if mask is None:
        raise ValueError("decode_tree needs a mask (decode_paged takes chains without one)")
    o_dtype = torch.float32 if out_fp32 else torch.bfloat16
    if out is None:
        out = _new(stream, shape, o_dtype, dev)
    if lse is None:
        lse = _new(stream, (B, Hq, T), torch.float32, dev)
    desc, need = _tree_desc(B, Hq, cache.Hkv, T, d,
                            1.0 / math.sqrt(d) if scale is None else scale, bool(out_fp32))
    ws, ref = _ws(ws, need, cache, stream)
    code = lib().dfa_decode_tree(desc, ref, T, _int32(q_lens, "q_lens", (B,), dev),
                                 _int32(mask, "mask", (B, T, _words(T)), dev), qp, qs,
                                 _plain(out, "out", o_dtype, dev, shape),
                                 _plain(lse, "lse", torch.float32, dev, (B, Hq, T)),
                                 ws.data_ptr(), ws.numel(), raw)
    if code:
        _check(code)
    return out, lse


def cache_compact(cache: PagedCache, kept, kept_lens=None, q_lens=None, T=None, ws=None,
                  stream=None):
    """Of the last q_lens [B] int32 (default: T) rows of every sequence, those whose
    numbers stand in kept [B,A] int32 (the first kept_lens [B] of each row, default: all;
    strictly increasing) move together, in place (dfa_cache_compact): row kept[i] of them
    becomes row i.  T: the most rows that q_lens names (default: what a sequence can have).
    seq_lens is the caller's to lower, after the last layer."""
    dev = cache.device
    raw = _raw_stream(dev, stream)
    if kept.dim() != 2:
        raise ValueError("kept must be [B, A]")
    if T is None:
        if q_lens is None:
            raise ValueError("give T or q_lens")
        T = max(cache.block_table.shape[1] * cache.page, kept.shape[1])
    ws, ref = _ws(ws, 256, cache, stream)
    code = lib().dfa_cache_compact(ref, T, _int32(q_lens, "q_lens", (cache.B,), dev),
                                   kept.shape[1],
                                   _int32(kept, "kept", (cache.B, kept.shape[1]), dev),
                                   _int32(kept_lens, "kept_lens", (cache.B,), dev),
                                   ws.data_ptr(), ws.numel(), raw)
    if code:
        _check(code)


def cache_copy(cache: PagedCache, jobs, info, ws=None, stream=None):
    """Copy pages of a cache, K, V and scales: the first info[0] (on the device) pairs
    (from, to) of jobs [J,2] int32 (dfa_cache_copy; pages_reserve makes both)."""
    dev = cache.device
    raw = _raw_stream(dev, stream)
    if jobs.dim() != 2:
        raise ValueError("jobs must be [J, 2]")
    J = jobs.shape[0]
    ws, ref = _ws(ws, 256, cache, stream)
    jobs = _int32(jobs, "jobs", (J, 2), dev)
    info = _int32(info, "info", (4,), dev)
    if J == 0:
        return
    code = lib().dfa_cache_copy(ref, jobs, J, info, ws.data_ptr(), ws.numel(), raw)
    if code:
        _check(code)


class PagePool:
    """The pages behind a cache, or behind the caches of all layers (dfa_page_pool), over
    the caller's tensors, which it keeps alive: block_table [B,max_pages] and seq_lens [B]
    int32, those of the caches; held [B] int32: the pages that each sequence holds, the
    first entries of its row; refs [npages] int32: how many hold each page, 0 where it is
    free.  Without held and refs a new pool of npages pages is made, which nobody holds yet.
    Its calls run one at a time, and report numbers that cannot be to the workspace they
    are given, or else to pool.status: stream_status(pool.status).  Graphs of its calls need
    it alive."""

    def __init__(self, block_table, seq_lens, page, held=None, refs=None, npages=None):
        dev = block_table.device
        if block_table.dim() != 2:
            raise ValueError("block_table must be [B, max_pages]")
        B, max_pages = block_table.shape
        if (held is None) != (refs is None) or (refs is None) == (npages is None):
            raise ValueError("give held and refs, or npages")
        made = ()
        if refs is None:
            held = torch.zeros(B, dtype=torch.int32, device=dev)
            refs = torch.zeros(npages, dtype=torch.int32, device=dev)
            made = held, refs
        if refs.dim() != 1:
            raise ValueError("refs must be [npages]")
        self.device, self.B, self.page, self.npages = dev, B, page, refs.shape[0]
        self.block_table, self.seq_lens, self.held, self.refs = block_table, seq_lens, held, refs
        self.desc = PagePoolDesc(page, B, max_pages, 0, self.npages,
                                 _int32(block_table, "block_table", (B, max_pages), dev),
                                 _int32(held, "held", (B,), dev),
                                 _int32(refs, "refs", (self.npages,), dev),
                                 _int32(seq_lens, "seq_lens", (B,), dev))
        self._ref = ctypes.byref(self.desc)
        # for calls without a workspace, whose own nobody could read
        self.status = torch.zeros(256, dtype=torch.uint8, device=dev)
        self._own = PagePoolDesc.from_buffer_copy(self.desc)
        self._own.status = self.status.data_ptr()
        self._own_ref = ctypes.byref(self._own)
        self._need = max(256, int(lib().dfa_pages_workspace_size(self._ref)))
        self._scratch = torch.empty(self._need, dtype=torch.uint8, device=dev)
        self._made = (*made, self.status, self._scratch)  # (else the caller's)
        self._raw = (torch.cuda.current_stream(dev).cuda_stream if dev.type == "cuda" else None)

    def __setattr__(self, name, value):
        if self.__dict__.get(name, value) is not value:
            raise AttributeError(f"{name} of a PagePool stays: change its contents, or make a "
                                 "new PagePool")
        super().__setattr__(name, value)

    def __delattr__(self, name):
        raise AttributeError(f"{name} of a PagePool stays: change its contents")


def _pool_ws(ws, nbytes, pool, stream, raw):
    """A call's workspace, and the pool as the call sees it: errors go to the caller's
    workspace, without one to the pool's status.  (The pool's calls run one at a time: what
    they need beside their arguments is the pool's.)"""
    if stream is not None or raw != pool._raw:
        at = stream or torch.cuda.current_stream(pool.device)
        for t in pool._made:  # the pool may go before the call has run
            t.record_stream(at)
    if ws is None:
        return pool._scratch, pool._own_ref
    return _ws(ws, nbytes, pool, stream)


def pages_workspace(pool: PagePool) -> torch.Tensor:
    """A workspace for the calls on this pool.  The device's errors are then reported to
    it."""
    return torch.zeros(pool._need, dtype=torch.uint8, device=pool.device)


def pages_fork(pool: PagePool, src, ws=None, stream=None):
    """Every sequence b becomes what sequence src[b] (src [B] int32) was: its pages, which
    both then hold, and its length; src[b] = b: stays, -1: becomes empty
    (dfa_pages_fork)."""
    raw = _raw_stream(pool.device, stream)
    ws, ref = _pool_ws(ws, pool._need, pool, stream, raw)
    if src is None:
        raise ValueError("src must be [B]")
    code = lib().dfa_pages_fork(ref, _int32(src, "src", (pool.B,), pool.device), ws.data_ptr(),
                                ws.numel(), raw)
    if code:
        _check(code)


def pages_reserve(pool: PagePool, T, new_lens=None, jobs=None, info=None, ws=None, stream=None):
    """Pages for the last new_lens [B] int32 (default: T, which is also the most of them)
    rows of every sequence, which seq_lens counts already: missing ones, and ones of their
    own in place of those that others hold too (dfa_pages_reserve).  Returns (jobs [J,2],
    info [4]) for cache_copy, to be called for every layer; info holds the number of jobs,
    the pages taken, and whether the call was refused for want of pages or of room in
    jobs, in which case it has changed nothing (the pages are then those that it would have
    taken).  Then no row may be stored or moved: the table may still name pages that other
    sequences hold.  Take seq_lens back by T * info[2] and give the calls of the step
    (1 - info[2]) times their lengths."""
    dev = pool.device
    raw = _raw_stream(dev, stream)
    if jobs is None:
        most = min(T // pool.page + 2, pool.block_table.shape[1])
        jobs = _new(stream, (pool.B * most, 2), torch.int32, dev)
    elif jobs.dim() != 2:
        raise ValueError("jobs must be [J, 2]")
    if info is None:
        info = _new(stream, (4,), torch.int32, dev)
    J = jobs.shape[0]
    ws, ref = _pool_ws(ws, pool._need, pool, stream, raw)
    code = lib().dfa_pages_reserve(ref, T, _int32(new_lens, "new_lens", (pool.B,), dev),
                                   _int32(jobs, "jobs", (J, 2), dev), J,
                                   _int32(info, "info", (4,), dev), ws.data_ptr(), ws.numel(),
                                   raw)
    if code:
        _check(code)
    return jobs, info


def pages_trim(pool: PagePool, ws=None, stream=None):
    """Every sequence gives back the pages that it holds behind its length
    (dfa_pages_trim)."""
    raw = _raw_stream(pool.device, stream)
    ws, ref = _pool_ws(ws, 256, pool, stream, raw)
    code = lib().dfa_pages_trim(ref, ws.data_ptr(), ws.numel(), raw)
    if code:
        _check(code)


# ----------------------------------------------------------------------------
# host-only helpers
# ----------------------------------------------------------------------------
def make_schedule(N, P, partition="contiguous", stripe=1, tile_m=128, tile_n=128, causal=True,
                  items=True):
    """Ring schedule (host only, dfa_make_schedule): returns a dict with
    pair_tokens [P][P] (worker, step), tile_counts [P][P][3], total_pairs,
    eta_slots, eta_flops, the pair list ``pairs`` [P*P] of (worker, step,
    kv_worker, tokens, first_item, n_items) and, with items=True, the tile
    work items [n_items] of (worker, step, q_tile, kv_begin, kv_end,
    mask_class) -- sized by a first call with capacity 0."""
    import numpy as np
    desc = make_desc(1, 1, 1, N, 64, causal=causal, P=P, partition=partition, stripe=stripe)
    pt = (ctypes.c_int64 * (P * P))()
    tc = (ctypes.c_int64 * (3 * P * P))()
    pr = (SchedPair * (P * P))()
    s = Schedule(ctypes.cast(pt, ctypes.POINTER(ctypes.c_int64)),
                 ctypes.cast(tc, ctypes.POINTER(ctypes.c_int64)), 0, 0.0, 0.0,
                 ctypes.cast(pr, ctypes.POINTER(SchedPair)), None, 0, 0)
    _check(lib().dfa_make_schedule(ctypes.byref(desc), tile_m, tile_n, ctypes.byref(s)))
    out = {"pair_tokens": np.array(pt[:], dtype=np.int64).reshape(P, P),
           "tile_counts": np.array(tc[:], dtype=np.int64).reshape(P, P, 3),
           "total_pairs": int(s.total_pairs), "eta_slots": float(s.eta_slots),
           "eta_flops": float(s.eta_flops), "n_items": int(s.n_items),
           "pairs": np.array([(x.worker, x.step, x.kv_worker, x.tokens, x.first_item, x.n_items)
                              for x in pr], dtype=np.int64)}
    if items:
        it = (SchedItem * max(1, s.n_items))()
        s.items = ctypes.cast(it, ctypes.POINTER(SchedItem))
        s.capacity = s.n_items
        _check(lib().dfa_make_schedule(ctypes.byref(desc), tile_m, tile_n, ctypes.byref(s)))
        out["items"] = np.array([(x.worker, x.step, x.q_tile, x.kv_begin, x.kv_end, x.mask_class)
                                 for x in it[:s.n_items]], dtype=np.int64).reshape(-1, 6)
    return out


def stream_status(ws, stream=None) -> int:
    """Synchronise, read and clear the device status word; raise on error."""
    code = lib().dfa_stream_status(_ptr(ws), _stream(stream))
    _check(code)
    return code


def selftest_timeout(ws, timeout_us=1000, stream=None):
    _check(lib().dfa_selftest_timeout(_ptr(ws), timeout_us, _stream(stream)))
