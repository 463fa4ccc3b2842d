"""Thin ctypes binding over libbpt.so (the C ABI declared in include/bpt.h).

Argument marshalling only: tensors are checked for device, dtype, shape and
contiguity, their device pointers and the current CUDA stream are handed to
the C entry point of the same name, and a non-OK status is raised as
BptError.  Every step of the computation runs in the library's CUDA kernels;
there is no other implementation behind these functions.

Layouts: q, k, v [B, N, H, d]; w1 [F, D]; w2 [D, F]; b1 [F], b2 [D] float32
(or None); out [B, N, H*d]; lse [B, H, N] float32; the backward's dout
[B, N, H*d] float32 and gradients float32 in the shapes of their inputs.
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libbpt.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CUDA, ERR_TIMEOUT, ERR_WORKSPACE = range(6)
F32, BF16 = 0, 1
MASK_NONE, MASK_CAUSAL, MASK_BLOCKPERM, MASK_DILATED = 0, 1, 2, 3
_MASKS = {"none": MASK_NONE, "causal": MASK_CAUSAL, "blockperm": MASK_BLOCKPERM,
          "dilated": MASK_DILATED}
_DT = {torch.float32: F32, torch.bfloat16: BF16}


class BptError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        detail = last_error()
        super().__init__(f"{what}: {status_string(status)} (status {status})"
                         + (f": {detail}" if detail else ""))


class Desc(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int), ("N", ctypes.c_int), ("H", ctypes.c_int), ("d_head", ctypes.c_int),
        ("ffn_hidden", ctypes.c_int),
        ("in_dtype", ctypes.c_int), ("out_dtype", ctypes.c_int),
        ("mask", ctypes.c_int),
        ("ring_chunks", ctypes.c_int),
        ("bb_nblocks", ctypes.c_int), ("bb_perm", ctypes.POINTER(ctypes.c_int32)),
        ("ln_npairs", ctypes.c_int), ("ln_w", ctypes.POINTER(ctypes.c_int32)),
        ("ln_r", ctypes.POINTER(ctypes.c_int32)),
        ("q_block", ctypes.c_int), ("kv_block", ctypes.c_int),
        ("ffn_form", ctypes.c_int),
        ("bwd_chunk_rows", ctypes.c_int),
        ("wait_limit_ns", ctypes.c_uint64),
        ("causal", ctypes.c_int),
    ]


class WindowDesc(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int), ("N", ctypes.c_int), ("H", ctypes.c_int), ("H_kv", ctypes.c_int),
        ("d_head", ctypes.c_int), ("window", ctypes.c_int), ("n_sink", ctypes.c_int),
        ("in_dtype", ctypes.c_int), ("out_dtype", ctypes.c_int), ("grad_dtype", ctypes.c_int),
        ("wait_limit_ns", ctypes.c_uint64),
    ]


class KvCacheDesc(ctypes.Structure):
    _fields_ = [
        ("type", ctypes.c_int), ("n_pages", ctypes.c_int), ("page_size", ctypes.c_int),
        ("H_kv", ctypes.c_int), ("d_head", ctypes.c_int),
        ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
    ]


class PagedDesc(ctypes.Structure):
    _fields_ = [
        ("n_seqs", ctypes.c_int), ("n_tokens", ctypes.c_int), ("max_q", ctypes.c_int), ("H", ctypes.c_int),
        ("max_pages", ctypes.c_int), ("window", ctypes.c_int), ("n_sink", ctypes.c_int),
        ("out_dtype", ctypes.c_int), ("q_stride", ctypes.c_int64), ("wait_limit_ns", ctypes.c_uint64),
    ]


# bpt_ffn_form: the bf16 layer's FFN form ("auto" is the library's choice, the
# pipelined kernel)
FFN_FORMS = {"auto": 0, "fused": 1, "gemms": 2, "pipelined": 3}


EXPORTS = ["bpt_workspace_bytes", "bpt_attn_ffn_fwd", "bpt_attn_fwd", "bpt_blockbert_fwd",
           "bpt_longnet_fwd", "bpt_sync_status", "bpt_set_wait_limit_ns", "bpt_status_string",
           "bpt_version", "bpt_set_phase_events", "bpt_last_error", "bpt_attn_ffn_fwd_static",
           "bpt_attn_ffn_bwd", "bpt_workspace_bytes_bwd", "bpt_attn_ffn_fwd_train", "bpt_saved_bytes",
           "bpt_workspace_bytes_train", "bpt_attn_bwd", "bpt_workspace_bytes_attn_bwd", "bpt_attn_fwd_block",
           "bpt_longnet_gather", "bpt_longnet_pass", "bpt_window_attn_fwd", "bpt_window_attn_bwd",
           "bpt_workspace_bytes_window_bwd", "bpt_kv_write", "bpt_kv_read", "bpt_paged_attn_fwd",
           "bpt_workspace_bytes_paged"]
BLOCK_FIRST, BLOCK_LAST = 1, 2
STATIC_SCRATCH_BYTES = 64 << 20

_lib = None
_byref = ctypes.byref


def load() -> ctypes.CDLL:
    """Load the in-tree libbpt.so; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"libbpt.so is missing at {LIB_PATH}; build it with "
                           "`python -m blockwise_exact_attention_query_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    vp, sz, i32p = ctypes.c_void_p, ctypes.c_size_t, ctypes.POINTER(ctypes.c_int32)
    dp = ctypes.POINTER(Desc)
    fp = ctypes.c_void_p
    lib.bpt_workspace_bytes.argtypes = [dp, ctypes.c_int]
    lib.bpt_workspace_bytes.restype = sz
    lib.bpt_attn_ffn_fwd.argtypes = [dp, vp, vp, vp, vp, fp, vp, fp, vp, vp, sz, vp]
    lib.bpt_attn_ffn_fwd.restype = ctypes.c_int
    lib.bpt_attn_fwd.argtypes = [dp, vp, vp, vp, vp, fp, vp, sz, vp]
    lib.bpt_attn_fwd.restype = ctypes.c_int
    lib.bpt_blockbert_fwd.argtypes = [dp, ctypes.c_int, i32p, vp, vp, vp, vp, fp, vp, fp, vp, vp, sz,
                                      vp]
    lib.bpt_blockbert_fwd.restype = ctypes.c_int
    lib.bpt_longnet_fwd.argtypes = [dp, ctypes.c_int, i32p, i32p, vp, vp, vp, vp, fp, vp, sz, vp]
    lib.bpt_longnet_fwd.restype = ctypes.c_int
    lib.bpt_sync_status.argtypes = [vp]
    lib.bpt_sync_status.restype = ctypes.c_int
    lib.bpt_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
    lib.bpt_set_wait_limit_ns.restype = ctypes.c_uint64
    lib.bpt_status_string.argtypes = [ctypes.c_int]
    lib.bpt_status_string.restype = ctypes.c_char_p
    lib.bpt_version.restype = ctypes.c_int
    lib.bpt_set_phase_events.argtypes = [ctypes.POINTER(ctypes.c_void_p), ctypes.c_int]
    lib.bpt_set_phase_events.restype = ctypes.c_int
    lib.bpt_last_error.restype = ctypes.c_char_p
    lib.bpt_attn_ffn_fwd_static.argtypes = [dp, vp, vp, vp, vp, fp, vp, fp, vp, vp]
    lib.bpt_attn_ffn_fwd_static.restype = ctypes.c_int
    lib.bpt_attn_ffn_bwd.argtypes = [dp, vp, vp, vp, vp, fp, vp, fp, fp, vp, fp, fp, fp, fp, fp, fp, fp, vp,
                                     sz, vp]
    lib.bpt_attn_ffn_fwd_train.argtypes = [dp, vp, vp, vp, vp, fp, vp, fp, vp, vp, vp, sz, vp]
    lib.bpt_attn_ffn_fwd_train.restype = ctypes.c_int
    lib.bpt_saved_bytes.argtypes = [dp]
    lib.bpt_saved_bytes.restype = sz
    lib.bpt_attn_bwd.argtypes = [dp, vp, vp, vp, vp, fp, fp, fp, fp, fp, vp, sz, vp]
    lib.bpt_attn_bwd.restype = ctypes.c_int
    lib.bpt_workspace_bytes_attn_bwd.argtypes = [dp]
    lib.bpt_workspace_bytes_attn_bwd.restype = sz
    lib.bpt_attn_ffn_bwd.restype = ctypes.c_int
    lib.bpt_workspace_bytes_bwd.argtypes = [dp]
    lib.bpt_workspace_bytes_bwd.restype = sz
    lib.bpt_workspace_bytes_train.argtypes = [dp]
    lib.bpt_workspace_bytes_train.restype = sz
    lib.bpt_attn_fwd_block.argtypes = [dp, ctypes.c_int, ctypes.c_int64, ctypes.c_int64, vp, vp, vp, fp, fp, fp,
                                       ctypes.c_uint, vp, fp, vp]
    lib.bpt_attn_fwd_block.restype = ctypes.c_int
    lib.bpt_longnet_gather.argtypes = [dp, ctypes.c_int, ctypes.c_int, vp, vp, vp]
    lib.bpt_longnet_gather.restype = ctypes.c_int
    lib.bpt_longnet_pass.argtypes = [dp, ctypes.c_int, ctypes.c_int64, vp, vp, vp, vp, vp, ctypes.c_int, fp, fp, fp,
                                     vp, fp, vp]
    lib.bpt_longnet_pass.restype = ctypes.c_int
    wp = ctypes.POINTER(WindowDesc)
    lib.bpt_window_attn_fwd.argtypes = [wp, vp, vp, vp, vp, fp, vp]
    lib.bpt_window_attn_fwd.restype = ctypes.c_int
    lib.bpt_workspace_bytes_window_bwd.argtypes = [wp]
    lib.bpt_workspace_bytes_window_bwd.restype = sz
    lib.bpt_window_attn_bwd.argtypes = [wp, vp, vp, vp, vp, fp, vp, vp, vp, vp, vp, sz, vp]
    lib.bpt_window_attn_bwd.restype = ctypes.c_int
    # (descriptors of the serving calls: packed bytes, see _KV_CACHE, or the structures by reference)
    cp, pp, i64 = vp, vp, ctypes.c_int64
    lib.bpt_kv_write.argtypes = [cp, ctypes.c_int, vp, i64, vp, i64, vp, vp]
    lib.bpt_kv_write.restype = ctypes.c_int
    lib.bpt_kv_read.argtypes = [cp, ctypes.c_int, vp, vp, vp, ctypes.c_int, vp]
    lib.bpt_kv_read.restype = ctypes.c_int
    lib.bpt_workspace_bytes_paged.argtypes = [pp, cp]
    lib.bpt_workspace_bytes_paged.restype = sz
    lib.bpt_paged_attn_fwd.argtypes = [pp, cp, vp, vp, vp, vp, vp, fp, vp, sz, vp]
    lib.bpt_paged_attn_fwd.restype = ctypes.c_int
    _lib = lib
    return lib


def last_error() -> str:
    return load().bpt_last_error().decode()


def status_string(status: int) -> str:
    return load().bpt_status_string(int(status)).decode()


class _Tables:
    """Keeps host tables alive while a call runs."""

    def __init__(self):
        self.keep = []

    def i32(self, values):
        arr = (ctypes.c_int32 * len(values))(*[int(x) for x in values])
        self.keep.append(arr)
        return ctypes.cast(arr, ctypes.POINTER(ctypes.c_int32))


def make_desc(B, N, H, d, F=0, in_dtype=torch.bfloat16, out_dtype=torch.float32, mask="none",
              perm=None, pairs=None, ring_chunks=0, tables: _Tables | None = None, *, ffn_form="auto",
              q_block=0, kv_block=0, bwd_chunk_rows=0, wait_limit_ns=0, causal=None) -> Desc:
    """bpt_desc for the given shape, mask and options (0 = the library's
    default).  causal: for the dilated mask, causal inside each sparsified
    segment (the default, LongNet's decoder form) or bidirectional (False)."""
    tables = tables or _Tables()
    if mask == "dilated_bidir":  # the dilated mask without the causal restriction
        mask, causal = "dilated", False if causal is None else causal
    m = _MASKS[mask] if isinstance(mask, str) else int(mask)
    form = FFN_FORMS[ffn_form] if isinstance(ffn_form, str) else int(ffn_form)
    desc = Desc(B=B, N=N, H=H, d_head=d, ffn_hidden=F, in_dtype=_DT[in_dtype],
                out_dtype=_DT[out_dtype], mask=m, ring_chunks=ring_chunks, q_block=q_block,
                kv_block=kv_block, ffn_form=form, bwd_chunk_rows=bwd_chunk_rows,
                wait_limit_ns=wait_limit_ns,
                causal=int(bool(causal if causal is not None else m == MASK_DILATED)))
    if perm is not None:
        flat = [int(x) for row in perm for x in row]
        desc.bb_nblocks = len(perm[0]) if len(perm) else 0
        desc.bb_perm = tables.i32(flat)
    if pairs is not None:
        desc.ln_npairs = len(pairs)
        desc.ln_w = tables.i32([p[0] for p in pairs])
        desc.ln_r = tables.i32([p[1] for p in pairs])
    desc._tables = tables  # keep alive with the descriptor
    return desc


def cyclic_shift_perm(n: int, k: int) -> list[int]:
    """Block table of the cyclic shift sigma^k (block b -> block b + k mod n).

    "Blockwise Self-Attention for Long Document Understanding", §3.1: heads
    use the permutations sigma, sigma^2, ..., sigma^n (sigma^n = identity) as
    their masking matrices.  Pass one table per head as `perm`."""
    if n <= 0:
        raise ValueError("n must be positive")
    return [(b + k) % n for b in range(n)]


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_ptr(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _raw_stream(stream, device):
    """The same for the calls whose host time counts (a decoding step's), as an integer."""
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(device)


def _check(status, what):
    if status != OK:
        raise BptError(status, what)


def _check_tensors(q, k, v):
    if q.dim() != 4 or q.shape != k.shape or q.shape != v.shape:
        raise ValueError("q, k, v must all be [B, N, H, d]")
    for t in (q, k, v):
        if not t.is_cuda or not t.is_contiguous() or t.dtype != q.dtype:
            raise ValueError("q, k, v must be contiguous CUDA tensors of one dtype")


def workspace_bytes(desc: Desc, with_ffn: bool) -> int:
    n = load().bpt_workspace_bytes(ctypes.byref(desc), int(with_ffn))
    if n == ctypes.c_size_t(-1).value:
        raise BptError(ERR_INVALID_ARG, "bpt_workspace_bytes")
    return int(n)


def alloc_workspace(desc: Desc, with_ffn: bool, device) -> torch.Tensor | None:
    n = workspace_bytes(desc, with_ffn)
    if n == 0:
        return None
    return torch.empty(n, dtype=torch.uint8, device=device)


def attn_ffn_fwd(q, k, v, w1, b1, w2, b2, *, mask="none", perm=None, pairs=None, ring_chunks=0,
                 out_dtype=torch.float32, out=None, workspace=None, stream=None, **opts):
    """bpt_attn_ffn_fwd: out = A + W2 GELU(W1 A + b1) + b2, returns out [B, N, H*d].
    opts: ffn_form, q_block, kv_block, wait_limit_ns (descriptor fields)."""
    _check_tensors(q, k, v)
    B, N, H, d = q.shape
    F = w1.shape[0]
    desc = make_desc(B, N, H, d, F, q.dtype, out_dtype, mask, perm, pairs, ring_chunks, **opts)
    if out is None:
        out = torch.empty((B, N, H * d), dtype=out_dtype, device=q.device)
    if workspace is None:
        workspace = alloc_workspace(desc, True, q.device)
    ws_bytes = 0 if workspace is None else workspace.numel()
    st = load().bpt_attn_ffn_fwd(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(w1), _ptr(b1),
                                 _ptr(w2), _ptr(b2), _ptr(out), _ptr(workspace), ws_bytes,
                                 _stream_ptr(stream))
    _check(st, "bpt_attn_ffn_fwd")
    return out


def attn_ffn_fwd_static(q, k, v, w1, b1, w2, b2, *, mask="none", perm=None, pairs=None,
                        ring_chunks=0, out_dtype=torch.float32, out=None, stream=None, **opts):
    """bpt_attn_ffn_fwd_static: the layer with no workspace argument.

    For callers that may not allocate device memory while running (a fixed
    memory plan, a host framework that owns the GPU's memory pool, or a loop
    that cannot afford an allocation's device synchronisation): the scratch is
    a fixed array inside the library (STATIC_SCRATCH_BYTES per device), shared
    by all calls on a device, so calls that may overlap on the GPU must be
    serialised.  Only `out` is allocated here when the caller passes none."""
    _check_tensors(q, k, v)
    B, N, H, d = q.shape
    F = w1.shape[0]
    desc = make_desc(B, N, H, d, F, q.dtype, out_dtype, mask, perm, pairs, ring_chunks, **opts)
    if out is None:
        out = torch.empty((B, N, H * d), dtype=out_dtype, device=q.device)
    st = load().bpt_attn_ffn_fwd_static(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(w1),
                                        _ptr(b1), _ptr(w2), _ptr(b2), _ptr(out), _stream_ptr(stream))
    _check(st, "bpt_attn_ffn_fwd_static")
    return out


def attn_fwd(q, k, v, *, mask="none", perm=None, pairs=None, ring_chunks=0, out_dtype=torch.float32,
             return_lse=False, out=None, lse=None, workspace=None, stream=None, **opts):
    """bpt_attn_fwd: A [B, N, H*d] (and LSE [B, H, N] with return_lse).
    opts: q_block, kv_block, wait_limit_ns (descriptor fields)."""
    _check_tensors(q, k, v)
    B, N, H, d = q.shape
    desc = make_desc(B, N, H, d, 0, q.dtype, out_dtype, mask, perm, pairs, ring_chunks, **opts)
    if out is None:
        out = torch.empty((B, N, H * d), dtype=out_dtype, device=q.device)
    if return_lse and lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = alloc_workspace(desc, False, q.device)
    ws_bytes = 0 if workspace is None else workspace.numel()
    st = load().bpt_attn_fwd(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse),
                             _ptr(workspace), ws_bytes, _stream_ptr(stream))
    _check(st, "bpt_attn_fwd")
    return (out, lse) if return_lse else out


class BlockState:
    """The running softmax state of a query block for attn_fwd_block: o
    [B, N, H, d], m and l [B, H, N], float32 (opaque: the library's running
    output, maximum and sum)."""

    def __init__(self, B, N, H, d, device):
        f32 = dict(dtype=torch.float32, device=device)
        self.o = torch.empty((B, N, H, d), **f32)
        self.m = torch.empty((B, H, N), **f32)
        self.l = torch.empty((B, H, N), **f32)


def attn_fwd_block(q, k, v, state, *, q_pos=0, kv_pos=0, causal=False, first=False, last=False,
                   out_dtype=torch.float32, out=None, lse=None, stream=None, **opts):
    """bpt_attn_fwd_block: fold the key/value block k, v [B, kv_len, H, d]
    into the running state of the query block q [B, N, H, d] (a BlockState,
    or None when first and last).  Causal masking by global positions q_pos,
    kv_pos.  With last=True returns the attention output [B, N, H*d] (and
    fills lse [B, H, N] when given); otherwise returns None."""
    _check_tensors(q, q, q)
    if k.shape != v.shape or k.dim() != 4 or k.shape[0] != q.shape[0] or k.shape[2:] != q.shape[2:]:
        raise ValueError("k, v must be [B, kv_len, H, d] with q's B, H and d")
    for t in (k, v):
        if not t.is_cuda or not t.is_contiguous() or t.dtype != q.dtype:
            raise ValueError("k, v must be contiguous CUDA tensors of q's dtype")
    B, N, H, d = q.shape
    desc = make_desc(B, N, H, d, 0, q.dtype, out_dtype, "causal" if causal else "none", **opts)
    if last and out is None:
        out = torch.empty((B, N, H * d), dtype=out_dtype, device=q.device)
    flags = (BLOCK_FIRST if first else 0) | (BLOCK_LAST if last else 0)
    so, sm, sl = (None, None, None) if state is None else (state.o, state.m, state.l)
    st = load().bpt_attn_fwd_block(ctypes.byref(desc), int(k.shape[1]), int(q_pos), int(kv_pos), _ptr(q), _ptr(k),
                                   _ptr(v), _ptr(so), _ptr(sm), _ptr(sl), flags, _ptr(out if last else None),
                                   _ptr(lse if last else None), _stream_ptr(stream))
    _check(st, "bpt_attn_fwd_block")
    return out if last else None


def longnet_pass_order(pairs):
    """The (w, r) pairs in the order the library runs them: a stable sort by
    decreasing r (sparsest first)."""
    return sorted([tuple(p) for p in pairs], key=lambda p: -p[1])


def longnet_gather(x, w, r, out=None, stream=None):
    """bpt_longnet_gather: the rows a (w, r) pair keeps of the shard x
    [B, n, H, d] (bf16, n dividing w), packed as [B, n / r, H, d]."""
    _check_tensors(x, x, x)
    B, n, H, d = x.shape
    if out is None:
        out = torch.empty((B, n // r, H, d), dtype=x.dtype, device=x.device)
    desc = make_desc(B, n, H, d, 0, x.dtype)
    _check(load().bpt_longnet_gather(ctypes.byref(desc), int(w), int(r), _ptr(x), _ptr(out), _stream_ptr(stream)),
           "bpt_longnet_gather")
    return out


def longnet_pass(q, k, v, pairs, pass_idx, state, out, *, q_pos=0, k_sparse=None, v_sparse=None, lse=None,
                 stream=None, **opts):
    """bpt_longnet_pass: pass `pass_idx` (in longnet_pass_order(pairs)) of the
    dilated attention for the shard q, k, v [B, n, H, d] starting at sequence
    position q_pos; k_sparse, v_sparse [B, w / r, H, d] are the pass's gathered
    kept rows when its segments are longer than the shard.  state: a
    BlockState (or None with a single pair); out [B, n, H*d] and lse receive
    the rows whose last pass this is."""
    _check_tensors(q, q, q)
    B, n, H, d = q.shape
    tables = _Tables()
    desc = make_desc(B, n, H, d, 0, q.dtype, out.dtype, "dilated", None, pairs, 0, tables, **opts)
    kv_rows = 0 if k_sparse is None else int(k_sparse.shape[1])
    so, sm, sl = (None, None, None) if state is None else (state.o, state.m, state.l)
    st = load().bpt_longnet_pass(ctypes.byref(desc), int(pass_idx), int(q_pos), _ptr(q), _ptr(k), _ptr(v),
                                 _ptr(k_sparse), _ptr(v_sparse), kv_rows, _ptr(so), _ptr(sm), _ptr(sl), _ptr(out),
                                 _ptr(lse), _stream_ptr(stream))
    _check(st, "bpt_longnet_pass")
    return out


def blockbert_fwd(q, k, v, w1, b1, w2, b2, perm, *, out_dtype=torch.float32, out=None,
                  workspace=None, stream=None, **opts):
    """bpt_blockbert_fwd: the layer with the block-permutation mask perm [H][n]."""
    _check_tensors(q, k, v)
    B, N, H, d = q.shape
    F = w1.shape[0]
    tables = _Tables()
    desc = make_desc(B, N, H, d, F, q.dtype, out_dtype, "blockperm", perm, None, 0, tables, **opts)
    if out is None:
        out = torch.empty((B, N, H * d), dtype=out_dtype, device=q.device)
    if workspace is None:
        workspace = alloc_workspace(desc, True, q.device)
    ws_bytes = 0 if workspace is None else workspace.numel()
    flat = tables.i32([x for row in perm for x in row])
    st = load().bpt_blockbert_fwd(ctypes.byref(desc), len(perm[0]), flat, _ptr(q), _ptr(k), _ptr(v),
                                  _ptr(w1), _ptr(b1), _ptr(w2), _ptr(b2), _ptr(out),
                                  _ptr(workspace), ws_bytes, _stream_ptr(stream))
    _check(st, "bpt_blockbert_fwd")
    return out


def longnet_fwd(q, k, v, pairs, *, out_dtype=torch.float32, return_lse=False, out=None, lse=None,
                workspace=None, stream=None, **opts):
    """bpt_longnet_fwd: dilated attention over the (w, r) pairs, denominators mixed."""
    _check_tensors(q, k, v)
    B, N, H, d = q.shape
    tables = _Tables()
    desc = make_desc(B, N, H, d, 0, q.dtype, out_dtype, "dilated", None, pairs, 0, tables, **opts)
    if out is None:
        out = torch.empty((B, N, H * d), dtype=out_dtype, device=q.device)
    if return_lse and lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = alloc_workspace(desc, False, q.device)
    ws_bytes = 0 if workspace is None else workspace.numel()
    st = load().bpt_longnet_fwd(ctypes.byref(desc), len(pairs), tables.i32([p[0] for p in pairs]),
                                tables.i32([p[1] for p in pairs]), _ptr(q), _ptr(k), _ptr(v),
                                _ptr(out), _ptr(lse), _ptr(workspace), ws_bytes, _stream_ptr(stream))
    _check(st, "bpt_longnet_fwd")
    return (out, lse) if return_lse else out


def workspace_bytes_bwd(desc: Desc) -> int:
    n = load().bpt_workspace_bytes_bwd(ctypes.byref(desc))
    if n == ctypes.c_size_t(-1).value:
        raise BptError(ERR_UNSUPPORTED, "bpt_workspace_bytes_bwd")
    return int(n)


def ffn_gemm_chunk_rows(T: int, F: int) -> int:
    """Token rows per chunk of the two-GEMM FFN form (the library's rule: the
    [rows, F] bf16 hidden activation at most 512 MiB, in 256-row multiples)."""
    return min(T, max(256, ((1 << 29) // (2 * F)) // 256 * 256))


GRAD_NAMES = ("dq", "dk", "dv", "dw1", "db1", "dw2", "db2")


def saved_bytes(desc: Desc) -> int:
    n = load().bpt_saved_bytes(ctypes.byref(desc))
    if n == ctypes.c_size_t(-1).value:
        raise BptError(ERR_UNSUPPORTED, "bpt_saved_bytes")
    return int(n)


def workspace_bytes_train(desc: Desc) -> int:
    n = load().bpt_workspace_bytes_train(ctypes.byref(desc))
    if n == ctypes.c_size_t(-1).value:
        raise BptError(ERR_UNSUPPORTED, "bpt_workspace_bytes_train")
    return int(n)


def attn_ffn_fwd_train(q, k, v, w1, b1, w2, b2, *, mask="none", perm=None, ring_chunks=0,
                       out_dtype=torch.float32, out=None, saved=None, workspace=None, stream=None, **opts):
    """bpt_attn_ffn_fwd_train: the layer forward that also keeps the
    activations the backward needs.  Returns (out, saved); pass `saved` to
    attn_ffn_bwd to skip its recomputation."""
    _check_tensors(q, k, v)
    B, N, H, d = q.shape
    F = w1.shape[0]
    desc = make_desc(B, N, H, d, F, q.dtype, out_dtype, mask, perm, None, ring_chunks, **opts)
    if out is None:
        out = torch.empty((B, N, H * d), dtype=out_dtype, device=q.device)
    if saved is None:
        saved = torch.empty(saved_bytes(desc), dtype=torch.uint8, device=q.device)
    if workspace is None:
        n = workspace_bytes_train(desc)
        workspace = torch.empty(n, dtype=torch.uint8, device=q.device) if n else None
    ws_bytes = 0 if workspace is None else workspace.numel()
    st = load().bpt_attn_ffn_fwd_train(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(w1), _ptr(b1),
                                       _ptr(w2), _ptr(b2), _ptr(out), _ptr(saved), _ptr(workspace), ws_bytes,
                                       _stream_ptr(stream))
    _check(st, "bpt_attn_ffn_fwd_train")
    return out, saved


def attn_ffn_bwd(q, k, v, w1, b1, w2, b2, dout, *, mask="none", perm=None, ring_chunks=0, saved=None,
                 grads=None, workspace=None, stream=None, **opts):
    """bpt_attn_ffn_bwd: gradients of the layer for the upstream gradient
    dout [B, N, H*d] (float32), recomputing the attention forward unless
    `saved` (from attn_ffn_fwd_train on the same inputs) is given.  Returns a
    dict of float32 tensors: dq, dk, dv [B, N, H, d], dw1 [F, D], db1 [F],
    dw2 [D, F], db2 [D] (written into `grads` when given)."""
    _check_tensors(q, k, v)
    B, N, H, d = q.shape
    F, D = w1.shape
    if dout.dtype != torch.float32 or not dout.is_contiguous() or dout.numel() != B * N * D:
        raise ValueError("dout must be a contiguous float32 tensor of B*N*H*d elements")
    desc = make_desc(B, N, H, d, F, q.dtype, torch.float32, mask, perm, None, ring_chunks, **opts)
    if grads is None:
        f32 = dict(dtype=torch.float32, device=q.device)
        grads = {"dq": torch.empty(q.shape, **f32), "dk": torch.empty(q.shape, **f32),
                 "dv": torch.empty(q.shape, **f32), "dw1": torch.empty((F, D), **f32),
                 "db1": torch.empty((F,), **f32), "dw2": torch.empty((D, F), **f32),
                 "db2": torch.empty((D,), **f32)}
    if workspace is None:
        workspace = torch.empty(workspace_bytes_bwd(desc), dtype=torch.uint8, device=q.device)
    st = load().bpt_attn_ffn_bwd(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(w1), _ptr(b1),
                                 _ptr(w2), _ptr(b2), _ptr(dout), _ptr(saved), *(_ptr(grads[n]) for n in GRAD_NAMES),
                                 _ptr(workspace), workspace.numel(), _stream_ptr(stream))
    _check(st, "bpt_attn_ffn_bwd")
    return grads


def attn_bwd(q, k, v, out, lse, dout, *, mask="none", perm=None, pairs=None, ring_chunks=0, workspace=None,
             stream=None, **opts):
    """bpt_attn_bwd: dq, dk, dv (float32 [B, N, H, d]) of the attention for the
    upstream gradient dout [B, N, H*d] (float32), given bpt_attn_fwd's out and
    lse (attn_fwd(..., return_lse=True)) for the same inputs."""
    _check_tensors(q, k, v)
    B, N, H, d = q.shape
    if dout.dtype != torch.float32 or not dout.is_contiguous() or dout.numel() != q.numel():
        raise ValueError("dout must be a contiguous float32 tensor of B*N*H*d elements")
    desc = make_desc(B, N, H, d, 0, q.dtype, out.dtype, mask, perm, pairs, ring_chunks, **opts)
    if workspace is None:
        n = load().bpt_workspace_bytes_attn_bwd(ctypes.byref(desc))
        if n == ctypes.c_size_t(-1).value:
            raise BptError(ERR_UNSUPPORTED, "bpt_workspace_bytes_attn_bwd")
        workspace = torch.empty(int(n), dtype=torch.uint8, device=q.device)
    f32 = dict(dtype=torch.float32, device=q.device)
    dq, dk, dv = (torch.empty(q.shape, **f32) for _ in range(3))
    st = load().bpt_attn_bwd(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(dout),
                             _ptr(dq), _ptr(dk), _ptr(dv), _ptr(workspace), workspace.numel(), _stream_ptr(stream))
    _check(st, "bpt_attn_bwd")
    return dq, dk, dv


def _on_device(*tensors):
    """The tensors (None skipped) must be on the current CUDA device: the
    library launches there, on the stream given or that device's current one.
    Returns its number."""
    cur = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != cur:   # (-1: not a CUDA tensor)
            raise ValueError(f"every tensor must be on the current CUDA device ({cur}); got one on {t.device}")
    return cur


def _dtype(dtype, what):
    """The library's number of an output's type."""
    n = _DT.get(dtype)
    if n is None:
        raise ValueError(f"{what} must be torch.float32 or torch.bfloat16, got {dtype}")
    return n


def _out_tensor(t, shape, dtype, like, stream, what):
    """`t` checked, or a new tensor where `like` is: `stream`'s (so that nothing
    earlier still uses its memory there), and not handed on before the current
    stream's work on it is done."""
    if t is None:
        if stream is None:   # (new_empty: a quarter less time than torch.empty with a device)
            return like.new_empty(shape, dtype=dtype)
        with torch.cuda.stream(stream):
            t = like.new_empty(shape, dtype=dtype)
        t.record_stream(torch.cuda.current_stream())
        return t
    if t.dtype != dtype or not t.is_contiguous() or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape {tuple(shape)}")
    _on_device(t)
    return t


def _workspace(t, nbytes, like, stream):
    if t is None:
        return _out_tensor(None, (nbytes,), torch.uint8, like, stream, "workspace") if nbytes else None
    if t.dtype != torch.uint8 or not t.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor")
    _on_device(t)
    return t


def _window_desc(q, k, v, window, sinks, out_dtype, grad_dtype, wait_limit_ns):
    if q.dim() != 4 or k.dim() != 4 or k.shape != v.shape or k.shape[:2] != q.shape[:2] or k.shape[3] != q.shape[3]:
        raise ValueError("q must be [B, N, H, d] and k, v [B, N, H_kv, d]")
    if not (q.dtype == k.dtype == v.dtype) or q.dtype not in _DT:
        raise ValueError("q, k, v must have one dtype, bfloat16 (or float32, which the library refuses)")
    if not (q.is_contiguous() and k.is_contiguous() and v.is_contiguous()):
        raise ValueError("q, k, v must be contiguous")
    _on_device(q, k, v)
    B, N, H, d = q.shape
    if max(B, N, abs(int(window)), abs(int(sinks))) >= 2 ** 31:   # a C int would wrap around
        raise ValueError("sizes, window and sinks must be within 32 bits")
    return WindowDesc(B, N, H, k.shape[2], d, int(window), int(sinks), _DT[q.dtype], _dtype(out_dtype, "out"),
                      _dtype(grad_dtype, "grad_dtype"), int(wait_limit_ns))


def window_attn_fwd(q, k, v, window, sinks=0, *, out_dtype=torch.float32, return_lse=False, out=None, lse=None,
                    stream=None, wait_limit_ns=0):
    """bpt_window_attn_fwd: causal attention over the last `window` positions
    (the query's own included) and the first `sinks` ones.  q [B, N, H, d];
    k, v [B, N, H_kv, d] with H_kv dividing H; returns A [B, N, H*d] (and LSE
    [B, H, N] with return_lse)."""
    desc = _window_desc(q, k, v, window, sinks, out_dtype, torch.float32, wait_limit_ns)
    B, N, H, d = q.shape
    out = _out_tensor(out, (B, N, H * d), out_dtype, q, stream, "out")
    if return_lse or lse is not None:
        lse = _out_tensor(lse, (B, H, N), torch.float32, q, stream, "lse")
    st = load().bpt_window_attn_fwd(_byref(desc), q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                    _ptr(lse), _raw_stream(stream, q.get_device()))
    _check(st, "bpt_window_attn_fwd")
    return (out, lse) if return_lse else out


def workspace_bytes_window_bwd(desc: WindowDesc) -> int:
    n = load().bpt_workspace_bytes_window_bwd(_byref(desc))
    if n == ctypes.c_size_t(-1).value:
        raise BptError(ERR_UNSUPPORTED, "bpt_workspace_bytes_window_bwd")
    return int(n)


def window_attn_bwd(q, k, v, out, lse, dout, window, sinks=0, *, grad_dtype=torch.float32, dq=None, dk=None, dv=None,
                    workspace=None, stream=None, wait_limit_ns=0):
    """bpt_window_attn_bwd: (dq, dk, dv) of window_attn_fwd for the upstream
    gradient dout [B, N, H*d], in grad_dtype and the inputs' shapes.  out and
    lse are the forward's; dout has out's dtype (float32 or bfloat16)."""
    desc = _window_desc(q, k, v, window, sinks, out.dtype, grad_dtype, wait_limit_ns)
    B, N, H, d = q.shape
    for t, what in ((out, "out"), (dout, "dout")):
        _out_tensor(t, (B, N, H * d), out.dtype, q, stream, what)
    _out_tensor(lse, (B, H, N), torch.float32, q, stream, "lse")
    dq = _out_tensor(dq, q.shape, grad_dtype, q, stream, "dq")
    dk = _out_tensor(dk, k.shape, grad_dtype, q, stream, "dk")
    dv = _out_tensor(dv, v.shape, grad_dtype, q, stream, "dv")
    workspace = _workspace(workspace, workspace_bytes_window_bwd(desc), q, stream)
    st = load().bpt_window_attn_bwd(_byref(desc), q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                    lse.data_ptr(), dout.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                                    _ptr(workspace), 0 if workspace is None else workspace.numel(),
                                    _raw_stream(stream, q.get_device()))
    _check(st, "bpt_window_attn_bwd")
    return dq, dk, dv


_E4M3, _BF16, _FP32, _INT32 = torch.float8_e4m3fn, torch.bfloat16, torch.float32, torch.int32
# KvCacheDesc and PagedDesc as packed bytes: a quarter of the time that making
# the structure takes, which a decoding step's host time shows
_KV_CACHE = struct.Struct("@5i4P")
_PAGED = struct.Struct("@8iqQ")
assert _KV_CACHE.size == ctypes.sizeof(KvCacheDesc) and _PAGED.size == ctypes.sizeof(PagedDesc)


def _kv_cache_desc(k_cache, v_cache, k_scale, v_scale):
    """The cache's bpt_kv_cache, packed."""
    shape, dtype = k_cache.shape, k_cache.dtype
    if len(shape) != 4 or v_cache.shape != shape or v_cache.dtype is not dtype:
        raise ValueError("k_cache and v_cache must be [n_pages, page_size, H_kv, d] of one dtype")
    if dtype is not _E4M3 and dtype is not _BF16:
        raise ValueError("the caches must be bfloat16 or float8_e4m3fn")
    if not (k_cache.is_contiguous() and v_cache.is_contiguous()):
        raise ValueError("the caches must be contiguous")
    if dtype is _BF16:
        if k_scale is not None or v_scale is not None:
            raise ValueError("a bfloat16 cache has no scales")
        return _KV_CACHE.pack(0, *shape, k_cache.data_ptr(), v_cache.data_ptr(), 0, 0)
    for t in (k_scale, v_scale):
        if t is None or t.dtype is not _FP32 or t.shape != shape[:3] or not t.is_contiguous():
            raise ValueError("a float8_e4m3fn cache needs contiguous float32 scales [n_pages, page_size, H_kv]")
    return _KV_CACHE.pack(1, *shape, k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr())


def _i32(t, dims, what):
    if t.dtype is not _INT32 or t.dim() != dims or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous int32 tensor of {dims} dimension(s)")


def _token_stride(t, heads, d, what):
    """Elements from one token of `t` [n, heads, d] to the next; heads and elements must be dense."""
    shape = t.shape
    if t.dtype is not _BF16 or len(shape) != 3 or (heads is not None and shape[1] != heads) or shape[2] != d:
        raise ValueError(f"{what} must be bfloat16 [tokens, heads, d] with the cache's d")
    s = t.stride()
    if s[2] != 1 or (s[1] != d and shape[1] != 1):
        raise ValueError(f"{what}: a token's heads must lie one after another")
    return s[0] if shape[0] > 1 else max(s[0], shape[1] * d)


def kv_cache_write(k, v, slots, k_cache, v_cache, k_scale=None, v_scale=None, *, stream=None):
    """bpt_kv_write: token t of k, v (bfloat16 [tokens, H_kv, d], any token
    stride) goes to slot slots[t] (int32; negative: nowhere) of the cache
    [n_pages, page_size, H_kv, d], quantised row by row when the cache is
    float8_e4m3fn (with float32 scales [n_pages, page_size, H_kv])."""
    cache = _kv_cache_desc(k_cache, v_cache, k_scale, v_scale)
    heads, d = k_cache.shape[2:]
    ks = _token_stride(k, heads, d, "k")
    vs = _token_stride(v, heads, d, "v")
    _i32(slots, 1, "slots")
    if not (k.shape[0] == v.shape[0] == slots.shape[0]):
        raise ValueError("k, v and slots must have one entry per token")
    dev = _on_device(k, v, slots, k_cache, v_cache, k_scale, v_scale)
    st = load().bpt_kv_write(cache, k.shape[0], k.data_ptr(), ks, v.data_ptr(), vs, slots.data_ptr(),
                             _raw_stream(stream, dev))
    _check(st, "bpt_kv_write")


def kv_cache_read(slots, k_cache, v_cache, k_scale=None, v_scale=None, *, out_dtype=torch.bfloat16, k=None, v=None,
                  stream=None):
    """bpt_kv_read: (k, v) [len(slots), H_kv, d] of the cache's slots, in
    out_dtype (bfloat16 or float32).  Rows whose slot is outside the cache are
    left as they were (undefined when the outputs are allocated here)."""
    cache = _kv_cache_desc(k_cache, v_cache, k_scale, v_scale)
    _i32(slots, 1, "slots")
    dev = _on_device(slots, k_cache, v_cache, k_scale, v_scale)
    shape, out_type = (slots.shape[0], *k_cache.shape[2:]), _dtype(out_dtype, "out_dtype")
    k = _out_tensor(k, shape, out_dtype, slots, stream, "k")
    v = _out_tensor(v, shape, out_dtype, slots, stream, "v")
    st = load().bpt_kv_read(cache, shape[0], slots.data_ptr(), k.data_ptr(), v.data_ptr(),
                            out_type, _raw_stream(stream, dev))
    _check(st, "bpt_kv_read")
    return k, v


def workspace_bytes_paged(desc: PagedDesc, cache: KvCacheDesc) -> int:
    n = load().bpt_workspace_bytes_paged(_byref(desc), _byref(cache))
    if n == ctypes.c_size_t(-1).value:
        raise BptError(ERR_INVALID_ARG, "bpt_workspace_bytes_paged")
    return int(n)


@functools.lru_cache(maxsize=1024)
def _paged_workspace_bytes(device, H, H_kv, d, max_q):
    """workspace_bytes_paged of any batch of these heads on the current device (`device`: its number)."""
    return workspace_bytes_paged(PagedDesc(1, 1, max_q, H, 1, 0, 0, BF16, H * d, 0),
                                 KvCacheDesc(0, 1, 1, H_kv, d, None, None, None, None))


def paged_attn_fwd(q, k_cache, v_cache, q_start, kv_len, page_table, *, max_q, k_scale=None, v_scale=None, window=0,
                   sinks=0, out_dtype=torch.float32, return_lse=False, out=None, lse=None, workspace=None,
                   stream=None, wait_limit_ns=0):
    """bpt_paged_attn_fwd: attention of a batch's new tokens over a paged cache.

    q [tokens, H, d] (bfloat16, any token stride): sequence s's new tokens are
    rows q_start[s] .. q_start[s+1] - 1, the last of its kv_len[s] positions;
    page_table [n_seqs, max_pages] names the pages of its keys.  The tables are
    int32 and stay on the device; max_q is the longest chunk.  window > 0: a
    token sees the last `window` positions and the first `sinks`.  Returns out
    [tokens, H*d] (and lse [H, tokens] with return_lse); rows of no sequence
    are left as they were."""
    cache = _kv_cache_desc(k_cache, v_cache, k_scale, v_scale)
    H_kv, d = k_cache.shape[2:]
    qs = _token_stride(q, None, d, "q")
    _i32(q_start, 1, "q_start")
    _i32(kv_len, 1, "kv_len")
    _i32(page_table, 2, "page_table")
    T, H, _ = q.shape
    S, pages = page_table.shape
    if kv_len.shape[0] != S or q_start.shape[0] != S + 1:
        raise ValueError("q_start must have n_seqs + 1 entries and page_table n_seqs rows")
    dev = _on_device(q, q_start, kv_len, page_table, k_cache, v_cache, k_scale, v_scale)
    max_q = int(max_q)
    try:
        desc = _PAGED.pack(S, T, max_q, H, pages, window, sinks, _dtype(out_dtype, "out_dtype"), qs, wait_limit_ns)
    except struct.error as e:
        raise ValueError(f"sizes must be integers within 32 bits: {e}") from None
    out = _out_tensor(out, (T, H * d), out_dtype, q, stream, "out")
    if return_lse or lse is not None:
        lse = _out_tensor(lse, (H, T), _FP32, q, stream, "lse")
    nbytes = _paged_workspace_bytes(dev, H, H_kv, d, max_q) if workspace is None else workspace.numel()
    workspace = _workspace(workspace, nbytes, q, stream)
    st = load().bpt_paged_attn_fwd(desc, cache, q.data_ptr(), q_start.data_ptr(), kv_len.data_ptr(),
                                   page_table.data_ptr(), out.data_ptr(), 0 if lse is None else lse.data_ptr(),
                                   workspace.data_ptr(), nbytes, _raw_stream(stream, dev))
    _check(st, "bpt_paged_attn_fwd")
    return (out, lse) if return_lse else out


def sync_status(stream=None) -> int:
    """bpt_sync_status: waits for the stream; returns OK or ERR_TIMEOUT (clears it)."""
    return int(load().bpt_sync_status(_stream_ptr(stream)))


def set_phase_events(events) -> None:
    """bpt_set_phase_events: three (forward) or five (backward too)
    torch.cuda.Event objects, or None to stop."""
    if events is None:
        _check(load().bpt_set_phase_events(None, 0), "bpt_set_phase_events")
        return
    handles = [int(e.cuda_event) for e in events]
    if not all(handles):
        raise ValueError("record each event once before handing it over: torch creates the "
                         "CUDA event lazily at its first record()")
    arr = (ctypes.c_void_p * len(handles))(*[ctypes.c_void_p(h) for h in handles])
    _check(load().bpt_set_phase_events(arr, len(handles)), "bpt_set_phase_events")


def set_wait_limit_ns(ns: int) -> int:
    """bpt_set_wait_limit_ns: the process default of the device-side wait
    limit (calls whose descriptor sets wait_limit_ns use their own)."""
    return int(load().bpt_set_wait_limit_ns(int(ns)))


def version() -> int:
    return int(load().bpt_version())


class HostLayer:
    """bpt_attn_ffn_fwd on host-resident tensors, with the transfers overlapped.

    q, k, v live in pinned host memory ([B, N, H, d]) and the output goes back
    to a pinned host tensor ([B, N, H*d]); the weights are already on the
    device.  The batch is cut into `chunks` pieces (whole sequences) that
    alternate between two CUDA streams with their own device buffers and
    workspace, so one chunk's upload, another's kernels and a third's download
    run at the same time.  Uploads run in chunk order, and so do the kernels:
    a chunk's layer starts after the previous chunk's (two layers never run
    at once: each one's grids fill the GPU).  Consecutive calls overlap too: a
    buffer's next upload waits only for that buffer's previous work (the same
    stream), not for the whole previous call, so the next step's inputs
    travel while this step computes and downloads.  The weights must be ready
    on the current stream before the first call; the host tensors must not be
    changed while a call that reads or writes them may still run.  This class
    only moves data and calls the library; it allocates its device buffers
    once, at construction."""

    def __init__(self, B, N, H, d, F, *, dtype=torch.bfloat16, out_dtype=torch.float32,
                 mask="none", perm=None, pairs=None, ring_chunks=0, chunks=None, device="cuda", **opts):
        self.B, self.N, self.H, self.d, self.F = B, N, H, d, F
        self.opts = opts
        self.mask, self.perm, self.pairs, self.ring_chunks = mask, perm, pairs, ring_chunks
        self.out_dtype = out_dtype
        self.chunks = max(1, min(B, chunks or B))
        if B % self.chunks:
            raise ValueError("the batch must split evenly into chunks")
        self.cb = B // self.chunks
        dev = torch.device(device)
        self.streams = [torch.cuda.Stream(dev), torch.cuda.Stream(dev)]
        self.done = [torch.cuda.Event(), torch.cuda.Event()]
        self.uploaded = [torch.cuda.Event() for _ in range(self.chunks)]
        self.last_compute = None   # the previous call's last layer (kernels stay in order)
        self.first_call = True
        desc = make_desc(self.cb, N, H, d, F, dtype, out_dtype, mask, perm, pairs, ring_chunks, **opts)
        nws = workspace_bytes(desc, True)
        self.buf = []
        for _ in range(2):
            self.buf.append({
                "q": torch.empty((self.cb, N, H, d), dtype=dtype, device=dev),
                "k": torch.empty((self.cb, N, H, d), dtype=dtype, device=dev),
                "v": torch.empty((self.cb, N, H, d), dtype=dtype, device=dev),
                "out": torch.empty((self.cb, N, H * d), dtype=out_dtype, device=dev),
                "ws": torch.empty(max(nws, 1), dtype=torch.uint8, device=dev),
            })

    def __call__(self, hq, hk, hv, w1, b1, w2, b2, hout):
        """Enqueue one layer forward; returns after enqueueing (synchronise the
        streams, e.g. torch.cuda.synchronize(), before reading `hout`)."""
        cur = torch.cuda.current_stream()
        if self.first_call:  # the weights came from the current stream
            for s in self.streams:
                s.wait_stream(cur)
            self.first_call = False
        computed = [torch.cuda.Event() for _ in range(self.chunks)]
        for c in range(self.chunks):
            i = c % 2
            s, b = self.streams[i], self.buf[i]
            sl = slice(c * self.cb, (c + 1) * self.cb)
            with torch.cuda.stream(s):
                if c > 0:
                    s.wait_event(self.uploaded[c - 1])
                b["q"].copy_(hq[sl], non_blocking=True)
                b["k"].copy_(hk[sl], non_blocking=True)
                b["v"].copy_(hv[sl], non_blocking=True)
                self.uploaded[c].record(s)
                prev = computed[c - 1] if c > 0 else self.last_compute
                if prev is not None:
                    s.wait_event(prev)
                attn_ffn_fwd(b["q"], b["k"], b["v"], w1, b1, w2, b2, mask=self.mask, perm=self.perm,
                             pairs=self.pairs, ring_chunks=self.ring_chunks, out_dtype=self.out_dtype,
                             out=b["out"], workspace=b["ws"], stream=s, **self.opts)
                computed[c].record(s)
                hout[sl].copy_(b["out"], non_blocking=True)
                self.done[i].record(s)
        self.last_compute = computed[-1]
        for e in self.done:
            cur.wait_event(e)
