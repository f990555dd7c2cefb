"""gqa_head_gated_gb300: gated causal GQA attention at head_dim 256 for GB300.

Thin PyTorch binding over the C ABI of libgqa_attn.so (include/gqa_attn.h).
It only checks and marshals arguments (pointers, sizes, the current CUDA
stream) and allocates outputs with torch; every step of the computation runs in
the library's CUDA kernels.  There is no CPU fallback: without the shared
library or a CUDA device the calls raise.  Every attention call takes bf16 or
fp16 tensors (one type per call) and picks the matching entry point.

    out = softmax(Q K^T / 16 + causal/offset mask) V * sigmoid(G)
"""
from __future__ import annotations

import ctypes
import functools
import math

import torch

from ._lib import GqaError, check, load  # noqa: F401

HEAD_DIM = 256

__all__ = ["prefill", "prefill_pair", "masked", "decode", "verify_tree", "kv_append", "kv_keep", "block_plan",
           "kv8_append", "kv8_keep", "kv8_decode", "kv8_workspace_size", "kv8_prefill",
           "kv8_prefill_workspace_size", "block_fork", "block_free", "block_compact", "kv8_copy", "rope",
           "rope_frequencies", "decode_plan", "decode_split", "lse_merge",
           "decode_workspace_size", "last_device_status", "set_wait_timeout_ns",
           "selftest_wait_timeout", "decode_noalloc", "launch_log", "GqaError",
           "load"]


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


_ELEM = {torch.bfloat16: "", torch.float16: "_f16"}


def _elem(t, name):
    """Entry-point suffix for the element type of `t` (bf16 or fp16)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in _ELEM:
        raise TypeError(f"{name} must be bfloat16 or float16, got {t.dtype}")
    return _ELEM[t.dtype]


def _need(t, dtype, ndim, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim or t.shape[-1] != HEAD_DIM and ndim >= 3:
        raise ValueError(f"{name} must be {ndim}-d with last dim {HEAD_DIM}, got {tuple(t.shape)}")
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")


def prefill(q, k, v, g=None, kv_offset=0, out=None, return_lse=False):
    """Prompt rows.  q, g: [B,Hq,Lq,256] bf16; k, v: [B,Hkv,Lkv,256] bf16.
    Row i sits at position kv_offset + i and sees keys 0..kv_offset+i.
    Returns out [B,Hq,Lq,256] bf16 (and lse [B,Hq,Lq] fp32 if return_lse).
    fp16 inputs run the fp16 kernels and give an fp16 out."""
    sfx = _elem(q, "q")
    _need(q, q.dtype, 4, "q")
    _need(k, q.dtype, 4, "k")
    _need(v, q.dtype, 4, "v")
    if g is not None:
        _need(g, q.dtype, 4, "g")
    B, Hq, Lq, _ = q.shape
    Hkv, Lkv = k.shape[1], k.shape[2]
    if out is None:
        out = torch.empty_like(q)
    lse = torch.empty((B, Hq, Lq), dtype=torch.float32, device=q.device) if return_lse else None
    _need(out, q.dtype, 4, "out")
    fn = getattr(load(), "gqa_attn_prefill" + sfx)
    code = fn(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(out), _ptr(lse), B, Hq, Hkv, Lq, Lkv,
              int(kv_offset), _stream())
    check(code, "gqa_attn_prefill" + sfx)
    return (out, lse) if return_lse else out


def prefill_pair(q, k, v, g=None, kv_offset=0, out=None, return_lse=False):
    """prefill() through gqa_attn_prefill_pair (CTA pairs sharing each K/V tile);
    bf16 only."""
    if q.dtype != torch.bfloat16:
        raise TypeError("prefill_pair takes bf16 inputs")
    _need(q, q.dtype, 4, "q")
    _need(k, q.dtype, 4, "k")
    _need(v, q.dtype, 4, "v")
    if g is not None:
        _need(g, q.dtype, 4, "g")
    B, Hq, Lq, _ = q.shape
    Hkv, Lkv = k.shape[1], k.shape[2]
    if out is None:
        out = torch.empty_like(q)
    lse = torch.empty((B, Hq, Lq), dtype=torch.float32, device=q.device) if return_lse else None
    _need(out, q.dtype, 4, "out")
    code = load().gqa_attn_prefill_pair(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(out), _ptr(lse),
                                        B, Hq, Hkv, Lq, Lkv, int(kv_offset), _stream())
    check(code, "gqa_attn_prefill_pair")
    return (out, lse) if return_lse else out


_MASK_KIND = {torch.bool: 1, torch.float32: 2, torch.bfloat16: 3, torch.float16: 4}


def masked(q, k, v, g=None, mask=None, causal=False, kv_offset=None, head_chunking=True,
           out=None, return_lse=False):
    """Gated attention with a general mask (the dense SDPA consumer's masks).

    q, g: [B,Hq,Lq,256]; k, v: [B,Hkv,Lkv,256]; bf16 or fp16.  mask: None, a bool
    tensor (True = attend) or a float32 / bf16 / fp16 tensor added to the scaled
    scores, of up to 4 dims broadcasting (trailing dims aligned) to [B, heads, Lq,
    Lkv]; any strides.  The head rule: with head_chunking, Lq <= 32 and Lq*GQA > 32
    the mask's head count must be 1 or the chunk size min(GQA, 32 // Lq) with no
    remainder chunk (chunk-local); otherwise 1 or Hq.  A mask that does not
    broadcast raises GqaError (GQA_ERR_INVALID_ARG) and launches nothing.
    causal: also hide keys j > kv_offset + i (kv_offset defaults to Lkv - Lq)."""
    sfx = _elem(q, "q")
    _need(q, q.dtype, 4, "q")
    _need(k, q.dtype, 4, "k")
    _need(v, q.dtype, 4, "v")
    if g is not None:
        _need(g, q.dtype, 4, "g")
    B, Hq, Lq, _ = q.shape
    Hkv, Lkv = k.shape[1], k.shape[2]
    if kv_offset is None:
        kv_offset = Lkv - Lq
    kind, mptr = 0, None
    shape = (ctypes.c_longlong * 4)(1, 1, 1, 1)
    strides = (ctypes.c_longlong * 4)(0, 0, 0, 0)
    if mask is not None:
        if not isinstance(mask, torch.Tensor) or mask.dtype not in _MASK_KIND:
            raise TypeError("mask must be a bool, float32, bfloat16 or float16 tensor")
        if not mask.is_cuda:
            raise ValueError("mask must be a CUDA tensor")
        if mask.dim() > 4:
            raise GqaError(1, "gqa_attn_masked: mask has more than 4 dimensions")
        pad = 4 - mask.dim()
        for d in range(4):
            if d >= pad:
                shape[d] = mask.shape[d - pad]
                strides[d] = mask.stride(d - pad)
        kind, mptr = _MASK_KIND[mask.dtype], _ptr(mask)
    if out is None:
        out = torch.empty_like(q)
    _need(out, q.dtype, 4, "out")
    lse = torch.empty((B, Hq, Lq), dtype=torch.float32, device=q.device) if return_lse else None
    fn = getattr(load(), "gqa_attn_masked" + sfx)
    code = fn(_ptr(q), _ptr(k), _ptr(v), _ptr(g), mptr, kind, shape, strides, _ptr(out),
              _ptr(lse), B, Hq, Hkv, Lq, Lkv, int(bool(causal)), int(kv_offset),
              int(bool(head_chunking)), _stream())
    check(code, "gqa_attn_masked" + sfx)
    return (out, lse) if return_lse else out


def decode_plan(B, T, Hq, Hkv, max_rows, max_kv_len):
    """(num_splits, split_keys) that decode() uses for these sizes."""
    s, c = ctypes.c_int(0), ctypes.c_int(0)
    check(load().gqa_attn_decode_plan(B, T, Hq, Hkv, max_rows, max_kv_len, ctypes.byref(s),
                                      ctypes.byref(c)), "gqa_attn_decode_plan")
    return s.value, c.value


def decode_workspace_size(B, T, Hq, Hkv, max_rows, max_kv_len):
    return int(load().gqa_attn_decode_workspace_size(B, T, Hq, Hkv, max_rows, max_kv_len))


def _decode_sizes(q, k_cache, kv_lens, cu_rows, max_rows, max_kv_len):
    T, Hq, _ = q.shape
    B, Hkv, Lcap, _ = k_cache.shape
    if kv_lens.dtype != torch.int32 or not kv_lens.is_cuda or kv_lens.numel() != B:
        raise ValueError("kv_lens must be an int32 CUDA tensor of B entries")
    if cu_rows is not None and (cu_rows.dtype != torch.int32 or not cu_rows.is_cuda
                                or cu_rows.numel() != B + 1):
        raise ValueError("cu_rows must be an int32 CUDA tensor of B+1 entries")
    if max_kv_len is None:           # synchronises; pass it to avoid the copy
        max_kv_len = int(kv_lens.max().item())
    if max_rows is None:
        max_rows = 1 if cu_rows is None else int((cu_rows[1:] - cu_rows[:-1]).max().item())
    return T, Hq, B, Hkv, Lcap, int(max_rows), int(max_kv_len)


def decode(q, k_cache, v_cache, g, kv_lens, cu_rows=None, max_rows=None, max_kv_len=None,
           workspace=None, out=None, return_lse=False):
    """Decode / chain-verify rows.  q, g: [T,Hq,256] bf16 token-major; caches
    [B,Hkv,Lcap,256] bf16; kv_lens int32 [B] (counts the new rows); cu_rows int32
    [B+1] or None (one row per sequence).  Returns out [T,Hq,256] bf16 (fp16 for
    fp16 inputs)."""
    sfx = _elem(q, "q")
    _need(q, q.dtype, 3, "q")
    _need(k_cache, q.dtype, 4, "k_cache")
    _need(v_cache, q.dtype, 4, "v_cache")
    if g is not None:
        _need(g, q.dtype, 3, "g")
    T, Hq, B, Hkv, Lcap, max_rows, max_kv_len = _decode_sizes(q, k_cache, kv_lens, cu_rows,
                                                               max_rows, max_kv_len)
    if workspace is None:    # (a given workspace is checked by the library itself)
        need = decode_workspace_size(B, T, Hq, Hkv, max_rows, max_kv_len)
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    if out is None:
        out = torch.empty_like(q)
    lse = torch.empty((T, Hq), dtype=torch.float32, device=q.device) if return_lse else None
    _need(out, q.dtype, 3, "out")
    fn = getattr(load(), "gqa_attn_decode" + sfx)
    code = fn(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(g), _ptr(kv_lens), _ptr(cu_rows),
              _ptr(out), _ptr(lse), B, T, Hq, Hkv, Lcap, max_rows, max_kv_len, _ptr(workspace),
              workspace.numel() * workspace.element_size(), _stream())
    check(code, "gqa_attn_decode" + sfx)
    return (out, lse) if return_lse else out


def decode_noalloc(q, k_cache, v_cache, g, kv_lens, cu_rows=None, max_rows=None,
                   max_kv_len=None, out=None, return_lse=False):
    """decode() through gqa_attn_decode_noalloc: the library's fixed 16 MiB area is the
    workspace (bf16 only; calls whose workspace would not fit raise GQA_ERR_WORKSPACE).
    Same kernels, plan and results as decode()."""
    if q.dtype != torch.bfloat16:
        raise TypeError("decode_noalloc takes bf16 inputs")
    _need(q, q.dtype, 3, "q")
    _need(k_cache, q.dtype, 4, "k_cache")
    _need(v_cache, q.dtype, 4, "v_cache")
    if g is not None:
        _need(g, q.dtype, 3, "g")
    T, Hq, B, Hkv, Lcap, max_rows, max_kv_len = _decode_sizes(q, k_cache, kv_lens, cu_rows,
                                                               max_rows, max_kv_len)
    if out is None:
        out = torch.empty_like(q)
    lse = torch.empty((T, Hq), dtype=torch.float32, device=q.device) if return_lse else None
    _need(out, q.dtype, 3, "out")
    code = load().gqa_attn_decode_noalloc(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(g),
                                          _ptr(kv_lens), _ptr(cu_rows), _ptr(out), _ptr(lse), B,
                                          T, Hq, Hkv, Lcap, max_rows, max_kv_len, _stream())
    check(code, "gqa_attn_decode_noalloc")
    return (out, lse) if return_lse else out


def launch_log(n=64):
    """The library's record of its last kernel launches (at most 64), newest first:
    dicts of kernel, seq, grid, block, dynamic_smem, as the launches used them."""
    from ._lib import LaunchInfo
    buf = (LaunchInfo * n)()
    got = load().gqa_launch_log(buf, n)
    if got < 0:
        check(-got, "gqa_launch_log")
    return [{"kernel": r.kernel.decode(), "seq": int(r.seq), "grid": int(r.grid),
             "block": int(r.block), "dynamic_smem": int(r.dynamic_smem)} for r in buf[:got]]


def verify_tree(q, k_cache, v_cache, g, kv_lens, cu_rows, tree_mask, max_rows=None,
                max_kv_len=None, workspace=None, out=None, return_lse=False):
    """Draft verify over token trees.  As decode(), plus tree_mask: int64 [T] CUDA
    tensor, one mask per new row over its sequence's new rows (bit k: new row k
    visible; its ancestors and itself).  Rows per sequence <= 64.  bf16 or fp16."""
    sfx = _elem(q, "q")
    _need(q, q.dtype, 3, "q")
    _need(k_cache, q.dtype, 4, "k_cache")
    _need(v_cache, q.dtype, 4, "v_cache")
    if g is not None:
        _need(g, q.dtype, 3, "g")
    if cu_rows is None:
        raise ValueError("cu_rows is required for tree verify")
    if (tree_mask.dtype != torch.int64 or not tree_mask.is_cuda or not tree_mask.is_contiguous()
            or tree_mask.numel() != q.shape[0]):
        raise ValueError("tree_mask must be a contiguous int64 CUDA tensor of T entries")
    T, Hq, B, Hkv, Lcap, max_rows, max_kv_len = _decode_sizes(q, k_cache, kv_lens, cu_rows,
                                                               max_rows, max_kv_len)
    need = decode_workspace_size(B, T, Hq, Hkv, max_rows, max_kv_len)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    if out is None:
        out = torch.empty_like(q)
    lse = torch.empty((T, Hq), dtype=torch.float32, device=q.device) if return_lse else None
    _need(out, q.dtype, 3, "out")
    fn = getattr(load(), "gqa_attn_verify_tree" + sfx)
    code = fn(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(g), _ptr(kv_lens), _ptr(cu_rows),
              _ptr(tree_mask), _ptr(out), _ptr(lse), B, T, Hq, Hkv, Lcap, max_rows, max_kv_len,
              _ptr(workspace), workspace.numel() * workspace.element_size(), _stream())
    check(code, "gqa_attn_verify_tree" + sfx)
    return (out, lse) if return_lse else out


def kv_append(k_new, v_new, kv_lens, k_cache, v_cache, cu_rows=None):
    """Writes new rows ([T,Hkv,256] bf16) after the kv_lens[b] keys each sequence
    holds in the caches ([B,Hkv,Lcap,256]); kv_lens itself is not updated.  The
    copy moves 16-bit elements: bf16 or fp16, the same type throughout."""
    _elem(k_cache, "k_cache")
    for t, n in ((k_new, "k_new"), (v_new, "v_new")):
        _need(t, k_cache.dtype, 3, n)
    _need(k_cache, k_cache.dtype, 4, "k_cache")
    _need(v_cache, k_cache.dtype, 4, "v_cache")
    T, Hkv, _ = k_new.shape
    B, _, Lcap, _ = k_cache.shape
    check(load().gqa_kv_append(_ptr(k_new), _ptr(v_new), _ptr(cu_rows), _ptr(kv_lens),
                               _ptr(k_cache), _ptr(v_cache), B, T, Hkv, Lcap, _stream()),
          "gqa_kv_append")


def kv_keep(k_cache, v_cache, kv_lens, cu_rows, keep_idx, cu_keep, kv_lens_out=None):
    """Moves the accepted draft rows (keep_idx, per sequence via cu_keep, strictly
    increasing draft-row indices) to the front of each sequence's draft region, in
    place; writes the new lengths into kv_lens_out when given.  bf16 or fp16."""
    _elem(k_cache, "k_cache")
    _need(k_cache, k_cache.dtype, 4, "k_cache")
    _need(v_cache, k_cache.dtype, 4, "v_cache")
    B, Hkv, Lcap, _ = k_cache.shape
    check(load().gqa_kv_keep(_ptr(k_cache), _ptr(v_cache), _ptr(kv_lens), _ptr(cu_rows),
                             _ptr(keep_idx), _ptr(cu_keep), _ptr(kv_lens_out), B, Hkv, Lcap,
                             _stream()), "gqa_kv_keep")


# The paged 8-bit cache.  A step's calls are short, so their checks are written to cost
# little: each gives the tensor's address, and the message is made only for a refusal.
_I32, _F32, _F8 = torch.int32, torch.float32, torch.float8_e4m3fn
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_entry = {}     # entry points by name


def _stream_of(d):
    return (_raw_stream(d) if _raw_stream is not None
            else torch.cuda.current_stream(d).cuda_stream)


def _at(t, dtype, shape, d, name):
    """Address of a contiguous CUDA tensor of this type and shape on device d."""
    try:
        if (t.dtype is dtype and t.shape == shape and t.get_device() == d
                and t.is_contiguous()):
            return t.data_ptr()
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} must be a contiguous tensor of shape {tuple(shape)} on cuda:{d}, got "
                     f"{tuple(t.shape)} on {t.device}")


def _cuda_index(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    d = t.get_device()
    if d < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return d


def _tables(block_tables, B, d):
    """(address, max_blocks) of int32 block_tables [B, max_blocks]."""
    if not isinstance(block_tables, torch.Tensor) or block_tables.dim() != 2:
        raise ValueError("block_tables must be an int32 CUDA tensor [B, max_blocks]")
    m = block_tables.shape[1]
    return _at(block_tables, _I32, (B, m), d, "block_tables"), m


def _kv8_pools(k_pool, v_pool, k_scale, v_scale):
    """Device, (num_blocks, Hkv, block_size) and addresses of checked pools and scales."""
    d = _cuda_index(k_pool, "k_pool")
    shape = k_pool.shape
    if len(shape) != 4 or shape[3] != HEAD_DIM:
        raise ValueError(f"k_pool must be [num_blocks, Hkv, block_size, {HEAD_DIM}], got "
                         f"{tuple(shape)}")
    N, Hkv, bs, _ = shape
    scales = (N, Hkv)
    return (d, N, Hkv, bs, _at(k_pool, _F8, shape, d, "k_pool"), _at(v_pool, _F8, shape, d, "v_pool"),
            _at(k_scale, _F32, scales, d, "k_scale"), _at(v_scale, _F32, scales, d, "v_scale"))


def _call(name, d, *args):
    """Runs an entry point on device d's current stream (its last argument)."""
    fn = _entry.get(name)
    if fn is None:
        fn = _entry[name] = getattr(load(), name)
    if _current_device() == d:
        code = fn(*args, _stream_of(d))
    else:
        with torch.cuda.device(d):
            code = fn(*args, _stream_of(d))
    if code:
        raise GqaError(code, name)


def block_plan(kv_lens, cu_rows, block_tables, n_blocks, free_list, free_count, block_size, T,
               slots=None, kv_lens_out=None):
    """Block tables and slot maps of a paged cache from request lengths, on the GPU.

    Sequence b holds kv_lens[b] keys and gets cu_rows[b+1] - cu_rows[b] new rows; after the
    call it owns exactly the blocks that they need.  int32 CUDA tensors, updated in place:
    block_tables [B, max_blocks], n_blocks [B], free_list [num_blocks] and free_count [1] (a
    stack).  A block that it releases is in no other table: blocks that block_fork() shared are given
    back by block_free().  Surplus blocks go back first (length 0 and no rows: a finished request), then
    growing sequences take theirs in order.  T: rows in the batch, cu_rows[B] or more.
    Returns (slots int32 [T], kv_lens_out int32 [B]): the place of each new row (block *
    block_size + row; -1 without one) for kv8_append, and the lengths with the new rows for
    kv8_decode.  A sequence that the pool has no blocks for keeps its length, its slots are
    -1, and last_device_status() gives GQA_ERR_NO_BLOCKS (7)."""
    d = _cuda_index(kv_lens, "kv_lens")
    B, T, N = kv_lens.numel(), int(T), free_list.numel()
    if slots is None:
        slots = torch.empty(max(T, 0), dtype=_I32, device=kv_lens.device)
    if kv_lens_out is None:
        kv_lens_out = torch.empty_like(kv_lens)
    tables, max_blocks = _tables(block_tables, B, d)
    _call("gqa_block_plan", d, _at(kv_lens, _I32, (B,), d, "kv_lens"),
          _at(cu_rows, _I32, (B + 1,), d, "cu_rows"), tables,
          _at(n_blocks, _I32, (B,), d, "n_blocks"), _at(free_list, _I32, (N,), d, "free_list"),
          _at(free_count, _I32, (1,), d, "free_count"), _at(slots, _I32, (T,), d, "slots"),
          _at(kv_lens_out, _I32, (B,), d, "kv_lens_out"), B, T, max_blocks, N, int(block_size))
    return slots, kv_lens_out


def kv8_append(k_new, v_new, slots, k_pool, v_pool, k_scale, v_scale):
    """Quantises new rows ([T,Hkv,256] bf16 or fp16) into the paged 8-bit cache at their slots
    (int32 [T], from block_plan; -1 skips a row).  k_pool, v_pool: float8_e4m3fn [num_blocks,
    Hkv, block_size, 256]; k_scale, v_scale: float32 [num_blocks, Hkv], one power of two per
    block and head, kept as large as the block's rows ask (rows that a block holds already
    are rounded again when its scale grows).  Rows of one block have increasing slots; a row
    that repeats an earlier one's is skipped, and last_device_status() gives
    GQA_ERR_DEVICE_RANGE (6)."""
    sfx = _elem(k_new, "k_new")
    d, N, Hkv, bs, *pools = _kv8_pools(k_pool, v_pool, k_scale, v_scale)
    T, shape = k_new.shape[0], (k_new.shape[0], Hkv, HEAD_DIM)
    _call("gqa_kv8_append" + sfx, d, _at(k_new, k_new.dtype, shape, d, "k_new"),
          _at(v_new, k_new.dtype, shape, d, "v_new"), _at(slots, _I32, (T,), d, "slots"), *pools, T,
          Hkv, N, bs)


def kv8_keep(k_pool, v_pool, k_scale, v_scale, block_tables, kv_lens, cu_rows, keep_idx, cu_keep,
             kv_lens_out=None):
    """kv_keep() for the paged 8-bit cache: the accepted draft rows (at most 64 per sequence)
    move to the front of each sequence's draft region, as if their values had been appended
    there; writes the new lengths into kv_lens_out when given."""
    d, N, Hkv, bs, *pools = _kv8_pools(k_pool, v_pool, k_scale, v_scale)
    _cuda_index(kv_lens, "kv_lens")
    _cuda_index(keep_idx, "keep_idx")
    B, n = kv_lens.numel(), keep_idx.numel()
    tables, max_blocks = _tables(block_tables, B, d)
    _call("gqa_kv8_keep", d, *pools, tables, _at(kv_lens, _I32, (B,), d, "kv_lens"),
          _at(cu_rows, _I32, (B + 1,), d, "cu_rows"), _at(keep_idx, _I32, (n,), d, "keep_idx"),
          _at(cu_keep, _I32, (B + 1,), d, "cu_keep"),
          None if kv_lens_out is None else _at(kv_lens_out, _I32, (B,), d, "kv_lens_out"), n, B,
          Hkv, N, bs, max_blocks)


def kv8_workspace_size(B, T, Hq, Hkv, max_rows, max_kv_len):
    """Bytes of workspace that kv8_decode() needs for these sizes (on the current device)."""
    return int(load().gqa_kv8_workspace_size(B, T, Hq, Hkv, max_rows, max_kv_len))


def kv8_decode(q, k_pool, v_pool, k_scale, v_scale, g, block_tables, kv_lens, cu_rows=None,
               tree_mask=None, max_rows=None, max_kv_len=None, workspace=None, out=None,
               return_lse=False):
    """Decode, chain-verify and (with tree_mask, int64 [T]) tree-verify rows over the paged
    8-bit cache.  q, g: [T,Hq,256] bf16 or fp16; pools and scales as kv8_append writes them;
    block_tables int32 [B, max_blocks]; kv_lens int32 [B] counts the new rows; cu_rows int32
    [B+1] or None (one row per sequence).  Returns out [T,Hq,256]; rows behind cu_rows[B] (a
    padded batch) are left as they were in a given out."""
    sfx = _elem(q, "q")
    d, N, Hkv, bs, *pools = _kv8_pools(k_pool, v_pool, k_scale, v_scale)
    if q.dim() != 3 or q.shape[2] != HEAD_DIM:
        raise ValueError(f"q must be [T, Hq, {HEAD_DIM}], got {tuple(q.shape)}")
    T, Hq, _ = shape = q.shape
    _cuda_index(kv_lens, "kv_lens")
    B = kv_lens.numel()
    tables, max_blocks = _tables(block_tables, B, d)
    if max_kv_len is None:           # synchronises; pass it to avoid the copy
        max_kv_len = max(1, int(kv_lens.max().item()))
    if max_rows is None:
        max_rows = 1 if cu_rows is None else max(1, int((cu_rows[1:] - cu_rows[:-1]).max().item()))
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:    # (a given workspace is checked by the library itself)
        with torch.cuda.device(d):
            need = kv8_workspace_size(B, T, Hq, Hkv, max_rows, max_kv_len)
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    elif workspace.get_device() != d or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{d}")
    lse = torch.empty((T, Hq), dtype=_F32, device=q.device) if return_lse else None
    dt = q.dtype
    _call("gqa_kv8_decode" + sfx, d, _at(q, dt, shape, d, "q"), *pools,
          None if g is None else _at(g, dt, shape, d, "g"), tables,
          _at(kv_lens, _I32, (B,), d, "kv_lens"),
          None if cu_rows is None else _at(cu_rows, _I32, (B + 1,), d, "cu_rows"),
          None if tree_mask is None else _at(tree_mask, torch.int64, (T,), d, "tree_mask"),
          _at(out, dt, shape, d, "out"), None if lse is None else lse.data_ptr(), B, T, Hq, Hkv, N,
          bs, max_blocks, int(max_rows), int(max_kv_len), workspace.data_ptr(),
          workspace.numel() * workspace.element_size())
    return (out, lse) if return_lse else out


def block_fork(src, dst, lens, kv_lens, block_tables, n_blocks, free_list, free_count, shares,
               block_size, copies=None):
    """Forks sequences of a paged cache: child dst[f] gets the first lens[f] keys (None: all) of parent
    src[f], sharing its full blocks; int32 CUDA tensors, kv_lens, block_tables, n_blocks, free_count and
    shares (int32 [num_blocks]: tables that hold a block beside the first) updated in place.  A child holds
    no blocks before, and is neither a parent nor a child twice.  Returns copies int32 [F, 3], what
    kv8_copy() has to copy (from, to, rows): the rows behind a prefix's last full block go to a block of the
    child's own.  A refused fork records GQA_ERR_DEVICE_RANGE (6), one without a free block
    GQA_ERR_NO_BLOCKS (7)."""
    d = _cuda_index(src, "src")
    F, B, N = src.numel(), kv_lens.numel(), free_list.numel()
    if copies is None:
        copies = src.new_empty((F, 3), dtype=_I32)
    tables, max_blocks = _tables(block_tables, B, d)
    _call("gqa_block_fork", d, _at(src, _I32, (F,), d, "src"), _at(dst, _I32, (F,), d, "dst"),
          None if lens is None else _at(lens, _I32, (F,), d, "lens"),
          _at(kv_lens, _I32, (B,), d, "kv_lens"), tables, _at(n_blocks, _I32, (B,), d, "n_blocks"),
          _at(free_list, _I32, (N,), d, "free_list"), _at(free_count, _I32, (1,), d, "free_count"),
          _at(shares, _I32, (N,), d, "shares"), _at(copies, _I32, (F, 3), d, "copies"), F, B, max_blocks,
          N, int(block_size))
    return copies


def block_free(kv_lens, block_tables, n_blocks, free_list, free_count, shares, block_size):
    """Gives blocks back that sequences may share: sequence b keeps those of its first kv_lens[b] keys (0: it has
    ended), and a block that no table holds any more goes on the stack.  int32 CUDA tensors, all but
    kv_lens updated in place.  (block_plan() does the same for blocks that are never shared.)"""
    d = _cuda_index(kv_lens, "kv_lens")
    B, N = kv_lens.numel(), free_list.numel()
    tables, max_blocks = _tables(block_tables, B, d)
    _call("gqa_block_free", d, _at(kv_lens, _I32, (B,), d, "kv_lens"), tables,
          _at(n_blocks, _I32, (B,), d, "n_blocks"), _at(free_list, _I32, (N,), d, "free_list"),
          _at(free_count, _I32, (1,), d, "free_count"), _at(shares, _I32, (N,), d, "shares"), B,
          max_blocks, N, int(block_size))


def block_compact(block_tables, n_blocks, free_list, free_count, shares, block_size):
    """Moves the live blocks of a pool to its first places.  Returns new tensors (block_tables, free_list,
    shares, new_index int32 [num_blocks], copies int32 [num_blocks // 2, 3]); the inputs stay as they
    are.  The new tables hold once kv8_copy(copies, ...) has run on the pools (every layer's, where layers share
    tables); free_count and n_blocks do not change.  new_index tells where a block went (-1: it is free)."""
    d = _cuda_index(block_tables, "block_tables")
    B, N = n_blocks.numel(), free_list.numel()
    tables, max_blocks = _tables(block_tables, B, d)
    out = torch.empty_like(block_tables)
    list_at = _at(free_list, _I32, (N,), d, "free_list")
    new_free, new_shares, index = (torch.empty_like(free_list) for _ in range(3))
    copies = free_list.new_empty((N // 2, 3))
    _call("gqa_block_compact", d, tables, _at(n_blocks, _I32, (B,), d, "n_blocks"),
          list_at, _at(free_count, _I32, (1,), d, "free_count"),
          _at(shares, _I32, (N,), d, "shares"), out.data_ptr(), new_free.data_ptr(),
          new_shares.data_ptr(), index.data_ptr(), copies.data_ptr(), B, max_blocks, N, int(block_size))
    return out, new_free, new_shares, index, copies


def kv8_copy(copies, k_pool, v_pool, k_scale, v_scale):
    """Copies blocks of the paged 8-bit cache, K, V and scales: copies int32 [n, 3] of (from, to, rows) as
    block_fork() and block_compact() list them (negative: none)."""
    d, N, Hkv, bs, *pools = _kv8_pools(k_pool, v_pool, k_scale, v_scale)
    _cuda_index(copies, "copies")
    n = copies.shape[0] if copies.dim() else 0
    _call("gqa_kv8_copy", d, _at(copies, _I32, (n, 3), d, "copies"), *pools, n, Hkv, N, bs)


def rope_frequencies(rot_dims, base=10000.0, method=None, factor=1.0, original_len=None, beta_fast=32.0,
                     beta_slow=1.0, device="cuda"):
    """(inv_freq float32 [rot_dims / 2] on `device`, scale) for rope(): base^(-2j / rot_dims), for contexts
    `factor` times longer than trained with the method
      "linear"  every frequency / factor (position interpolation);
      "ntk"     base * factor^(rot_dims / (rot_dims - 2)), which leaves the highest frequency as it is;
      "yarn"    the frequencies that turn less than beta_slow times over original_len / factor, those that turn
                more than beta_fast times kept, a ramp between them; scale 0.1 ln(factor) + 1.
    Worked out in 64 bits."""
    if rot_dims < 16 or rot_dims > HEAD_DIM or rot_dims % 16:
        raise ValueError(f"rot_dims must be a multiple of 16 up to {HEAD_DIM}, got {rot_dims}")
    if method not in (None, "linear", "ntk", "yarn"):
        raise ValueError(f"method must be None, 'linear', 'ntk' or 'yarn', got {method!r}")
    if not (base > 1 and factor >= 1):
        raise ValueError("base must be above 1 and factor 1 or more")
    if method == "ntk":
        base = base * factor ** (rot_dims / (rot_dims - 2))
    j = torch.arange(rot_dims // 2, dtype=torch.float64)
    freq, scale = base ** (-2.0 * j / rot_dims), 1.0
    if method == "linear":
        freq = freq / factor
    elif method == "yarn":
        if not original_len or beta_fast <= beta_slow:
            raise ValueError("yarn needs original_len, and beta_fast above beta_slow")
        # the pair that turns `beta` times over original_len
        pair = lambda beta: (rot_dims * math.log(original_len / (beta * 2 * math.pi))  # noqa: E731
                             / (2 * math.log(base)))
        low = max(math.floor(pair(beta_fast)), 0)
        high = min(math.ceil(pair(beta_slow)), rot_dims - 1)
        ramp = ((j - low) / (high - low)).clamp(0, 1) if high > low else (j >= high).double()
        freq = freq / factor * ramp + freq * (1 - ramp)
        scale = 0.1 * math.log(factor) + 1.0
    return freq.float().to(device), scale


@functools.lru_cache(maxsize=256)
def _rope_strides(*strides):
    return (ctypes.c_longlong * len(strides))(*strides)


def _rope_rows(t, dtype, shape, d, name):
    """Address and (batch, token, head) strides of [T, H, 256] or [B, H, L, 256] with the last dim in a row."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == d:
            s = t.stride()
            if s[-1] == 1:
                return (t.data_ptr(), 0, s[0], s[1]) if len(s) == 3 else (t.data_ptr(), s[0], s[2], s[1])
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} must be {tuple(shape)} on cuda:{d} with its last dim in a row, got {tuple(t.shape)} "
                     f"of strides {tuple(t.stride())} on {t.device}")


def rope(q, k, positions, inv_freq, interleaved=False, scale=1.0, inverse=False, q_out=None, k_out=None):
    """Rotary positions of queries and keys in one launch; returns (q, k) rotated.

    q [T,Hq,256] and k [T,Hkv,256] (or None) with positions int32 [T], or the prefill layout [B,Hq,L,256] /
    [B,Hkv,L,256] with positions int32 [L] or [B,L]; bf16 or fp16, any strides with the last dim in a row
    (slices of a fused projection).  inv_freq: float32 [rot_dims / 2], see rope_frequencies(); the first rot_dims
    dims of a head turn, in pairs (j, j + rot_dims / 2) or, interleaved, (2 j, 2 j + 1), the others are copied.
    scale multiplies what is turned.  inverse: the rotation back (also the gradient's).  q_out / k_out may be
    q / k themselves; by default the outputs are new and contiguous."""
    sfx = _elem(q, "q")
    d = _cuda_index(q, "q")
    shape, dt = q.shape, q.dtype
    if len(shape) == 3:
        B, (L, Hq, D) = 1, shape
    elif len(shape) == 4:
        B, Hq, L, D = shape
    else:
        D = None
    if D != HEAD_DIM:
        raise ValueError(f"q must be [T, Hq, {HEAD_DIM}] or [B, Hq, L, {HEAD_DIM}], got {tuple(shape)}")
    if q_out is None:
        q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
    qa, *qs = _rope_rows(q, dt, shape, d, "q")
    oa, *os_ = _rope_rows(q_out, dt, shape, d, "q_out")
    if k is None:
        if k_out is not None:
            raise ValueError("k_out without k")
        Hkv, ka, koa, ks, kos = 0, None, None, (), ()
    else:
        if not isinstance(k, torch.Tensor) or k.dim() != len(shape):
            raise ValueError("k must be a tensor of q's layout")
        Hkv = k.shape[1]
        k_shape = (L, Hkv, D) if len(shape) == 3 else (B, Hkv, L, D)
        if k_out is None:
            k_out = torch.empty_like(k, memory_format=torch.contiguous_format)
        ka, *ks = _rope_rows(k, dt, k_shape, d, "k")
        koa, *kos = _rope_rows(k_out, dt, k_shape, d, "k_out")
    _cuda_index(positions, "positions")
    batch = positions.dim() == 2
    where = _at(positions, _I32, (B, L) if batch else (L,), d, "positions")
    _cuda_index(inv_freq, "inv_freq")
    half = inv_freq.numel()
    _call("gqa_rope" + sfx, d, qa, ka, where, _at(inv_freq, _F32, (half,), d, "inv_freq"), oa, koa,
          _rope_strides(*qs, *os_, *ks, *kos), B, L, Hq, Hkv, 2 * half, batch, bool(interleaved),
          bool(inverse), scale)
    return q_out, k_out


def kv8_prefill_workspace_size():
    """Bytes of workspace that kv8_prefill() needs, whatever the sizes (on the current device)."""
    return int(load().gqa_kv8_prefill_workspace_size())


def kv8_prefill(q, k_pool, v_pool, k_scale, v_scale, g, block_tables, kv_lens, cu_rows,
                max_rows=None, max_kv_len=None, workspace=None, out=None, return_lse=False):
    """Prompt chunks over the paged 8-bit cache: kv8_decode() for many new rows a sequence, without
    a tree.  New row i of sequence b sees the keys before the chunk and the chunk's first i + 1, which
    kv8_append() has put into the cache.  q, g: [T,Hq,256] bf16 or fp16; kv_lens int32 [B] counts the
    new rows; cu_rows int32 [B+1].  workspace: kv8_prefill_workspace_size() bytes (about 40 MB).  Up
    to a hundred packed rows (new rows x Hq / Hkv) a sequence kv8_decode() is faster, from some 500 on this.
    Returns out [T,Hq,256]; rows behind cu_rows[B] are left as they were in a given out."""
    sfx = _elem(q, "q")
    d, N, Hkv, bs, *pools = _kv8_pools(k_pool, v_pool, k_scale, v_scale)
    if q.dim() != 3 or q.shape[2] != HEAD_DIM:
        raise ValueError(f"q must be [T, Hq, {HEAD_DIM}], got {tuple(q.shape)}")
    T, Hq, _ = shape = q.shape
    _cuda_index(kv_lens, "kv_lens")
    B = kv_lens.numel()
    tables, max_blocks = _tables(block_tables, B, d)
    if max_kv_len is None:           # synchronises; pass it to avoid the copy
        max_kv_len = max(1, int(kv_lens.max().item()))
    if max_rows is None:
        max_rows = max(1, int((cu_rows[1:] - cu_rows[:-1]).max().item()))
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:    # (a given workspace is checked by the library itself)
        with torch.cuda.device(d):
            need = kv8_prefill_workspace_size()
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    elif workspace.get_device() != d or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{d}")
    lse = torch.empty((T, Hq), dtype=_F32, device=q.device) if return_lse else None
    dt = q.dtype
    _call("gqa_kv8_prefill" + sfx, d, _at(q, dt, shape, d, "q"), *pools,
          None if g is None else _at(g, dt, shape, d, "g"), tables,
          _at(kv_lens, _I32, (B,), d, "kv_lens"), _at(cu_rows, _I32, (B + 1,), d, "cu_rows"),
          _at(out, dt, shape, d, "out"), None if lse is None else lse.data_ptr(), B, T, Hq, Hkv, N,
          bs, max_blocks, int(max_rows), int(max_kv_len), workspace.data_ptr(),
          workspace.numel() * workspace.element_size())
    return (out, lse) if return_lse else out


def decode_split(q, k_cache, v_cache, kv_lens, cu_rows=None, max_rows=None, max_kv_len=None,
                 num_splits=None, split_keys=None, o_parts=None, lse_parts=None):
    """First half of decode: partial results (O/l [S,T*Hq,256] fp32, lse [S,T*Hq]).
    bf16 or fp16 inputs.  split_keys=0 selects balanced shares with num_splits part
    slots (the one-call decode's form on the mma.sync path)."""
    sfx = _elem(q, "q")
    _need(q, q.dtype, 3, "q")
    _need(k_cache, q.dtype, 4, "k_cache")
    _need(v_cache, q.dtype, 4, "v_cache")
    T, Hq, B, Hkv, Lcap, max_rows, max_kv_len = _decode_sizes(q, k_cache, kv_lens, cu_rows,
                                                               max_rows, max_kv_len)
    if num_splits is None or split_keys is None:
        num_splits, split_keys = decode_plan(B, T, Hq, Hkv, max_rows, max_kv_len)
    if o_parts is None:
        o_parts = torch.empty((num_splits, T * Hq, HEAD_DIM), dtype=torch.float32, device=q.device)
    if lse_parts is None:
        lse_parts = torch.empty((num_splits, T * Hq), dtype=torch.float32, device=q.device)
    fn = getattr(load(), "gqa_attn_decode_split" + sfx)
    code = fn(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(kv_lens), _ptr(cu_rows), _ptr(o_parts),
              _ptr(lse_parts), B, T, Hq, Hkv, Lcap, max_rows, max_kv_len, num_splits, split_keys,
              _stream())
    check(code, "gqa_attn_decode_split" + sfx)
    return o_parts, lse_parts


def lse_merge(o_parts, lse_parts, g=None, out=None, return_lse=False, dtype=None):
    """Merge S partial results: o_parts [S,N,256] fp32, lse_parts [S,N] fp32,
    g None or [N,256] (any shape with N*256 elements).  Returns out [N,256] in the
    element type `dtype` (bf16 or fp16; default: that of g, else of out, else bf16)."""
    if o_parts.dtype != torch.float32 or lse_parts.dtype != torch.float32:
        raise TypeError("o_parts and lse_parts must be float32")
    if not (o_parts.is_cuda and o_parts.is_contiguous() and lse_parts.is_contiguous()):
        raise ValueError("o_parts and lse_parts must be contiguous CUDA tensors")
    S, N, D = o_parts.shape
    if D != HEAD_DIM or tuple(lse_parts.shape) != (S, N):
        raise ValueError("shapes must be [S,N,256] and [S,N]")
    if dtype is None:
        dtype = g.dtype if g is not None else out.dtype if out is not None else torch.bfloat16
    if dtype not in _ELEM:
        raise TypeError(f"dtype must be bfloat16 or float16, got {dtype}")
    sfx = _ELEM[dtype]
    if g is not None and (g.dtype != dtype or g.numel() != N * HEAD_DIM
                          or not g.is_contiguous()):
        raise ValueError(f"g must be contiguous {dtype} with N*256 elements")
    if out is None:
        out = torch.empty((N, HEAD_DIM), dtype=dtype, device=o_parts.device)
    if out.dtype != dtype or out.numel() != N * HEAD_DIM or not out.is_contiguous():
        raise ValueError(f"out must be contiguous {dtype} with N*256 elements")
    lse = torch.empty(N, dtype=torch.float32, device=o_parts.device) if return_lse else None
    fn = getattr(load(), "attn_lse_merge" + sfx)
    code = fn(_ptr(o_parts), _ptr(lse_parts), S, N, _ptr(g), _ptr(out), _ptr(lse), _stream())
    check(code, "attn_lse_merge" + sfx)
    return (out, lse) if return_lse else out


def last_device_status():
    """Synchronises the current stream; returns and clears the device status code."""
    return load().gqa_last_device_status(_stream())


def set_wait_timeout_ns(ns):
    load().gqa_set_wait_timeout_ns(int(ns))


def selftest_wait_timeout():
    """Runs the kernels' bounded wait on a barrier nothing completes.  Returns
    (device status, nanoseconds the wait took); the status should be
    GQA_ERR_TIMEOUT (4) and the time about the configured bound."""
    el = torch.zeros(1, dtype=torch.int64, device="cuda")
    check(load().gqa_selftest_wait_timeout(_ptr(el), _stream()), "gqa_selftest_wait_timeout")
    st = last_device_status()
    return st, int(el.item())
