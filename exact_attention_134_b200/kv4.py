"""The paged 4-bit key/value cache and attention over it.

    pool = kv4_alloc(num_pages, Hkv, d, page_size)               # uint8, one layer
    kv4_append(k, v, pool, page_table, seq_lens)                 # new tokens in
    o, lse = attn_fwd_kv4(q, pool, page_table, seq_lens, causal=True)        # decoding
    k, v = kv4_gather(pool, page_table, seq_lens, total, cu)     # a prompt's chunk: bf16 for attn_fwd_varlen

Keys and values are held in pages of page_size tokens, 5 bits a value: a bf16
minimum and scale and 4-bit codes for every token, kv head and 32 channels
(include/attn.h has the definition, csrc/kv4_format.cuh the layout). page_table
(int32 [num_seqs, max_pages]) says in which page token j of sequence s is:
page_table[s, j // page_size]. seq_lens (int32 [num_seqs]) counts the tokens in
the cache, those of the call included: a call's rows are its sequences' last
tokens. kv4_pages.KV4Pages keeps the table on the host.

A page id outside the pool is not followed: get_status() then reports
ATTN_ERR_INVALID_ARG with where = 0x500 (attention), 0x510 (append), 0x520
(gather) or 0x530 (copy).
"""
from __future__ import annotations

import math

from . import _call, _changed, _check_scratch, lib


def kv4_page_bytes(Hkv: int, d: int, page_size: int) -> int:
    """Bytes of a page in one layer; 0 for sizes that the cache does not have."""
    return int(lib().attn_kv4_page_bytes(int(Hkv), int(d), int(page_size)))


def kv4_alloc(num_pages: int, Hkv: int, d: int, page_size: int, num_layers: int | None = None, device="cuda"):
    """A pool of pages: uint8 [num_pages, Hkv, page_size // 16, 20 d], with
    num_layers a leading axis of layers (pool[i] is layer i's pool). Its contents
    need no initial value."""
    import torch
    if kv4_page_bytes(Hkv, d, page_size) == 0:
        raise ValueError("page_size must be a power of two from 16 to 1024 and d 64, 96, 128 or 256")
    shape = (num_pages, Hkv, page_size // 16, 20 * d)
    return torch.empty(shape if num_layers is None else (num_layers, *shape), dtype=torch.uint8, device=device)


def _cache_args(pool, page_table, seq_lens, cu_seqlens, d=None):
    """(num_seqs, max_pages, num_pages, page_size, Hkv, d, device index) after the checks that all calls share."""
    import torch
    index = pool.get_device()
    shape = pool.shape
    if pool.dtype is not torch.uint8 or index < 0 or len(shape) != 4 or shape[3] % 20 or not pool.is_contiguous():
        raise ValueError("pool must be a contiguous uint8 CUDA tensor [num_pages, Hkv, page_size / 16, 20 d]")
    i32 = torch.int32
    if page_table.dtype is not i32 or page_table.get_device() != index or page_table.dim() != 2 or \
            not page_table.is_contiguous():
        raise ValueError("page_table must be a contiguous int32 CUDA tensor [num_seqs, max_pages] on the pool's device")
    if seq_lens.dtype is not i32 or seq_lens.get_device() != index or seq_lens.dim() != 1 or not seq_lens.is_contiguous():
        raise ValueError("seq_lens must be a contiguous int32 CUDA vector on the pool's device")
    if cu_seqlens is not None and (cu_seqlens.dtype is not i32 or cu_seqlens.get_device() != index or
                                   cu_seqlens.dim() != 1 or not cu_seqlens.is_contiguous()):
        raise ValueError("cu_seqlens must be a contiguous int32 CUDA vector on the pool's device")
    num_pages, Hkv, tiles, record = shape
    n, max_pages = page_table.shape
    if seq_lens.shape[0] != n:
        raise ValueError("page_table and seq_lens must hold the same sequences")
    if cu_seqlens is not None and cu_seqlens.shape[0] != n + 1:
        raise ValueError("cu_seqlens must hold num_seqs + 1 offsets")
    if d is not None and record != 20 * d:
        raise ValueError(f"the pool holds records of d = {record // 20}, not {d}")
    return n, max_pages, num_pages, 16 * tiles, Hkv, record // 20, index


def _ptr(t):
    return None if t is None else t.data_ptr()


def kv4_append(k, v, pool, page_table, seq_lens, cu_seqlens=None):
    """Writes new tokens into the cache.

    k, v: bf16 cuda [total, Hkv, d], any strides that are multiples of 8 elements,
    channels contiguous. Sequence s's rows are cu_seqlens[s] .. cu_seqlens[s + 1]
    - 1 (int32 cuda [num_seqs + 1]; None: total / num_seqs each), its last tokens
    of seq_lens[s]. A page shared by several sequences is copied before one of
    them appends to it (KV4Pages.extend names the copies)."""
    import torch
    shape = k.shape
    if len(shape) != 3 or v.shape != shape:
        raise ValueError(f"k and v must both be [total, Hkv, d], not {tuple(shape)} and {tuple(v.shape)}")
    total, Hkv, d = shape
    n, max_pages, num_pages, page_size, pool_heads, _, index = _cache_args(pool, page_table, seq_lens, cu_seqlens, d)
    if Hkv != pool_heads:
        raise ValueError(f"the pool holds {pool_heads} kv heads, not {Hkv}")
    sk, sv, bf16 = k.stride(), v.stride(), torch.bfloat16
    if k.dtype is not bf16 or v.dtype is not bf16 or k.get_device() != index or v.get_device() != index or \
            ((sk[2] != 1 or sv[2] != 1) and d > 1):
        raise ValueError("k and v must be bf16 CUDA tensors with contiguous channels on the pool's device")
    # the stride of an axis of one is never used: torch leaves anything there
    strides = (sk[0] if total > 1 else 0, sk[1] if Hkv > 1 else 0, sv[0] if total > 1 else 0, sv[1] if Hkv > 1 else 0)
    _call("attn_kv4_append", index, k.data_ptr(), v.data_ptr(), *strides, pool.data_ptr(), page_table.data_ptr(),
          seq_lens.data_ptr(), _ptr(cu_seqlens), n, max_pages, num_pages, page_size, total, Hkv, d)
    _changed(pool)


def kv4_gather(pool, page_table, seq_lens, total: int, cu_seqlens=None, k=None, v=None):
    """Reads tokens back as bf16 [total, Hkv, d] each: the last cu_seqlens[s + 1] -
    cu_seqlens[s] tokens of every sequence (None: total / num_seqs), packed as
    attn_fwd_varlen takes them. Rows that no sequence owns are left as they were.
    Returns (k, v)."""
    import torch
    n, max_pages, num_pages, page_size, Hkv, d, index = _cache_args(pool, page_table, seq_lens, cu_seqlens)
    shape = (int(total), Hkv, d)
    for name, t in (("k", k), ("v", v)):
        if t is not None and (t.dtype is not torch.bfloat16 or t.get_device() != index or t.shape != shape or
                              not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous bf16 CUDA tensor {shape} on the pool's device")
    given = k, v
    k = pool.new_empty(shape, dtype=torch.bfloat16) if k is None else k
    v = torch.empty_like(k) if v is None else v
    _call("attn_kv4_gather", index, pool.data_ptr(), page_table.data_ptr(), seq_lens.data_ptr(), _ptr(cu_seqlens), n,
          max_pages, num_pages, page_size, shape[0], Hkv, d, k.data_ptr(), v.data_ptr())
    _changed(*given)
    return k, v


def kv4_copy_pages(pool, src, dst):
    """Copies pages within the pool, in every layer: page dst[i] = page src[i].

    pool: [num_pages, ...] of one layer (4-D) or [num_layers, num_pages, ...]
    (5-D). src, dst: int32 cuda vectors; no dst may be another pair's dst or src."""
    import torch
    index, shape = pool.get_device(), pool.shape
    if pool.dtype is not torch.uint8 or index < 0 or len(shape) not in (4, 5) or not pool.is_contiguous():
        raise ValueError("pool must be a contiguous uint8 CUDA tensor of 4 dimensions, or 5 with layers")
    for name, t in (("src", src), ("dst", dst)):
        if t.dtype is not torch.int32 or t.get_device() != index or t.dim() != 1 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous int32 CUDA vector on the pool's device")
    n = src.shape[0]
    if dst.shape[0] != n:
        raise ValueError("src and dst must have the same length")
    layers, num_pages, H, tiles, record = shape if len(shape) == 5 else (1, *shape)
    _call("attn_kv4_copy_pages", index, pool.data_ptr(), layers, num_pages, H * tiles * record, src.data_ptr(),
          dst.data_ptr(), n)
    _changed(pool)


def fwd_kv4_workspace_size(Hq: int, Hkv: int, max_seqlen_q: int, d: int) -> int:
    """Bytes of scratch that attn_fwd_kv4 needs (5 MB at most; any number of sequences)."""
    return int(lib().attn_fwd_kv4_workspace_size(Hq, Hkv, int(max_seqlen_q), d))


def attn_fwd_kv4(q, pool, page_table, seq_lens, cu_seqlens_q=None, max_seqlen_q: int | None = None,
                 causal: bool = False, scale: float | None = None, workspace=None, out=None, lse=None):
    """Attention of a few query tokens a sequence over the 4-bit cache (decoding;
    drafted tokens checked together).

    q: bf16 cuda [total_q, Hq, d], sequence s's rows cu_seqlens_q[s] ..
    cu_seqlens_q[s + 1] - 1 (None: total_q / num_seqs each), standing at its last
    tokens: with causal, row i of n sees tokens 0 .. seq_lens[s] - n + i.
    max_seqlen_q: the longest sequence's query rows (a bound of them chooses the
    kernel; total_q / num_seqs, rounded up, when not given). workspace: a uint8
    cuda buffer of fwd_kv4_workspace_size(Hq, Hkv, max_seqlen_q, d) bytes, one
    for each call that may run at the same time (allocated here if None and the
    table holds more than 512 tokens a sequence, which need it).
    Returns (o bf16 [total_q, Hq, d], lse fp32 [Hq, total_q]); a row that sees no
    token gets o = 0 and lse = -inf.
    """
    import torch
    shape = q.shape
    if q.dtype is not torch.bfloat16 or len(shape) != 3 or q.get_device() != pool.get_device() or not q.is_contiguous():
        raise ValueError("q must be a contiguous bf16 CUDA tensor [total, H, d] on the pool's device")
    total, Hq, d = shape
    n, max_pages, num_pages, page_size, Hkv, _, index = _cache_args(pool, page_table, seq_lens, cu_seqlens_q, d)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if max_seqlen_q is None:
        max_seqlen_q = -(-total // max(n, 1))
    given = out, lse
    if out is None:
        out = torch.empty_like(q)
    elif out.dtype is not torch.bfloat16 or out.get_device() != index or out.shape != shape or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous bf16 CUDA tensor {tuple(shape)} on the device of q")
    if lse is None:
        lse = q.new_empty((Hq, total), dtype=torch.float32)
    elif lse.dtype is not torch.float32 or lse.get_device() != index or lse.shape != (Hq, total) or \
            not lse.is_contiguous():
        raise ValueError(f"lse must be a contiguous fp32 CUDA tensor {(Hq, total)} on the device of q")
    if workspace is None and max_pages * page_size > 512:  # shorter caches leave no partial results
        workspace = lse.new_empty((fwd_kv4_workspace_size(Hq, Hkv, max_seqlen_q, d) // 4,))
    else:
        _check_scratch("workspace", workspace, index)
    _call("attn_fwd_kv4", index, q.data_ptr(), pool.data_ptr(), page_table.data_ptr(), seq_lens.data_ptr(),
          _ptr(cu_seqlens_q), out.data_ptr(), lse.data_ptr(), n, max_pages, num_pages, page_size, int(max_seqlen_q),
          total, Hq, Hkv, d, 1 if causal else 0, float(scale), _ptr(workspace),
          0 if workspace is None else workspace.nbytes)
    _changed(*given)
    return out, lse
