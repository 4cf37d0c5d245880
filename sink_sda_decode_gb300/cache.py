"""Operators that fill a paged cache, and attend over one held in 8 bits.

The cache's geometry is paged.py's: position j of sequence b lies in pool row

    base + block_table[b, j // k_per_block] * k_per_block + j % k_per_block

and kv_len[b] counts the new tokens' own rows, the last m_b of the sequence.  In 8 bits a
row is its E4M3 codes times the scale of its block, block_scale[block_table[b, j //
k_per_block]]: one scale for each block, as all heads share the cached rows.

Streams are as in paged.py.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib, _memory
from .paged import _int32, _need, _nothing_to_do, _on, _stream_of, _workspace_bytes


def _codes(t: torch.Tensor) -> torch.Tensor:
    return t.view(torch.uint8) if getattr(t, "dtype", None) is torch.float8_e4m3fn else t


def _need_scales(block_scale, pages: int, base: int, k_per_block: int, dev) -> None:
    _need(block_scale, "block_scale", torch.float32, 1, dev)
    if block_scale.numel() < -(-(pages - base) // k_per_block):
        raise ValueError("block_scale must have an entry for each block of the pool from base on")


def append_rows(kv: torch.Tensor, cos_cache: torch.Tensor, sin_cache: torch.Tensor,
                block_table: torch.Tensor, q_indptr: torch.Tensor, kv_len: torch.Tensor, *,
                k_per_block: int, base: int = 0, kv_norm_w: torch.Tensor | None = None,
                q: torch.Tensor | None = None, q_norm_w: torch.Tensor | None = None,
                eps: float = 1e-6, unified_kv: torch.Tensor | None = None,
                kv_fp8: torch.Tensor | None = None, block_scale: torch.Tensor | None = None,
                q_out: torch.Tensor | None = None, status: torch.Tensor | None = None,
                stream: torch.cuda.Stream | None = None):
    """The new tokens' rows into a paged cache, normed and rotated on the way, with
    their queries: the step in front of chunk_attention() or chunk_attention_fp8().

    kv [T, D] bf16, the sequences' new rows one after the other (q_indptr [B + 1]);
    kv_len [B] cached positions, these rows included; cos_cache, sin_cache [max_pos, half]
    fp32: the last 2 * half dimensions are rotated, adjacent pairs together, by the row's
    position (half = 0: none).  kv_norm_w, q_norm_w [D] bf16: RMSNorm weights (None: no
    norm).  q [T, H, D] bf16 (None: rows alone) gets the same norm and rotation into q_out
    (may be q).  The rows go to unified_kv [P, D] bf16, or to kv_fp8 [P, D] (float8_e4m3fn,
    or uint8 with the codes) and block_scale, which has an entry for each block: a block's
    scale is the least power of two that its rows need; where new rows need a larger one
    the codes that are there are rounded to it.  Returns (q_out or None, status [1]
    int32: bits 1 a token without a position in the caches, 2 a table entry outside the
    pool, 4 lengths outside the contract: such a sequence is left out, and where q_indptr
    descends others may be, too).

    D a multiple of 16 up to 1024, half one of 4 up to D / 2.  A block that is written
    belongs to one sequence.
    Asynchronous on `stream`; with q_out and status given the call allocates nothing and
    can be captured into a CUDA graph.
    """
    lib = _lib.load()
    _need(kv, "kv", torch.bfloat16, 2)
    dev = kv.device
    T, D = kv.shape
    _need(block_table, "block_table", torch.int32, 2, dev)
    _need(q_indptr, "q_indptr", torch.int32, 1, dev)
    _need(kv_len, "kv_len", torch.int32, 1, dev)
    _need(cos_cache, "cos_cache", torch.float32, 2, dev)
    _need(sin_cache, "sin_cache", torch.float32, 2, dev)
    B = kv_len.numel()
    tables, max_blocks = block_table.shape
    if tables != B or q_indptr.numel() != B + 1:
        raise ValueError("block_table must have a row and q_indptr an interval per entry of kv_len")
    angles = cos_cache.shape
    if angles != sin_cache.shape:
        raise ValueError("cos_cache and sin_cache must have the same shape")
    max_pos, half = angles
    if half % 4 or 2 * half > D:
        raise ValueError("cos_cache must have a multiple of 4 columns, at most D / 2")
    if (unified_kv is None) == (kv_fp8 is None):
        raise ValueError("pass exactly one of unified_kv (bf16 pool) or kv_fp8 + block_scale")
    K, base = _int32(k_per_block, "k_per_block", 1), int(base)
    if unified_kv is not None:
        pool = unified_kv
        _need(pool, "unified_kv", torch.bfloat16, 2, dev)
    else:
        pool = _codes(kv_fp8)
        _need(pool, "kv_fp8", torch.uint8, 2, dev)
        _need_scales(block_scale, pool.shape[0], base, K, dev)
    pages, width = pool.shape
    if width != D:
        raise ValueError("pool rows must have kv's length")
    for name, w in (("kv_norm_w", kv_norm_w), ("q_norm_w", q_norm_w)):
        if w is not None:
            _need(w, name, torch.bfloat16, 1, dev)
            if w.numel() != D:
                raise ValueError(f"{name} must have D entries")
    H = 0
    if q is None:
        if q_norm_w is not None or q_out is not None:
            raise ValueError("q_norm_w and q_out go with q")
    else:
        _need(q, "q", torch.bfloat16, 3, dev)
        shape = q.shape
        H = shape[1]
        if shape[0] != T or shape[2] != D:
            raise ValueError("q must be [T, H, D] with kv [T, D]")
        if q_out is None:
            q_out = _memory.empty(shape, torch.bfloat16, dev, stream)
        else:
            _need(q_out, "q_out", torch.bfloat16, 3, dev)
            if q_out.shape != shape:
                raise ValueError("q_out must have q's shape")
    if status is None:
        status = _memory.empty(1, torch.int32, dev, stream)
    else:
        _need(status, "status", torch.int32, 1, dev)
        if status.numel() < 1:
            raise ValueError("status must hold one int32")
    args = (None if q is None else q.data_ptr(), kv.data_ptr(),
            None if q_norm_w is None else q_norm_w.data_ptr(),
            None if kv_norm_w is None else kv_norm_w.data_ptr(),
            cos_cache.data_ptr() if half else None, sin_cache.data_ptr() if half else None, max_pos,
            block_table.data_ptr(), max_blocks, K, base, q_indptr.data_ptr(),
            kv_len.data_ptr(), B, T, H, D, 2 * half, float(eps), pages,
            None if q is None else q_out.data_ptr(), pool.data_ptr())
    with _on(dev):
        if unified_kv is not None:
            rc = lib.sda_append_rows(*args, status.data_ptr(), _stream_of(dev, stream))
        else:
            rc = lib.sda_append_rows_fp8(*args, block_scale.data_ptr(), status.data_ptr(),
                                         _stream_of(dev, stream))
    _lib.check(rc, "sda_append_rows")
    return q_out, status


def chunk_attention_fp8_workspace_size(B: int, T: int, H: int, D: int, max_blocks: int = 0,
                                       k_per_block: int = 1) -> int:
    """Bytes of workspace for chunk_attention_fp8() on the current CUDA device, for B
    sequences and T tokens in all and tables of max_blocks blocks.  Without max_blocks: the
    least that a call takes, with which long prompts are slower."""
    lib = _lib.load()
    n = ctypes.c_size_t(0)
    _lib.check(lib.sda_chunk_attention_fp8_workspace_size(
        _int32(B, "B"), _int32(T, "T"), _int32(H, "H"), _int32(D, "D"), _int32(max_blocks, "max_blocks"),
        _int32(k_per_block, "k_per_block", 1), ctypes.byref(n)), "sda_chunk_attention_fp8_workspace_size")
    return int(n.value)


def chunk_attention_fp8(q: torch.Tensor, kv_fp8: torch.Tensor, block_scale: torch.Tensor,
                        block_table: torch.Tensor, q_indptr: torch.Tensor, kv_len: torch.Tensor,
                        attn_sink: torch.Tensor, softmax_scale: float, *, k_per_block: int,
                        base: int = 0, window: int = 0, first: int = 0,
                        out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                        workspace: torch.Tensor | None = None,
                        stream: torch.cuda.Stream | None = None):
    """chunk_attention() over a cache of E4M3 codes with one scale for each block.

    kv_fp8 [P, D] float8_e4m3fn (or uint8 with the codes) and block_scale [blocks] fp32 as
    append_rows() fills them; the other arguments, results, the workspace
    (chunk_attention_fp8_workspace_size(...) bytes) and its error word (paged_error_flag())
    as chunk_attention().  Codes are exact, whatever the scales.  Long prompts lay the cached
    rows side by side in the workspace: a call without one allocates 2 D + 5 bytes for each
    position of block_table (at most 2 GB), one with the least that is taken is slower.
    """
    lib = _lib.load()
    _need(q, "q", torch.bfloat16, 3)
    dev = q.device
    codes = _codes(kv_fp8)
    _need(codes, "kv_fp8", torch.uint8, 2, dev)
    _need(block_table, "block_table", torch.int32, 2, dev)
    _need(q_indptr, "q_indptr", torch.int32, 1, dev)
    _need(kv_len, "kv_len", torch.int32, 1, dev)
    _need(attn_sink, "attn_sink", torch.float32, 1, dev)
    T, H, D = q.shape
    B = kv_len.numel()
    K, base = _int32(k_per_block, "k_per_block", 1), int(base)
    if codes.shape[1] != D:
        raise ValueError("kv_fp8 row length must equal q's head dim")
    if block_table.shape[0] != B or q_indptr.numel() != B + 1:
        raise ValueError("block_table must have a row and q_indptr an interval per entry of kv_len")
    _need_scales(block_scale, codes.shape[0], base, K, dev)
    if attn_sink.numel() != H:
        raise ValueError("attn_sink must have H entries")
    if out is None:
        out = _memory.empty(q.shape, q.dtype, dev, stream)
    else:
        _need(out, "out", torch.bfloat16, 3, dev)
        if out.shape != q.shape:
            raise ValueError("out must have q's shape")
    if lse is None:
        lse = _memory.empty((T, H), torch.float32, dev, stream)
    else:
        _need(lse, "lse", torch.float32, 2, dev)
        if lse.shape != (T, H):
            raise ValueError("lse must be [T, H]")
    with _on(dev):
        if workspace is None:
            workspace = _memory.workspace(
                _workspace_bytes(dev.index, chunk_attention_fp8_workspace_size, B, T, H, D,
                                 block_table.shape[1], K), dev, stream)
        else:
            _need(workspace, "workspace", torch.uint8, 1, dev)
        rc = lib.sda_chunk_attention_fp8(
            q.data_ptr(), codes.data_ptr(), block_scale.data_ptr(), codes.shape[0],
            block_table.data_ptr(), block_table.shape[1], K, base, q_indptr.data_ptr(),
            kv_len.data_ptr(), attn_sink.data_ptr(), float(softmax_scale), _int32(window, "window"),
            _int32(first, "first"), B, T, H, D, out.data_ptr(), lse.data_ptr(), workspace.data_ptr(),
            workspace.numel(), _stream_of(dev, stream))
        if B == 0 or T == 0:
            _nothing_to_do(workspace, stream)
    _lib.check(rc, "sda_chunk_attention_fp8")
    return out, lse
