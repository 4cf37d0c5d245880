"""Operators on a paged cache: attention of a chunk of new tokens, the weight
that every cached position received, and eviction by that weight.

A sequence's cached positions are found through a block table: position j of
sequence b lies in pool row

    base + block_table[b, j // k_per_block] * k_per_block + j % k_per_block

(`base` is the first pool row of the block region; k_per_block = 1 makes the
table one of single slots).  With m_b new tokens and n_b = kv_len[b] cached
positions, the new tokens' own rows the last m_b of them, token i stands at
p = n_b - m_b + i and sees the positions j <= p with window == 0, or
j > p - window, or j < first.

A call runs on `stream` (None: the current one).  With another stream than the
current one, the caller orders the two, as for any kernel: before the call for
tensors that are written on the current stream, after it for its results.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
from typing import NamedTuple

import torch

from . import _lib, _memory


def _need(t, name: str, dtype, ndim: int, dev=None):
    """_req() with the checks of a good tensor in one expression: these run on
    every step of a decode loop."""
    if not (type(t) is torch.Tensor and t.dtype is dtype and t.dim() == ndim and t.is_cuda
            and t.is_contiguous() and (dev is None or t.device == dev)):
        from . import _req
        _req(t, name, dtype, ndim, dev)


_HERE = contextlib.nullcontext()


def _on(dev):
    """Makes dev the current device, at no cost where it is already."""
    return _HERE if torch.cuda.current_device() == dev.index else torch.cuda.device(dev)


def _stream_of(dev, stream) -> int:
    return (stream.cuda_stream if stream is not None
            else torch._C._cuda_getCurrentRawStream(dev.index))


_HEADER = 256  # bytes of a workspace that say how the last call went


def _nothing_to_do(workspace, stream) -> None:
    """A call without work leaves its workspace alone; its error word is 0 all the same."""
    with torch.cuda.stream(stream) if stream is not None else _HERE:
        workspace[:_HEADER].zero_()


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(device: int, size, *args) -> int:
    """A workspace size depends on the device's SM count and these sizes only."""
    return size(*args)


def _int32(v, name: str, low: int = 0) -> int:
    v = int(v)
    if not low <= v < 2 ** 31:
        raise ValueError(f"{name} must be in [{low}, 2^31), got {v}")
    return v


def _tables(q, unified_kv, block_table, q_indptr, kv_len):
    """Checks the tensors that the paged operators share; returns (B, T, H, D)."""
    _need(q, "q", torch.bfloat16, 3)
    dev = q.device
    _need(unified_kv, "unified_kv", torch.bfloat16, 2, dev)
    _need(block_table, "block_table", torch.int32, 2, dev)
    _need(q_indptr, "q_indptr", torch.int32, 1, dev)
    _need(kv_len, "kv_len", torch.int32, 1, dev)
    T, H, D = q.shape
    B = kv_len.numel()
    if unified_kv.shape[1] != D:
        raise ValueError("unified_kv row length must equal q's head dim")
    if block_table.shape[0] != B or q_indptr.numel() != B + 1:
        raise ValueError("block_table must have a row and q_indptr an interval per entry of kv_len")
    return B, T, H, D


def chunk_attention_workspace_size(B: int, T: int, H: int, D: int) -> int:
    """Bytes of workspace chunk_attention() needs on the current CUDA device
    for B sequences and T tokens in all."""
    lib = _lib.load()
    n = ctypes.c_size_t(0)
    _lib.check(lib.sda_chunk_attention_workspace_size(_int32(B, "B"), _int32(T, "T"), _int32(H, "H"),
                                                      _int32(D, "D"), ctypes.byref(n)),
               "sda_chunk_attention_workspace_size")
    return int(n.value)


def chunk_attention(q: torch.Tensor, unified_kv: torch.Tensor, block_table: torch.Tensor,
                    q_indptr: torch.Tensor, kv_len: torch.Tensor, attn_sink: torch.Tensor,
                    softmax_scale: float, *, k_per_block: int, base: int = 0, window: int = 0,
                    first: int = 0, out: torch.Tensor | None = None,
                    lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                    stream: torch.cuda.Stream | None = None):
    """Causal attention of every sequence's new tokens over its cached positions.

    q [T, H, D] bf16, the sequences' tokens one after the other; unified_kv
    [P, D] bf16 (a row is key and value); block_table [B, max_blocks] int32;
    q_indptr [B + 1] int32 (sequence b's tokens: q_indptr[b] .. q_indptr[b + 1]);
    kv_len [B] int32, cached positions including the new tokens' own; attn_sink
    [H] fp32 sink logits.  Returns (out [T, H, D] bf16, lse [T, H] fp32, the log
    of the softmax denominator, sink included).  A row that sees nothing gets
    out = 0 and lse = the sink; rows outside [q_indptr[0], q_indptr[B]) are not
    written.  H up to 256, D in {64, 128, 256, 512}.  Fast where k_per_block is a
    multiple of 16 and unified_kv holds, from `base` on, a multiple of 8 rows; else
    cached rows are loaded one by one.

    Asynchronous on `stream`.  With out, lse and `workspace` (uint8, at least
    chunk_attention_workspace_size(...) bytes) given the call allocates nothing
    and can be captured into a CUDA graph; calls that may overlap on the GPU
    need a workspace each.  paged_error_flag(workspace) reads its error word
    (2: lengths outside the contract, nothing computed; 3: a table entry
    outside the pool).
    """
    lib = _lib.load()
    B, T, H, D = _tables(q, unified_kv, block_table, q_indptr, kv_len)
    dev = q.device
    _need(attn_sink, "attn_sink", torch.float32, 1, dev)
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
                _workspace_bytes(dev.index, chunk_attention_workspace_size, B, T, H, D), dev, stream)
        else:
            _need(workspace, "workspace", torch.uint8, 1, dev)
        rc = lib.sda_chunk_attention(
            q.data_ptr(), unified_kv.data_ptr(), unified_kv.shape[0], block_table.data_ptr(),
            block_table.shape[1], _int32(k_per_block, "k_per_block", 1), int(base),
            q_indptr.data_ptr(), kv_len.data_ptr(), attn_sink.data_ptr(), float(softmax_scale),
            _int32(window, "window"), _int32(first, "first"), B, T, H, D, out.data_ptr(),
            lse.data_ptr(), workspace.data_ptr(), workspace.numel(), _stream_of(dev, stream))
        if B == 0 or T == 0:
            _nothing_to_do(workspace, stream)
    _lib.check(rc, "sda_chunk_attention")
    return out, lse


def paged_error_flag(workspace: torch.Tensor, stream: torch.cuda.Stream | None = None) -> int:
    """Device error word of the last chunk_attention() or attention_mass() on
    `workspace` (synchronises): 0 = fine; 1 = a pipeline wait timed out; 2 =
    q_indptr or kv_len outside their contract (nothing was computed); 3 = a table
    entry outside the pool (its rows counted as zeros)."""
    lib = _lib.load()
    _need(workspace, "workspace", torch.uint8, 1)
    dev = workspace.device
    with _on(dev):
        if workspace.numel() < _workspace_bytes(dev.index, attention_mass_workspace_size, 0, 0, 1):
            raise ValueError("workspace is smaller than any that a call can have used")
        flag = torch.zeros(1, dtype=torch.int32, device=dev)
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream(dev))
        _lib.check(lib.sda_paged_error_flag(workspace.data_ptr(), flag.data_ptr(),
                                            _stream_of(dev, stream)), "sda_paged_error_flag")
        if stream is not None:
            stream.synchronize()
        return int(flag.item())


def attention_mass_workspace_size(B: int, max_blocks: int, k_per_block: int) -> int:
    """Bytes of workspace attention_mass() needs on the current CUDA device."""
    lib = _lib.load()
    n = ctypes.c_size_t(0)
    _lib.check(lib.sda_attention_mass_workspace_size(_int32(B, "B"), _int32(max_blocks, "max_blocks"),
                                                     _int32(k_per_block, "k_per_block", 1),
                                                     ctypes.byref(n)),
               "sda_attention_mass_workspace_size")
    return int(n.value)


def attention_mass(q: torch.Tensor, unified_kv: torch.Tensor, block_table: torch.Tensor,
                   q_indptr: torch.Tensor, kv_len: torch.Tensor, lse: torch.Tensor,
                   softmax_scale: float, *, k_per_block: int, base: int = 0, window: int = 0,
                   first: int = 0, scores: torch.Tensor | None = None, decay: float = 1.0,
                   out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                   stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """The attention weight every cached position received from the tokens in q.

    The arguments and their meaning are chunk_attention()'s, whose `lse` [T, H]
    this takes.  Returns out [B, S] fp32, S = max_blocks * k_per_block:

        out[b, j] = decay * scores[b, j] + sum of softmax weights of position j
                    over the tokens and heads of sequence b that see it

    for j < kv_len[b] and 0 behind it.  `scores` [B, S] fp32 (None: zeros) may be
    given as `out` too.  To rank positions by the last few tokens only, pass
    those tokens (and their lse): they still stand at the end of the cache.
    All of `out` is written, so a table much wider than its sequences costs its width.
    Deterministic.  Asynchronous on `stream`; with `out` and `workspace` (uint8,
    attention_mass_workspace_size(...) bytes) given, the call can be captured.
    """
    lib = _lib.load()
    B, T, H, D = _tables(q, unified_kv, block_table, q_indptr, kv_len)
    dev = q.device
    S = block_table.shape[1] * _int32(k_per_block, "k_per_block", 1)
    _need(lse, "lse", torch.float32, 2, dev)
    if lse.shape != (T, H):
        raise ValueError("lse must be [T, H]")
    for name, t in (("scores", scores), ("out", out)):
        if t is not None:
            _need(t, name, torch.float32, 2, dev)
            if t.shape != (B, S):
                raise ValueError(f"{name} must be [B, max_blocks * k_per_block]")
    if out is None:
        out = _memory.empty((B, S), torch.float32, dev, stream)
    with _on(dev):
        if workspace is None:
            workspace = _memory.workspace(
                _workspace_bytes(dev.index, attention_mass_workspace_size, B, block_table.shape[1],
                                 k_per_block), dev, stream)
        else:
            _need(workspace, "workspace", torch.uint8, 1, dev)
        rc = lib.sda_attention_mass(
            q.data_ptr(), unified_kv.data_ptr(), unified_kv.shape[0], block_table.data_ptr(),
            block_table.shape[1], int(k_per_block), int(base), q_indptr.data_ptr(),
            kv_len.data_ptr(), lse.data_ptr(), float(softmax_scale), _int32(window, "window"),
            _int32(first, "first"), None if scores is None else scores.data_ptr(), float(decay), B,
            T, H, D, out.data_ptr(), workspace.data_ptr(), workspace.numel(), _stream_of(dev, stream))
        if B == 0 or S == 0:
            _nothing_to_do(workspace, stream)
    _lib.check(rc, "sda_attention_mass")
    return out


class Evicted(NamedTuple):
    """What evict_slots() returns."""
    scores: torch.Tensor        # [B, W] fp32, kept positions' scores, then 0
    slot_table: torch.Tensor    # [B, W] int32, kept positions' slots, then -1
    kv_len: torch.Tensor        # [B] int32
    freed_slots: torch.Tensor   # int32, sequence by sequence, then -1
    freed_indptr: torch.Tensor  # [B + 1] int32
    status: torch.Tensor        # [1] int32: bits 1 (a bad length), 8 (a NaN competed)


def evict_slots(scores: torch.Tensor, slot_table: torch.Tensor, kv_len: torch.Tensor, budget: int, *,
                first: int = 0, recent: int = 0, out: Evicted | None = None,
                stream: torch.cuda.Stream | None = None) -> Evicted:
    """Cut every sequence's cache down to `budget` positions by score.

    scores [B, S] fp32 and slot_table [B, S] int32 (a block table with
    k_per_block = 1), kv_len [B] int32.  A sequence of more than `budget`
    positions keeps its first `first`, its last `recent` and the best-scored
    others, in their order; equal scores keep the lower position, NaN goes
    first.  Returns an Evicted with tables of min(S, budget) columns.  `out`
    (an Evicted of preallocated tensors) keeps the call free of allocations; its
    scores, slot_table and kv_len may be the inputs themselves, which is the
    update in place.  All of them is written, so a table much wider than its
    sequences costs its width.  Asynchronous on `stream`.
    """
    lib = _lib.load()
    _need(scores, "scores", torch.float32, 2)
    dev = scores.device
    _need(slot_table, "slot_table", torch.int32, 2, dev)
    _need(kv_len, "kv_len", torch.int32, 1, dev)
    B, S = scores.shape
    if slot_table.shape != (B, S) or kv_len.numel() != B:
        raise ValueError("scores and slot_table must be [B, S] and kv_len [B]")
    budget = _int32(budget, "budget")
    freed = B * max(S - budget, 0)
    if out is None:
        W = min(S, budget)
        i32 = torch.int32
        out = Evicted(*_memory.empties(dev, stream, ((B, W), torch.float32), ((B, W), i32), (B, i32),
                                       (freed, i32), (B + 1, i32), (1, i32)))
    else:
        _need(out.scores, "out.scores", torch.float32, 2, dev)
        for name in ("slot_table", "kv_len", "freed_slots", "freed_indptr", "status"):
            _need(getattr(out, name), f"out.{name}", torch.int32, 2 if name == "slot_table" else 1, dev)
        if out.scores.shape != out.slot_table.shape or out.scores.shape[0] != B:
            raise ValueError("out.scores and out.slot_table must be [B, W]")
        if out.kv_len.numel() != B or out.freed_indptr.numel() != B + 1 or out.status.numel() != 1:
            raise ValueError("out.kv_len must be [B], out.freed_indptr [B + 1] and out.status [1]")
        if out.scores.shape[1] < min(S, budget) or out.freed_slots.numel() < freed:
            raise ValueError("out's tables need min(S, budget) columns and freed_slots "
                             "B * max(S - budget, 0) entries")
    with _on(dev):
        rc = lib.sda_evict_slots(
            scores.data_ptr(), slot_table.data_ptr(), S, kv_len.data_ptr(), B, budget,
            _int32(first, "first"), _int32(recent, "recent"), out.scores.data_ptr(),
            out.slot_table.data_ptr(), out.scores.shape[1], out.kv_len.data_ptr(),
            out.freed_slots.data_ptr(), out.freed_slots.numel(), out.freed_indptr.data_ptr(),
            out.status.data_ptr(), _stream_of(dev, stream))
    _lib.check(rc, "sda_evict_slots")
    return out
