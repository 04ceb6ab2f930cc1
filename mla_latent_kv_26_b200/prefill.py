"""Torch-facing prefill: attention of a chunk of new tokens over the paged
latent cache, in three library calls (``include/mla_prefill.h``).

* :func:`cache_read`        — cached rows back from the paged cache (bf16 or fp8)
* :func:`expand_kv`         — their per-head keys and values
* :func:`prefill_attention` — ragged attention of the new tokens over them
* :class:`MlaPrefill`       — the three with their buffers, for one capacity

The wrappers check dtypes, shapes and devices and pass raw pointers; all
arithmetic happens in libmla's kernels. Offsets and lengths stay on the
device, nothing synchronises, and a captured CUDA graph replays with other
lengths within the same capacities.

Sequence b's new tokens are rows ``[cu_q[b], cu_q[b + 1])`` of ``q`` and its
keys rows ``[cu_k[b], cu_k[b + 1])`` of ``kv``: all its tokens, the new ones
last (insert them into the cache first). For a few new tokens per sequence
(fewer than about 170) :class:`~mla_latent_kv_26_b200.decoder.MlaDecoder` with
a causal descriptor does less work.
"""

from __future__ import annotations

from typing import Optional, Tuple

import torch

from . import binding as B


def _check(name, t, dtype, shape, dev):
    if not isinstance(t, torch.Tensor) or t.device != dev or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name}: need a contiguous {dtype} tensor on {dev}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)} != {tuple(shape)}")


def _device(name, t):
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise ValueError(f"{name}: need a CUDA tensor")
    return t.device


def _row_stride(name, t, dev, width, exact):
    """Elements between the rows of a bf16 matrix whose rows are dense."""
    if t.device != dev or t.dtype != torch.bfloat16 or t.dim() != 2:
        raise ValueError(f"{name}: need a two-dimensional bfloat16 tensor on {dev}")
    if t.shape[1] != width if exact else t.shape[1] < width:
        raise ValueError(f"{name}: rows of {t.shape[1]} values, {'' if exact else 'at least '}{width} needed")
    if t.shape[0] <= 1:
        stride = (t.shape[1] + 7) // 8 * 8  # the stride of a single row is never used
    else:
        stride = t.stride(0)
    if (t.numel() and t.stride(1) != 1) or stride < width or stride % 8 or t.data_ptr() % 16:
        raise ValueError(f"{name}: rows must be dense, 16-byte aligned and a multiple of 8 elements apart")
    return stride


def _error_word(error_word, dev):
    if error_word is not None and (error_word.device != dev or error_word.dtype != torch.int32
                                   or error_word.numel() < 1):
        raise ValueError(f"error_word: need an int32 tensor on {dev}")


def _stream(stream, dev):
    return torch.cuda.current_stream(dev) if stream is None else stream


def cache_read(kv_cache: torch.Tensor, block_table: torch.Tensor, row_offsets: torch.Tensor, *,
               starts: Optional[torch.Tensor] = None, num_rows: Optional[int] = None,
               out: Optional[torch.Tensor] = None, error_word: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """Row ``row_offsets[b] + j`` of the result is the cache row of position
    ``starts[b] + j`` of sequence b (``starts`` None: 0), as 576 bf16 values.

    ``kv_cache``: bf16 [pages, 64, 576], or uint8 [pages, 64, 656] for an fp8
    latent cache; ``block_table`` int32 [batch, max_pages]; ``row_offsets``
    int32 [batch + 1]. ``out`` [rows, 576] bf16, or ``num_rows`` of it to
    allocate. Rows that no sequence owns are left as they were; a position
    without a page gives a row of zeros and a bit in ``error_word``."""
    dev = _device("kv_cache", kv_cache)
    fp8 = kv_cache.dtype == torch.uint8
    _check("kv_cache", kv_cache, torch.uint8 if fp8 else torch.bfloat16, None, dev)
    _check("block_table", block_table, torch.int32, None, dev)
    if kv_cache.dim() != 3 or tuple(kv_cache.shape[1:]) != (64, 656 if fp8 else 576) or block_table.dim() != 2:
        raise ValueError("kv_cache must be [pages, 64, 576] bf16 or [pages, 64, 656] uint8, "
                         "block_table [batch, max_pages_per_seq]")
    batch = block_table.shape[0]
    _check("row_offsets", row_offsets, torch.int32, (batch + 1,), dev)
    if starts is not None:
        _check("starts", starts, torch.int32, (batch,), dev)
    _error_word(error_word, dev)
    if out is None:
        if num_rows is None:
            raise ValueError("cache_read needs out or num_rows")
        out = torch.empty(num_rows, 576, dtype=torch.bfloat16, device=dev)
    _check("out", out, torch.bfloat16, (out.shape[0], 576), dev)
    desc = B.make_read_desc(batch=batch, max_pages_per_seq=max(block_table.shape[1], 1),
                            num_pages=max(kv_cache.shape[0], 1), num_rows=out.shape[0])
    if batch and out.shape[0] and (kv_cache.shape[0] == 0 or block_table.shape[1] == 0):
        raise ValueError("cache_read: rows asked of an empty cache or block table")
    with torch.cuda.device(dev):
        fn = B.mlap_cache_read_fp8 if fp8 else B.mlap_cache_read
        B.check(fn(desc, kv_cache, block_table, row_offsets, starts, out, error_word, _stream(stream, dev)),
                "mlap_cache_read")
    return out


def expand_kv(rows: torch.Tensor, wkv_b: torch.Tensor, *, out: Optional[torch.Tensor] = None,
              row_count: Optional[torch.Tensor] = None, error_word: Optional[torch.Tensor] = None,
              stream=None) -> torch.Tensor:
    """``kv[t, h] = wkv_b[h] @ rows[t, :512]``: [rows, H, 256], the no-rope key
    (128) and the value (128) of every head. ``rows`` bf16 [M, 512 or more]
    with any row stride that is a multiple of 8; ``row_count``: optional int32
    tensor on the device, rows from its first value on are neither computed
    nor written."""
    dev = _device("rows", rows)
    stride = _row_stride("rows", rows, dev, 512, False)
    M = rows.shape[0]
    if not isinstance(wkv_b, torch.Tensor) or wkv_b.dim() != 3:
        raise ValueError("wkv_b: need a [heads, 256, 512] tensor")
    H = wkv_b.shape[0]
    _check("wkv_b", wkv_b, torch.bfloat16, (H, 256, 512), dev)
    if row_count is not None and (row_count.device != dev or row_count.dtype != torch.int32 or row_count.numel() < 1):
        raise ValueError(f"row_count: need an int32 tensor on {dev}")
    _error_word(error_word, dev)
    if out is None:
        out = torch.empty(M, H, 256, dtype=torch.bfloat16, device=dev)
    _check("out", out, torch.bfloat16, (M, H, 256), dev)
    with torch.cuda.device(dev):
        B.check(B.mlap_expand_kv(B.make_expand_desc(num_rows=M, num_heads=H, row_stride=stride), rows, wkv_b,
                                 row_count, out, error_word, _stream(stream, dev)), "mlap_expand_kv")
    return out


def attention_workspace_bytes(num_q: int, num_heads: int, num_k: int, *, batch: int = 1, num_sms: int = 0) -> int:
    """Bytes of a workspace for :func:`prefill_attention` on the current device."""
    n = B.mlap_attention_workspace_bytes(B.make_attention_desc(batch=batch, num_heads=num_heads, num_q=num_q,
                                                               num_k=num_k, num_sms=num_sms))
    if n == 0:
        raise B.MlaError(B.MLA_ERR_INVALID_ARG, "descriptor rejected by the sizing query")
    return n


def prefill_attention(q: torch.Tensor, kv: torch.Tensor, k_pe: torch.Tensor, cu_q: torch.Tensor, cu_k: torch.Tensor,
                      *, causal: bool = True, softmax_scale: float = B.DEFAULT_SOFTMAX_SCALE,
                      out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None, num_sms: int = 0,
                      error_word: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Attention of ragged queries ``q`` [Nq, H, 192] over ``kv`` [Nk, H, 256]
    (key 128, value 128) and ``k_pe`` [Nk, 64] (any row stride that is a
    multiple of 8): ``(out [Nq, H, 128] bf16, lse [Nq, H] float32)``.

    ``cu_q``, ``cu_k`` int32 [batch + 1]. Causal: a sequence's queries are its
    last positions; otherwise every query sees every key of its sequence (one
    part of a context, merged with others by :func:`merge_parts`). A row
    without keys gets zeros and -inf; rows that no sequence owns are left as
    they were. ``workspace`` (uint8, :func:`attention_workspace_bytes`) is
    allocated when not given; calls that may run at the same time, and graphs
    that may replay at the same time, need one each."""
    dev = _device("q", q)
    if q.dim() != 3:
        raise ValueError("q: need a [queries, heads, 192] tensor")
    Nq, H = q.shape[0], q.shape[1]
    _check("q", q, torch.bfloat16, (Nq, H, 192), dev)
    Nk = kv.shape[0]
    _check("kv", kv, torch.bfloat16, (Nk, H, 256), dev)
    stride = _row_stride("k_pe", k_pe, dev, 64, True)
    if k_pe.shape[0] != Nk:
        raise ValueError(f"k_pe: {k_pe.shape[0]} rows, kv has {Nk}")
    if cu_q.dim() != 1 or cu_q.shape[0] < 1:
        raise ValueError("cu_q: need batch + 1 offsets")
    _check("cu_q", cu_q, torch.int32, None, dev)
    _check("cu_k", cu_k, torch.int32, tuple(cu_q.shape), dev)
    _error_word(error_word, dev)
    if out is None:
        out = torch.empty(Nq, H, 128, dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty(Nq, H, dtype=torch.float32, device=dev)
    _check("out", out, torch.bfloat16, (Nq, H, 128), dev)
    _check("lse", lse, torch.float32, (Nq, H), dev)
    desc = B.make_attention_desc(batch=cu_q.shape[0] - 1, num_heads=H, num_q=Nq, num_k=Nk, pe_stride=stride,
                                 causal=causal, softmax_scale=softmax_scale, num_sms=num_sms)
    s = _stream(stream, dev)
    with torch.cuda.device(dev):
        if workspace is None:
            n = max(B.mlap_attention_workspace_bytes(desc), 16)
            with torch.cuda.stream(s):
                workspace = torch.empty(n, dtype=torch.uint8, device=dev)
        _check("workspace", workspace, torch.uint8, None, dev)
        B.check(B.mlap_attention(desc, q, kv, k_pe, cu_q, cu_k, out, lse, workspace, workspace.numel(), error_word, s),
                "mlap_attention")
    return out, lse


def merge_parts(part_out: torch.Tensor, part_lse: torch.Tensor, *, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Merge of attention results over disjoint parts of each row's keys:
    ``part_out`` [parts, ..., 128] bf16, ``part_lse`` [parts, ...] float32
    (``mla_merge``)."""
    dev = _device("part_out", part_out)
    _check("part_out", part_out, torch.bfloat16, None, dev)
    _check("part_lse", part_lse, torch.float32, tuple(part_out.shape[:-1]), dev)
    if part_out.dim() < 2 or part_out.shape[-1] != 128:
        raise ValueError("part_out: need [parts, ..., 128]")
    out = torch.empty(part_out.shape[1:], dtype=torch.bfloat16, device=dev)
    lse = torch.empty(part_lse.shape[1:], dtype=torch.float32, device=dev)
    with torch.cuda.device(dev):
        B.check(B.mla_merge(B.make_merge_desc(parts=part_out.shape[0], rows=lse.numel(), d_latent=128), part_out,
                            part_lse, out, lse, _stream(stream, dev)), "mla_merge")
    return out, lse


class MlaPrefill:
    """The prefill of ragged chunks over the paged cache: read back, expand,
    attend. Owns the buffers for up to ``max_queries`` new tokens and
    ``max_keys`` cached tokens (all sequences of a call together; 512 * H + 1152
    bytes per key); a call with more is clipped and sets a bit of ``error_word``."""

    def __init__(self, *, max_queries: int, max_keys: int, num_heads: int,
                 softmax_scale: float = B.DEFAULT_SOFTMAX_SCALE, num_sms: int = 0, device="cuda"):
        dev = torch.device(device)
        if dev.type == "cuda" and dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        self.device = dev
        self.num_heads, self.softmax_scale, self.num_sms = num_heads, softmax_scale, num_sms
        with torch.cuda.device(dev):
            n = attention_workspace_bytes(max_queries, num_heads, max_keys, num_sms=num_sms)
        self.workspace = torch.empty(n, dtype=torch.uint8, device=dev)
        self.rows = torch.zeros(max_keys, 576, dtype=torch.bfloat16, device=dev)
        self.kv = torch.empty(max_keys, num_heads, 256, dtype=torch.bfloat16, device=dev)
        self.out = torch.empty(max_queries, num_heads, 128, dtype=torch.bfloat16, device=dev)
        self.lse = torch.empty(max_queries, num_heads, dtype=torch.float32, device=dev)
        self.error_word = torch.zeros(1, dtype=torch.int32, device=dev)

    def __call__(self, q: torch.Tensor, wkv_b: torch.Tensor, kv_cache: torch.Tensor, block_table: torch.Tensor,
                 cu_q: torch.Tensor, cu_k: torch.Tensor, *, starts: Optional[torch.Tensor] = None,
                 causal: bool = True, stream=None) -> torch.Tensor:
        """``q`` [Nq, H, 192], Nq at most ``max_queries``; sequence b attends to
        its cached positions ``starts[b] .. starts[b] + cu_k[b + 1] - cu_k[b] - 1``
        (``starts`` None: from 0). Returns ``out`` [Nq, H, 128], a view of a
        buffer that the next call overwrites; its log-sum-exp is ``self.lse[:Nq]``."""
        nq = q.shape[0]
        if nq > self.out.shape[0] or q.dim() != 3 or q.shape[1] != self.num_heads:
            raise ValueError(f"q: shape {tuple(q.shape)}, need at most {self.out.shape[0]} queries of "
                             f"{self.num_heads} heads")
        e = self.error_word
        cache_read(kv_cache, block_table, cu_k, starts=starts, out=self.rows, error_word=e, stream=stream)
        expand_kv(self.rows, wkv_b, out=self.kv, row_count=cu_k[-1:], error_word=e, stream=stream)
        out, _ = prefill_attention(q, self.kv, self.rows[:, 512:], cu_q, cu_k, causal=causal,
                                   softmax_scale=self.softmax_scale, out=self.out[:nq], lse=self.lse[:nq],
                                   workspace=self.workspace, num_sms=self.num_sms, error_word=e, stream=stream)
        return out
