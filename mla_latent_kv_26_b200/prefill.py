"""Torch-facing prefill: attention of a chunk of new tokens over the paged
latent cache, in three library calls (``include/mla_prefill.h``).

* :func:`cache_read`        — cached rows back from the paged cache (bf16 or fp8)
* :func:`expand_kv`         — their per-head keys and values
* :func:`prefill_attention` — ragged attention of the new tokens over them
* :class:`MlaPrefill`       — the three with their buffers, for one capacity

The wrappers check dtypes, shapes and devices and pass raw pointers; all
arithmetic happens in libmla's kernels. Offsets and lengths stay on the
device, no call synchronises, and a captured CUDA graph replays with other
lengths within the same capacities. ``stream`` (a torch stream or a raw handle;
the current one when not given) is where a call's kernels run and where what it
allocates belongs; inputs made on another stream are the caller's to order and
to keep.

Sequence b's new tokens are rows ``[cu_q[b], cu_q[b + 1])`` of ``q`` and its
keys rows ``[cu_k[b], cu_k[b + 1])`` of ``kv``: all its tokens, the new ones
last (insert them into the cache first). For a few new tokens per sequence
:class:`~mla_latent_kv_26_b200.decoder.MlaDecoder` with a causal descriptor is
faster: with 16 heads below about 10, with 128 heads below 50 (8 sequences of 600
tokens), 90 (one of 4096 or 16384) or 130 (4 of 8192).
"""

from __future__ import annotations

import contextlib
import math
from typing import Optional, Tuple

import torch

from . import binding as B

_BF16, _I32, _U8, _F32 = torch.bfloat16, torch.int32, torch.uint8, torch.float32
_INT_MAX = 0x7fffffff
_HERE = contextlib.nullcontext()


def _check(name, t, dtype, shape, dev):
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.device != dev or not t.is_contiguous():
        raise ValueError(f"{name}: need a contiguous {dtype} tensor on {dev}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)} != {tuple(shape)}")


def _device(name, t):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name}: need a CUDA tensor")
    return t.device


def _row_stride(name, t, dev, width, exact):
    """Elements between the rows of a bf16 matrix whose rows are dense."""
    if not isinstance(t, torch.Tensor) or t.device != dev or t.dtype != _BF16 or t.dim() != 2:
        raise ValueError(f"{name}: need a two-dimensional bfloat16 tensor on {dev}")
    rows, cols = t.shape
    if cols != width if exact else cols < width:
        raise ValueError(f"{name}: rows of {cols} values, {'' if exact else 'at least '}{width} needed")
    s0, s1 = t.stride()
    stride = s0 if rows > 1 else (cols + 7) // 8 * 8  # the stride of a single row is never used
    if (rows and s1 != 1) or stride < width or stride % 8 or stride > _INT_MAX or t.data_ptr() % 16:
        raise ValueError(f"{name}: rows must be dense, 16-byte aligned and a multiple of 8 (below 2^31) elements apart")
    return stride


def _optional_i32(name, t, dev):
    if t is not None and (not isinstance(t, torch.Tensor) or t.device != dev or t.dtype != _I32 or t.numel() < 1):
        raise ValueError(f"{name}: need an int32 tensor on {dev}")


def _on(dev):
    """The device as a context; nothing when it is the current one."""
    return _HERE if torch.cuda.current_device() == dev.index else torch.cuda.device(dev)


def _stream(stream, dev):
    # the raw handle: making a torch.cuda.Stream object takes longer than a launch
    return torch._C._cuda_getCurrentRawStream(dev.index) if stream is None else stream


def _allocate(stream, dev, *shape, dtype):
    """A tensor that belongs to the stream the kernels are launched on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    if isinstance(stream, int):  # 0: the default stream, which is not an external one
        stream = torch.cuda.ExternalStream(stream, device=dev) if stream else torch.cuda.default_stream(dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _check_cache(kv_cache, block_table, row_offsets, starts, dev):
    """(fp8, batch) of a paged cache and its tables."""
    if not isinstance(kv_cache, torch.Tensor) or not isinstance(block_table, torch.Tensor):
        raise ValueError("kv_cache, block_table: need tensors")
    fp8 = kv_cache.dtype == _U8
    if kv_cache.dim() != 3 or kv_cache.shape[1:] != (64, 656 if fp8 else 576) or block_table.dim() != 2:
        raise ValueError("kv_cache must be [pages, 64, 576] bf16 or [pages, 64, 656] uint8, "
                         "block_table [batch, max_pages_per_seq]")
    batch, width = block_table.shape
    if kv_cache.shape[0] == 0 or not 0 < width <= _INT_MAX or batch > _INT_MAX:
        raise ValueError("kv_cache, block_table: empty, or more than 2^31 - 1 pages per sequence or sequences")
    _check("kv_cache", kv_cache, _U8 if fp8 else _BF16, None, dev)
    _check("block_table", block_table, _I32, None, dev)
    _check("row_offsets", row_offsets, _I32, (batch + 1,), dev)
    if starts is not None:
        _check("starts", starts, _I32, (batch,), dev)
    return fp8, batch


def _launch_read(fp8, kv_cache, block_table, row_offsets, starts, out, error_word, stream):
    desc = B.mlap_read_desc_t(block_table.shape[0], block_table.shape[1], kv_cache.shape[0], out.shape[0], 512, 64, 64)
    fn = B.mlap_cache_read_fp8 if fp8 else B.mlap_cache_read
    B.check(fn(desc, kv_cache, block_table, row_offsets, starts, out, error_word, stream), "mlap_cache_read")


def _check_wkv_b(wkv_b, dev):
    if not isinstance(wkv_b, torch.Tensor) or wkv_b.dim() != 3:
        raise ValueError("wkv_b: need a [heads, 256, 512] tensor")
    _check("wkv_b", wkv_b, _BF16, (wkv_b.shape[0], 256, 512), dev)
    return wkv_b.shape[0]


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
    fp8, _ = _check_cache(kv_cache, block_table, row_offsets, starts, dev)
    _optional_i32("error_word", error_word, dev)
    if out is None:
        if num_rows is None:
            raise ValueError("cache_read needs out or num_rows")
        out = _allocate(stream, dev, num_rows, 576, dtype=_BF16)
    elif not isinstance(out, torch.Tensor) or out.dim() != 2:
        raise ValueError("out: need a [rows, 576] tensor")
    _check("out", out, _BF16, (out.shape[0], 576), dev)
    with _on(dev):
        _launch_read(fp8, kv_cache, block_table, row_offsets, starts, out, error_word, _stream(stream, dev))
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
    M, H = rows.shape[0], _check_wkv_b(wkv_b, dev)
    _optional_i32("row_count", row_count, dev)
    _optional_i32("error_word", error_word, dev)
    if out is None:
        out = _allocate(stream, dev, M, H, 256, dtype=_BF16)
    _check("out", out, _BF16, (M, H, 256), dev)
    with _on(dev):
        B.check(B.mlap_expand_kv(B.mlap_expand_desc_t(M, H, stride, 128, 512, 128), rows, wkv_b, row_count, out,
                                 error_word, _stream(stream, dev)), "mlap_expand_kv")
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
    without keys gets zeros and -inf, a NaN or an infinity in a row of ``q`` NaN
    for its head (``kv`` and ``k_pe`` must be finite in the rows that a sequence
    owns); rows that no sequence owns are left as they were. ``workspace`` (uint8, :func:`attention_workspace_bytes`) is
    allocated when not given; calls that may run at the same time, and graphs
    that may replay at the same time, need one each."""
    dev = _device("q", q)
    if q.dim() != 3:
        raise ValueError("q: need a [queries, heads, 192] tensor")
    Nq, H = q.shape[0], q.shape[1]
    _check("q", q, _BF16, (Nq, H, 192), dev)
    if not isinstance(kv, torch.Tensor) or kv.dim() != 3:
        raise ValueError("kv: need a [keys, heads, 256] tensor")
    Nk = kv.shape[0]
    _check("kv", kv, _BF16, (Nk, H, 256), dev)
    stride = _row_stride("k_pe", k_pe, dev, 64, True)
    if k_pe.shape[0] != Nk:
        raise ValueError(f"k_pe: {k_pe.shape[0]} rows, kv has {Nk}")
    _check("cu_q", cu_q, _I32, None, dev)
    if cu_q.dim() != 1 or not 1 <= cu_q.shape[0] <= _INT_MAX:
        raise ValueError("cu_q: need batch + 1 offsets, batch below 2^31")
    _check("cu_k", cu_k, _I32, cu_q.shape, dev)
    _optional_i32("error_word", error_word, dev)
    if out is None:
        out = _allocate(stream, dev, Nq, H, 128, dtype=_BF16)
    if lse is None:
        lse = _allocate(stream, dev, Nq, H, dtype=_F32)
    _check("out", out, _BF16, (Nq, H, 128), dev)
    _check("lse", lse, _F32, (Nq, H), dev)
    desc = B.mlap_attention_desc_t(cu_q.shape[0] - 1, H, Nq, Nk, stride, int(bool(causal)), softmax_scale, num_sms,
                                   128, 64, 128)
    with _on(dev):
        if workspace is None:
            n = max(B.mlap_attention_workspace_bytes(desc), 32)
            workspace = _allocate(stream, dev, n, dtype=_U8)
        _check("workspace", workspace, _U8, None, dev)
        B.check(B.mlap_attention(desc, q, kv, k_pe, cu_q, cu_k, out, lse, workspace, workspace.numel(), error_word,
                                 _stream(stream, dev)), "mlap_attention")
    return out, lse


def merge_parts(part_out: torch.Tensor, part_lse: torch.Tensor, *, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Merge of attention results over disjoint parts of each row's keys:
    ``part_out`` [parts, ..., 128] bf16, ``part_lse`` [parts, ...] float32
    (``mla_merge``). A part with lse -inf weighs nothing, a NaN lse makes its
    row NaN."""
    dev = _device("part_out", part_out)
    _check("part_out", part_out, torch.bfloat16, None, dev)
    _check("part_lse", part_lse, torch.float32, tuple(part_out.shape[:-1]), dev)
    if part_out.dim() < 2 or part_out.shape[-1] != 128:
        raise ValueError("part_out: need [parts, ..., 128]")
    out = _allocate(stream, dev, *part_out.shape[1:], dtype=_BF16)
    lse = _allocate(stream, dev, *part_lse.shape[1:], dtype=_F32)
    with _on(dev):
        B.check(B.mla_merge(B.make_merge_desc(parts=part_out.shape[0], rows=lse.numel(), d_latent=128), part_out,
                            part_lse, out, lse, _stream(stream, dev)), "mla_merge")
    return out, lse


class MlaPrefill:
    """The prefill of ragged chunks over the paged cache: read back, expand,
    attend. Keys and values are rounded to bf16 in between (2^-8 of each value at
    most), as a bf16 kv up-projection of the model makes them. Owns the buffers for
    up to ``max_queries`` new tokens and ``max_keys`` cached tokens (all sequences
    of a call together; 512 * H + 1152 bytes per key); a call with more is clipped
    and sets a bit of ``error_word``. ``num_sms`` bounds the attention's SMs alone.

    Calls of one object share its buffers and must not overlap: order them, also
    across streams, or use an object for each. The constructor waits for the work
    that its stream holds (unless that is being captured), so that the first call
    may come on any stream. Buffers stay allocated for calls on a ``torch.cuda.Stream``
    given as ``stream`` when the object goes away; it has to outlive calls on a
    raw handle, an external stream or one that was only the current one, and graphs
    captured from it."""

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
        self.rows = torch.empty(max_keys, 576, dtype=torch.bfloat16, device=dev)
        self.kv = torch.empty(max_keys, num_heads, 256, dtype=torch.bfloat16, device=dev)
        self.out = torch.zeros(max_queries, num_heads, 128, dtype=torch.bfloat16, device=dev)
        self.lse = torch.full((max_queries, num_heads), -math.inf, dtype=torch.float32, device=dev)
        self.error_word = torch.zeros(1, dtype=torch.int32, device=dev)
        self._expand_desc = B.make_expand_desc(num_rows=max_keys, num_heads=num_heads)
        self._streams = set()  # handles of the streams that the buffers are recorded on
        # the fills above, and whatever used this memory before, lie on this stream
        with torch.cuda.device(dev):
            if not torch.cuda.is_current_stream_capturing():
                torch.cuda.current_stream(dev).synchronize()

    def _record(self, stream):
        """Ties the buffers to a stream that the allocator may still ask for its
        work when they go away; not to an external one, which may be gone by then."""
        if isinstance(stream, torch.cuda.Stream) and not isinstance(stream, torch.cuda.ExternalStream):
            for t in (self.workspace, self.rows, self.kv, self.out, self.lse, self.error_word):
                t.record_stream(stream)
            self._streams.add(stream.cuda_stream)

    def __call__(self, q: torch.Tensor, wkv_b: torch.Tensor, kv_cache: torch.Tensor, block_table: torch.Tensor,
                 cu_q: torch.Tensor, cu_k: torch.Tensor, *, starts: Optional[torch.Tensor] = None,
                 causal: bool = True, stream=None) -> torch.Tensor:
        """``q`` [Nq, H, 192], Nq at most ``max_queries``; sequence b attends to
        its cached positions ``starts[b] .. starts[b] + cu_k[b + 1] - cu_k[b] - 1``
        (``starts`` None: from 0). Returns ``out`` [Nq, H, 128], a view of a
        buffer that the next call overwrites; its log-sum-exp is ``self.lse[:Nq]``.
        Rows outside ``[cu_q[0], cu_q[batch])`` belong to no sequence and keep what
        an earlier call left there, 0 and -inf where none did: a program whose
        lengths on the device cover fewer than Nq rows takes only those."""
        dev = self.device
        if not isinstance(q, torch.Tensor) or q.dim() != 3 or q.shape[0] > self.out.shape[0]:
            raise ValueError(f"q: need a [queries, {self.num_heads}, 192] tensor of at most {self.out.shape[0]} queries")
        nq, H, M = q.shape[0], self.num_heads, self.rows.shape[0]
        _check("q", q, _BF16, (nq, H, 192), dev)
        if _check_wkv_b(wkv_b, dev) != H:
            raise ValueError(f"wkv_b: {wkv_b.shape[0]} heads, {H} needed")
        fp8, batch = _check_cache(kv_cache, block_table, cu_k, starts, dev)
        _check("cu_q", cu_q, _I32, (batch + 1,), dev)
        out, e = self.out[:nq], self.error_word
        if stream is not None and getattr(stream, "cuda_stream", stream) not in self._streams:
            self._record(stream)
        with _on(dev):
            s = _stream(stream, dev)
            _launch_read(fp8, kv_cache, block_table, cu_k, starts, self.rows, e, s)
            B.check(B.mlap_expand_kv(self._expand_desc, self.rows, wkv_b, cu_k.data_ptr() + 4 * batch, self.kv, e, s),
                    "mlap_expand_kv")
            desc = B.mlap_attention_desc_t(batch, H, nq, M, 576, int(bool(causal)), self.softmax_scale, self.num_sms,
                                           128, 64, 128)
            B.check(B.mlap_attention(desc, q, self.kv, self.rows.data_ptr() + 1024, cu_q, cu_k, out, self.lse,
                                     self.workspace, self.workspace.numel(), e, s), "mlap_attention")
        return out
