"""Prefill of a chunk of new tokens over the paged latent cache, the plain definition.

TEST INFRASTRUCTURE ONLY: imported by tests and ``__graft_entry__.smoke()``;
never by the product path.

Source: "深度解读DeepSeek：源码解读 DeepSeek-V3", section "MLA", the unabsorbed
branch (the latent expanded through ``wkv_b`` into per-head keys and values,
``k = [k_nope, k_pe]`` with ``k_pe`` shared by all heads, standard attention);
"DeepSeek-V2-Lite 模型结构详解", section "五、MLA：注意力" (widths 128 + 64 and 128).

Readings where the pages are silent:

* Ragged batches: sequence b owns rows ``[offsets[b], offsets[b + 1])``.
* Causal: a sequence's n queries are its last n positions, query i sees keys
  ``t <= L - n + i`` (decode's rule); with n > L the first n - L rows see none.
* A row without keys: out = 0, lse = -inf.
"""

from __future__ import annotations

import math

import torch

from .decode import DEFAULT_SOFTMAX_SCALE, PAGE_SIZE, attention_probs
from .fp8_cache import dequantize_cache


def cache_read(cache, block_table, row_offsets, starts, rows):
    """``rows`` [M, 576] with the rows of every sequence replaced by the cache
    rows of positions ``starts[b] + j``; positions or pages that do not exist
    give zeros. ``cache``: [pages, 64, 576] values, or uint8 [pages, 64, 656]."""
    out = rows.to(torch.float64).clone()
    values = dequantize_cache(cache) if cache.dtype == torch.uint8 else cache
    num_pages, width = values.shape[0], block_table.shape[1]
    off = [int(x) for x in row_offsets]
    for b in range(len(off) - 1):
        first = 0 if starts is None else int(starts[b])
        for r in range(off[b], min(off[b + 1], out.shape[0])):
            p = first + r - off[b]
            page = int(block_table[b, p // PAGE_SIZE]) if 0 <= p < width * PAGE_SIZE else -1
            out[r] = values[page, p % PAGE_SIZE].to(torch.float64) if 0 <= page < num_pages else 0.0
    return out


def expand_kv(rows, wkv_b):
    """``kv[t, h, j] = sum_c wkv_b[h, j, c] rows[t, c]`` over the first 512 columns."""
    return torch.einsum("tc,hjc->thj", rows[:, :512].to(torch.float64), wkv_b.to(torch.float64))


def prefill_attention(q, kv, k_pe, cu_q, cu_k, *, causal=True, softmax_scale: float = DEFAULT_SOFTMAX_SCALE,
                      absolute: bool = False):
    """``(out [Nq, H, 128], lse [Nq, H])`` in float64 (rows no sequence owns: NaN).

    With ``absolute`` also ``(mag, smag, smax)`` per row, from which tests take
    rounding bounds: ``sum_t p_t |v_t|`` [Nq, H, 128], the largest
    ``scale * sum_d |q_d k_d|`` and the largest ``|s_t|`` over the visible keys
    [Nq, H] (0 for a row without keys)."""
    Nq, H = q.shape[:2]
    q, kv, k_pe = q.to(torch.float64), kv.to(torch.float64), k_pe.to(torch.float64)
    out = torch.full((Nq, H, 128), math.nan, dtype=torch.float64)
    lse = torch.full((Nq, H), math.nan, dtype=torch.float64)
    mag, smag, smax = torch.zeros(Nq, H, 128).double(), torch.zeros(Nq, H).double(), torch.zeros(Nq, H).double()
    for b in range(len(cu_q) - 1):
        q0, q1, k0, k1 = int(cu_q[b]), int(cu_q[b + 1]), int(cu_k[b]), int(cu_k[b + 1])
        n, L = q1 - q0, k1 - k0
        for h in range(H):
            key = torch.cat([kv[k0:k1, h, :128], k_pe[k0:k1]], -1)
            val = kv[k0:k1, h, 128:]
            s_all = softmax_scale * (q[q0:q1, h] @ key.T)
            a_all = softmax_scale * (q[q0:q1, h].abs() @ key.abs().T) if absolute else None
            for i in range(n):
                seen = max(min(L, L - n + i + 1), 0) if causal else L
                if seen == 0:
                    out[q0 + i, h], lse[q0 + i, h] = 0.0, -math.inf
                    continue
                p, l = attention_probs(s_all[i, :seen])
                out[q0 + i, h], lse[q0 + i, h] = p @ val[:seen], l
                if absolute:
                    mag[q0 + i, h] = p @ val[:seen].abs()
                    smag[q0 + i, h], smax[q0 + i, h] = a_all[i, :seen].max(), s_all[i, :seen].abs().max()
    return (out, lse, mag, smag, smax) if absolute else (out, lse)
