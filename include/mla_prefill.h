/*
 * libmla, prefill — attention of a chunk of new tokens over the paged latent
 * KV cache, for NVIDIA B200 (sm_100a).
 *
 * Decode (mla.h) works in the latent space: 2 * (576 + 512) operations per
 * query, head and key. For a chunk of many new tokens the other branch of MLA
 * is cheaper: expand the cached latents once into per-head keys and values and
 * run standard attention over them, 2 * (192 + 128) operations per query, head
 * and key, plus 2 * 512 * 256 per key and head for the expansion ("深度解读
 * DeepSeek：源码解读 DeepSeek-V3", section "MLA", the unabsorbed branch;
 * "DeepSeek-V2-Lite 模型结构详解", section "五、MLA：注意力"). As operations the
 * two are equal at about 170 new tokens per sequence. Measured, the three calls
 * below take less time than absorb, decode and un-absorb from about 10 new tokens
 * per sequence on with 16 heads, and with 128 heads from about 50 (8 sequences of
 * 600 tokens), 90 (one of 4096 or 16384) or 130 (4 of 8192). In order, on one
 * stream:
 *
 *   mlap_cache_read  -> rows of the sequences, read back from the paged cache
 *   mlap_expand_kv   -> per-head keys and values of those rows
 *   mlap_attention   -> ragged (causal) attention of the new tokens over them
 *
 * Everything is asynchronous on the stream, with no host synchronisation and
 * no allocation: lengths live on the device, so a captured CUDA graph replays
 * with other lengths within the same capacities. Ownership, alignment and
 * errors are those of mla.h: bad arguments are reported before any launch; bad
 * lengths, positions or page ids seen on the device never trap, set a bit of
 * the caller's error word (device uint32 or NULL; bits are OR-ed in, never
 * cleared) and are clipped or skipped.
 *
 * Ragged rows: sequence b owns rows [offsets[b], offsets[b + 1]) of a matrix;
 * offsets is int32 [batch + 1], non-decreasing. Rows before offsets[0] and from
 * offsets[batch] on belong to no sequence and are left as they were. A call
 * without sequences, or without rows to write, launches and reports nothing.
 */
#ifndef LIBMLA_MLA_PREFILL_H_
#define LIBMLA_MLA_PREFILL_H_

#include "mla.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------------------
 * Cache read-back:
 *
 *   rows[row_offsets[b] + j] = cache row of position starts[b] + j of sequence b
 *
 * for 0 <= j < row_offsets[b + 1] - row_offsets[b]. mlap_cache_read copies rows
 * of the bf16 cache; mlap_cache_read_fp8 turns the 656-byte rows of the fp8
 * cache into the values they stand for, latent bf16(float32(code * scale)) and
 * k_pe unchanged (the values mla_decode_fp8 works on).
 *
 *   kv_cache     bf16 [num_pages, 64, 576], or 656-byte rows [num_pages, 64, 656]
 *   block_table  int32 [batch, max_pages_per_seq]
 *   row_offsets  int32 [batch + 1]
 *   starts       int32 [batch] first position of each sequence, or NULL: 0
 *   rows         bf16 [num_rows, 576], 16-byte aligned
 *
 * A position outside [0, max_pages_per_seq * 64) sets MLA_DEVERR_POSITION, a
 * page id outside [0, num_pages) MLA_DEVERR_PAGE_ID: that row is written as
 * zeros. row_offsets beyond num_rows or out of order set MLA_DEVERR_SEQ_LEN;
 * no row outside [0, num_rows) is touched. */
typedef struct {
  int32_t batch;             /* 0..2^22 */
  int32_t max_pages_per_seq; /* block_table row stride (entries), >= 1 */
  int32_t num_pages;         /* physical pages in kv_cache, >= 1 */
  int32_t num_rows;          /* capacity of rows, >= 0 */
  int32_t d_latent;          /* must be 512 */
  int32_t d_rope;            /* must be 64 */
  int32_t page_size;         /* must be 64 */
} mlap_read_desc_t;

MLA_API mla_status_t mlap_cache_read(const mlap_read_desc_t* desc, const void* kv_cache, const int32_t* block_table,
                                     const int32_t* row_offsets, const int32_t* starts, void* rows,
                                     uint32_t* error_word, mla_stream_t stream);
MLA_API mla_status_t mlap_cache_read_fp8(const mlap_read_desc_t* desc, const void* kv_cache_fp8,
                                         const int32_t* block_table, const int32_t* row_offsets,
                                         const int32_t* starts, void* rows, uint32_t* error_word,
                                         mla_stream_t stream);

/* ---------------------------------------------------------------------------
 * Key / value expansion:
 *
 *   kv[t, h, j] = sum_c wkv_b[h, j, c] * rows[t, c]      j < 256, c < 512
 *
 * kv[t, h, 0:128] is head h's no-rope key of row t, kv[t, h, 128:256] its value
 * (wkv_b: the model's kv up-projection [H, 256, 512], as in mla_absorb_query).
 * bf16 in and out, float32 accumulation on the tensor cores, one kernel.
 *
 *   rows       bf16, row t at rows + t * row_stride, the latent its first 512 values
 *   wkv_b      bf16 [H, 256, 512]
 *   kv         bf16 [num_rows, H, 256]
 *   row_count  device int32 or NULL: only rows below *row_count (at most num_rows)
 *              are computed and written
 * rows, wkv_b, kv 16-byte aligned. */
typedef struct {
  int32_t num_rows;   /* >= 0 */
  int32_t num_heads;  /* H: 1..128 */
  int32_t row_stride; /* elements between rows, >= 512, a multiple of 8 */
  int32_t d_nope;     /* must be 128 */
  int32_t d_latent;   /* must be 512 */
  int32_t d_v;        /* must be 128 */
} mlap_expand_desc_t;

MLA_API mla_status_t mlap_expand_kv(const mlap_expand_desc_t* desc, const void* rows, const void* wkv_b,
                                    const int32_t* row_count, void* kv, uint32_t* error_word, mla_stream_t stream);

/* ---------------------------------------------------------------------------
 * Ragged attention of new tokens over expanded keys and values. Sequence b has
 * n = cu_q[b + 1] - cu_q[b] queries and L = cu_k[b + 1] - cu_k[b] keys; for its
 * query i, key t and head h
 *
 *   s_t  = scale * ( q[i,h,0:128] . kv[t,h,0:128] + q[i,h,128:192] . k_pe[t] )
 *   T    = all t < L, or, causal, t <= L - n + i (the queries are the last n positions)
 *   lse  = ln sum_{t in T} exp(s_t)
 *   out  = sum_{t in T} exp(s_t - lse) * kv[t,h,128:256]
 *
 * A row with no visible key gets out = 0, lse = -inf. A NaN or an infinity in
 * q[i,h] makes out and lse of that query and head NaN if it sees a key, and touches
 * no other row. Without `causal` the call computes one part of a longer context;
 * mla_merge (d_latent = 128) joins the parts. Rows of kv and k_pe that no sequence
 * owns may hold anything; a sequence's own rows must be finite (a masked value
 * still enters the tensor cores' products with weight 0).
 *
 *   q      bf16 [num_q, H, 192]  (q_nope[128] || q_pe[64], q_pe rotated)
 *   kv     bf16 [num_k, H, 256]  (mlap_expand_kv)
 *   k_pe   bf16, row t at k_pe + t * pe_stride, 64 values (columns 512.. of the rows
 *          read back, or a [num_k, 64] matrix)
 *   cu_q, cu_k  int32 [batch + 1]
 *   out    bf16 [num_q, H, 128]   lse  fp32 [num_q, H] (natural log)
 *   workspace   at least mlap_attention_workspace_bytes: partial results of split
 *          work; calls that may overlap on the GPU need one each
 * q, kv, k_pe 16-byte aligned, out and workspace 32-byte aligned. cu_q / cu_k beyond num_q / num_k or
 * out of order set MLA_DEVERR_SEQ_LEN and are clipped. Two kernels. Probabilities
 * are rounded to bf16 for the product with the values (their sums are not);
 * everything else is float32. The result does not depend on timing: work is
 * split by the lengths alone. */
typedef struct {
  int32_t batch;       /* 0..2^22 */
  int32_t num_heads;   /* H: 1..128 */
  int32_t num_q;       /* rows of q, out, lse; >= 0 */
  int32_t num_k;       /* rows of kv and k_pe; >= 0 */
  int32_t pe_stride;   /* elements between rows of k_pe, >= 64, a multiple of 8 */
  int32_t causal;      /* 0 or 1 */
  float softmax_scale; /* > 0; 1/sqrt(192) for DeepSeek V2/V3 */
  int32_t num_sms;     /* SMs to spread the work over, in pairs (1: one pair); 0 = all of the current device */
  int32_t d_nope;      /* must be 128 */
  int32_t d_rope;      /* must be 64 */
  int32_t d_v;         /* must be 128 */
} mlap_attention_desc_t;

/* Bytes of the workspace on the current device (0 if the descriptor is invalid). */
MLA_API size_t mlap_attention_workspace_bytes(const mlap_attention_desc_t* desc);

MLA_API mla_status_t mlap_attention(const mlap_attention_desc_t* desc, const void* q, const void* kv,
                                    const void* k_pe, const int32_t* cu_q, const int32_t* cu_k, void* out, float* lse,
                                    void* workspace, size_t workspace_bytes, uint32_t* error_word,
                                    mla_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LIBMLA_MLA_PREFILL_H_ */
