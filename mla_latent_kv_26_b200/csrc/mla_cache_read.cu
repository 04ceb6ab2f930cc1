// Read-back of cached rows: the rows of ragged runs of positions, gathered
// from the paged latent cache into a dense [rows, 576] bf16 matrix.
//
//   rows[off[b] + j] = row of position starts[b] + j of sequence b
//
// bf16 cache: the 1152-byte row as it is. fp8 cache (656 bytes: 512 e4m3
// codes, 64 bf16 rope values, the float32 scale): the latent as
// bf16(float32(code * scale)), the values the fp8 decode works on, and the
// rope unchanged.
//
// Bound by HBM: 1152 (bf16) or 644 of 656 (fp8) bytes read and 1152 written
// per row. One warp handles four output rows: 4 x 72 sixteen-byte pieces are
// nine per lane, so that every lane has nine loads in flight and the warp's
// stores are one contiguous run of 4608 bytes. Blocks of four warps: 270k fp8
// rows take 80 us (0.89 of the copy bandwidth), with eight 84 us, with eight
// rows to a warp 89 us.
#include <cuda_runtime.h>

#include "mla.h"
#include "mla_prefill.h"
#include "prefill.cuh"

namespace mla {
namespace prefill {

struct ReadArgs {
  const uint8_t* cache;
  const int32_t* block_table;  // [batch, max_pages_per_seq]
  const int32_t* offsets;      // [batch + 1]
  const int32_t* starts;       // [batch] or nullptr: 0
  uint8_t* rows;               // [num_rows, 576] bf16
  uint32_t* error;
  int batch, max_pages_per_seq, num_pages, num_rows;
};

constexpr int kReadWarps = 4;
constexpr int kRowsPerWarp = 4;
constexpr int kRowBytes = kDQK * 2;
constexpr int kPieces = kRowBytes / 16;                        // 72 per row
constexpr int kLanePieces = kRowsPerWarp * kPieces / 32;       // 9 per lane
static_assert(kLanePieces * 32 == kRowsPerWarp * kPieces, "the warp's pieces divide evenly");

// Largest b in [0, batch) with offsets[b] <= row (0 if there is none): 32-way
// steps of the whole warp, one round of loads per factor 32 of the batch.
MLA_DEV int find_sequence(const int32_t* offsets, int batch, int row, int lane) {
  int a = 0, e = batch - 1;
  while (a < e) {
    const int step = (e - a + 31) / 32;
    const int q = min(a + (lane + 1) * step, e);
    const unsigned le = __ballot_sync(~0u, __ldg(offsets + q) <= row);
    const int m = le == ~0u ? 32 : __ffs(~le) - 1;  // leading lanes whose offset is not beyond the row
    const int below = __shfl_sync(~0u, q, max(m - 1, 0)), above = __shfl_sync(~0u, q, min(m, 31));
    if (m < 32) e = above - 1;
    if (m > 0) a = below;
    if (e < a) e = a;
  }
  return a;
}

template <bool kF8>
__global__ void __launch_bounds__(kReadWarps * 32) mla_cache_read_kernel(const ReadArgs a) {
  const int lane = threadIdx.x & 31;
  const int row0 = (int)(blockIdx.x * kReadWarps + (threadIdx.x >> 5)) * kRowsPerWarp;
  allow_dependents();
  grid_dependency_wait();
  const int end = __ldg(a.offsets + a.batch);
  uint32_t err = 0u;
  if (blockIdx.x == 0) {  // the first block reports offsets out of range or out of order
    for (int b = threadIdx.x; b <= a.batch; b += kReadWarps * 32) {
      const int o = __ldg(a.offsets + b);
      if (o < (b > 0 ? __ldg(a.offsets + b - 1) : 0) || o > a.num_rows) set_error(a.error, kErrSeqLen);
    }
  }
  if (row0 >= a.num_rows) return;
  // lanes 0..3 find the cache row of output rows row0 .. row0 + 3: its index,
  // -1 = a bad position or page (zeros are written), -2 = no sequence's row (left as it is)
  int src = -2;
  if (row0 < end) {
    int b = find_sequence(a.offsets, a.batch, row0, lane);
    const int r = row0 + lane;
    if (lane < kRowsPerWarp && r < a.num_rows && r < end) {
      while (b + 1 < a.batch && __ldg(a.offsets + b + 1) <= r) ++b;
      const int o0 = __ldg(a.offsets + b), o1 = __ldg(a.offsets + b + 1);
      if (r >= o0 && r < o1) {
        const long long p = (long long)r - o0 + (a.starts ? __ldg(a.starts + b) : 0);
        src = -1;
        if (p < 0 || p >= (long long)a.max_pages_per_seq * kPage) {
          err |= kErrPosition;
        } else {
          const int page = __ldg(a.block_table + (size_t)b * a.max_pages_per_seq + p / kPage);
          if (page < 0 || page >= a.num_pages) err |= kErrPageId;
          else src = page * kPage + (int)(p % kPage);
        }
      }
    }
  }
  if (err) set_error(a.error, err);
  float scale = 0.f;
  if (kF8 && src >= 0) scale = __ldg(reinterpret_cast<const float*>(a.cache + (size_t)src * kF8RowBytes + kF8ScaleOff));

  uint4 v[kLanePieces];
  int from[kLanePieces];
#pragma unroll
  for (int i = 0; i < kLanePieces; ++i) {
    const int piece = lane + 32 * i, r = piece / kPieces, c = piece % kPieces;
    from[i] = __shfl_sync(~0u, src, r);
    v[i] = make_uint4(0, 0, 0, 0);
    if (from[i] >= 0) {
      if constexpr (!kF8) {
        v[i] = __ldcs(reinterpret_cast<const uint4*>(a.cache + (size_t)from[i] * kRowBytes) + c);
      } else {
        const uint8_t* row = a.cache + (size_t)from[i] * kF8RowBytes;
        if (c < kDLatent / 8) {
          const uint2 w = __ldcs(reinterpret_cast<const uint2*>(row) + c);
          v[i].x = w.x;
          v[i].y = w.y;
        } else {
          v[i] = __ldcs(reinterpret_cast<const uint4*>(row + kF8RopeOff) + (c - kDLatent / 8));
        }
      }
    }
  }
  uint4* dst = reinterpret_cast<uint4*>(a.rows + (size_t)row0 * kRowBytes);
#pragma unroll
  for (int i = 0; i < kLanePieces; ++i) {
    const int piece = lane + 32 * i, r = piece / kPieces, c = piece % kPieces;
    const float s = kF8 ? __shfl_sync(~0u, scale, r) : 0.f;
    if (from[i] == -2) continue;
    if (kF8 && c < kDLatent / 8) v[i] = dequant8_e4m3(v[i].x, v[i].y, s);
    dst[piece] = v[i];
  }
}

mla_status_t cache_read(const mlap_read_desc_t* d, const void* cache, const int32_t* block_table,
                        const int32_t* offsets, const int32_t* starts, void* rows, uint32_t* error, bool fp8,
                        cudaStream_t stream) {
  if (!d) return MLA_ERR_INVALID_ARG;
  if (d->batch < 0 || d->max_pages_per_seq < 1 || d->num_pages < 1 || d->num_rows < 0) return MLA_ERR_INVALID_ARG;
  if (d->d_latent != kDLatent || d->d_rope != kDRope || d->page_size != kPage || d->batch > kMaxBatch)
    return MLA_ERR_UNSUPPORTED;
  if ((long long)d->num_pages * kPage > 0x7fffffffLL || (long long)d->max_pages_per_seq * kPage > 0x7fffffffLL ||
      d->num_rows > 0x7fffffff - kRowsPerWarp * kReadWarps)
    return MLA_ERR_UNSUPPORTED;
  if (d->batch == 0 || d->num_rows == 0) return MLA_OK;
  if (!cache || !block_table || !offsets || !rows) return MLA_ERR_INVALID_ARG;
  const auto off = [](const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) != 0; };
  if (off(cache, 16) || off(rows, 16) || off(block_table, 4) || off(offsets, 4) || off(starts, 4) || off(error, 4))
    return MLA_ERR_INVALID_ARG;
  ReadArgs a{static_cast<const uint8_t*>(cache), block_table, offsets, starts, static_cast<uint8_t*>(rows), error,
             d->batch, d->max_pages_per_seq, d->num_pages, d->num_rows};
  const int per = kReadWarps * kRowsPerWarp;
  const int grid = (d->num_rows + per - 1) / per;
  return launch_dependent(fp8 ? mla_cache_read_kernel<true> : mla_cache_read_kernel<false>, dim3(grid), kReadWarps * 32, 0,
                          stream, a) == cudaSuccess
             ? MLA_OK
             : MLA_ERR_CUDA;
}

}  // namespace prefill
}  // namespace mla

extern "C" MLA_API mla_status_t mlap_cache_read(const mlap_read_desc_t* desc, const void* kv_cache,
                                                const int32_t* block_table, const int32_t* row_offsets,
                                                const int32_t* starts, void* rows, uint32_t* error_word,
                                                mla_stream_t stream) {
  return mla::prefill::cache_read(desc, kv_cache, block_table, row_offsets, starts, rows, error_word, false,
                                  (cudaStream_t)stream);
}

extern "C" MLA_API mla_status_t mlap_cache_read_fp8(const mlap_read_desc_t* desc, const void* kv_cache_fp8,
                                                    const int32_t* block_table, const int32_t* row_offsets,
                                                    const int32_t* starts, void* rows, uint32_t* error_word,
                                                    mla_stream_t stream) {
  return mla::prefill::cache_read(desc, kv_cache_fp8, block_table, row_offsets, starts, rows, error_word, true,
                                  (cudaStream_t)stream);
}
