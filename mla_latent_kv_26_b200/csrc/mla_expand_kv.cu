// Key / value expansion: per-head keys and values of cached rows, the product
// of the latents with the model's kv up-projection,
//
//   kv[t, h, j] = sum_c wkv_b[h, j, c] * rows[t, c]     t < rows, j < 256, c < 512
//
// one GEMM of M = rows, N = H * 256, K = 512 on tcgen05. A CTA pair
// (cta_group::2) makes tiles of 256 rows x one head: M 256, N 256, each CTA with
// 128 of the rows and half of the head's weight rows in shared memory and its
// 128 rows of the float32 accumulator in TMEM (256 columns, two of them, so that
// one tile is written while the next is computed). Tiles are dealt to the pairs
// in runs, heads fastest, and a CTA's latents (128 KB for the whole K) stay in
// shared memory for a run of heads: per 4096 cycles of products an SM loads
// 128 KB of weights and nothing else. 8209 rows x 128 heads, replayed: 227 us,
// 1.22 PFLOP/s in bursts at 1965 MHz, 257 us at 1.44 GHz under the power cap; a
// library product of the size 238 and 276. (Loading both operands for every tile of
// 128 x 256 on single CTAs, 384 KB per 4096 cycles, took 292 us when this took 280.)
//
// Per row and head 262144 operations and 512 bytes written: compute bound for
// all but a few rows.
//
// Per CTA (192 threads): warps 0-3 epilogue (TMEM -> bf16 -> shared memory ->
// TMA store of 64-column boxes), warp 4 issues the MMAs (even CTA), warp 5 loads
// (TMA).
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <mutex>

#include "mla.h"
#include "mla_prefill.h"
#include "prefill.cuh"

namespace mla {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

namespace prefill {

constexpr int kExpThreads = 192;
constexpr int kKBlocks = kDLatent / 64;    // 64-column blocks of the latents and weights
constexpr int kExpStages = 5;              // ring of weight blocks (128 weight rows x 64 columns)
constexpr int kOutBytes = 32 * 128;        // an epilogue warp's 32 rows x 64 columns on their way out
constexpr int kExpSmem = 1024 + (kKBlocks + kExpStages) * kBox + 4 * kOutBytes;
constexpr int kExpRows = 256;              // rows of a pair's tile

struct ExpandMaps {
  CUtensorMap rows;  // [num_rows, 512 of row_stride]
  CUtensorMap w;     // [H * 256, 512]
  CUtensorMap kv;    // [num_rows, H * 256], boxes of 32 rows
};

struct ExpandArgs {
  const int32_t* row_count;  // device or nullptr
  __nv_bfloat16* kv;
  uint32_t* error;
  int num_rows, heads;
};

struct ExpandShared {
  // "even": only the even CTA's is used, by both CTAs; "both": each CTA's own
  uint64_t a_full[kKBlocks];       // even: a block of both CTAs' latents has landed
  uint64_t a_empty;                // both: the products of a run of heads are done
  uint64_t full[kExpStages];       // even: both halves of a weight block have landed
  uint64_t empty[kExpStages];      // both
  uint64_t t_full[2];              // both: an accumulator is complete
  uint64_t t_empty[2];             // even: both CTAs have read it
  uint64_t done;
  uint32_t tmem;
  uint32_t abort_flag;
};

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kExpThreads, 1)
    mla_expand_kv_kernel(const __grid_constant__ ExpandMaps maps, const ExpandArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ ExpandShared sh;
  const uint32_t latents = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t ring = latents + kKBlocks * kBox, stage_out = ring + kExpStages * kBox;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_ctarank();
  Waiter W{&sh.abort_flag, a.error};
  allow_dependents();
  grid_dependency_wait();
  const int rows = a.row_count ? min(max(__ldg(a.row_count), 0), a.num_rows) : a.num_rows;
  const long long tiles = (long long)((rows + kExpRows - 1) / kExpRows) * a.heads;
  const int pairs = gridDim.x / 2;
  const long long per = (tiles + pairs - 1) / pairs;
  const long long i0 = min(cluster_id_x() * per, tiles), i1 = min(i0 + per, tiles);
  if (i0 >= i1) return;  // both CTAs of the pair

  if (threadIdx.x == 0) {
    for (int k = 0; k < kKBlocks; ++k) mbar_init(smem_addr(&sh.a_full[k]), 2);
    mbar_init(smem_addr(&sh.a_empty), 1);
    for (int s = 0; s < kExpStages; ++s) {
      mbar_init(smem_addr(&sh.full[s]), 2);
      mbar_init(smem_addr(&sh.empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_addr(&sh.t_full[b]), 1);
      mbar_init(smem_addr(&sh.t_empty[b]), 8);  // four epilogue warps of either CTA
    }
    mbar_init(smem_addr(&sh.done), 1);
    sh.abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == 4) {
    tmem_alloc_pair(smem_addr(&sh.tmem), 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const auto leader = [&](uint64_t* bar) { return map_to_rank(smem_addr(bar), 0); };
  const auto m_tile = [&](long long i) { return (int)(i / a.heads); };

  if (warp == 5) {
    if (elect_one()) {
      int n = 0, na = 0;  // weight blocks, sets of latents
      bool ok = true;
      for (long long i = i0; i < i1 && ok; ++i) {
        const int m = m_tile(i), h = (int)(i % a.heads);
        const bool load_a = i == i0 || m != m_tile(i - 1);
        if (load_a && !(ok = W.wait(&sh.a_empty, (na & 1) ^ 1))) break;
        for (int k = 0; k < kKBlocks; ++k, ++n) {
          if (load_a) {
            const uint32_t af = leader(&sh.a_full[k]);
            mbar_arrive_expect_tx_cluster(af, kBox);
            tma_load_2d_pair(latents + k * kBox, &maps.rows, 64 * k, m * kExpRows + rank * 128, af);
          }
          const int s = n % kExpStages;
          if (!(ok = W.wait(&sh.empty[s], ((n / kExpStages) & 1) ^ 1))) break;
          const uint32_t f = leader(&sh.full[s]);
          mbar_arrive_expect_tx_cluster(f, kBox);
          tma_load_2d_pair(ring + s * kBox, &maps.w, 64 * k, h * 256 + rank * 128, f);
        }
        na += load_a;
      }
      // Every load was waited for by its reader, unless a wait ran out: then
      // the copies in flight get ample time before the CTA exits.
      if (W.aborted()) {
        const uint64_t t = global_timer_ns();
        while (global_timer_ns() - t < 10000000ull) {}
      }
    }
    __syncwarp();
  } else if (warp == 4) {
    if (rank == 0 && elect_one()) {
      constexpr uint32_t idesc = idesc_bf16_f32(256, 256, 0, 0);
      int n = 0, nt = 0, na = 0;
      bool ok = true;
      for (long long i = i0; i < i1 && ok; ++i, ++nt) {
        const int b = nt & 1;
        const bool new_a = i == i0 || m_tile(i) != m_tile(i - 1);
        if (!(ok = W.wait(&sh.t_empty[b], ((nt >> 1) & 1) ^ 1))) break;
        for (int k = 0; k < kKBlocks; ++k, ++n) {
          const int s = n % kExpStages;
          if (new_a && !(ok = W.wait(&sh.a_full[k], na & 1))) break;
          if (!(ok = W.wait(&sh.full[s], (n / kExpStages) & 1))) break;
          tc_fence_after();
          const uint64_t ad = smem_desc_sw128(latents + k * kBox, 16, 1024), bd = smem_desc_sw128(ring + s * kBox, 16, 1024);
#pragma unroll
          for (int u = 0; u < 4; ++u)
            mma_ss_pair(tmem + 256 * b, ad + 2 * u, bd + 2 * u, idesc, (k > 0 || u > 0) ? 1u : 0u);
          mma_commit_pair(smem_addr(&sh.empty[s]));
        }
        if (!ok) break;
        na += new_a;
        mma_commit_pair(smem_addr(&sh.t_full[b]));
        if (i + 1 < i1 && m_tile(i + 1) != m_tile(i)) mma_commit_pair(smem_addr(&sh.a_empty));
      }
      mma_commit_pair(smem_addr(&sh.done));
      W.wait(&sh.done, 0, true);
    }
    __syncwarp();
  } else {
    // each warp for itself: 32 rows, 64 columns at a time
    const uint32_t box = stage_out + warp * kOutBytes;
    const uint64_t policy = l2_evict_first();
    int nt = 0;
    for (long long i = i0; i < i1; ++i, ++nt) {
      const int m0 = m_tile(i) * kExpRows + rank * 128 + 32 * warp, h = (int)(i % a.heads), b = nt & 1;
      if (!W.wait_warp(&sh.t_full[b], (nt >> 1) & 1)) break;
      tc_fence_after();
      const uint32_t acc = tmem + ((uint32_t)(32 * warp) << 16) + 256 * b;
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t r[2][32];
        tmem_ld_32x32b_32(acc + 64 * c, r[0]);
        tmem_ld_32x32b_32(acc + 64 * c + 32, r[1]);
        tmem_wait_ld();
        if (c == 3) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(leader(&sh.t_empty[b]));
        }
        if (lane == 0) bulk_wait_read();  // the columns before have left the buffer
        __syncwarp();
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int u = 0; u < 4; ++u)
            st_shared_v4(box + lane * 128 + (((uint32_t)(4 * x + u) ^ (uint32_t)(lane & 7)) << 4),
                         make_uint4(pack_bf16x2(__uint_as_float(r[x][8 * u + 0]), __uint_as_float(r[x][8 * u + 1])),
                                    pack_bf16x2(__uint_as_float(r[x][8 * u + 2]), __uint_as_float(r[x][8 * u + 3])),
                                    pack_bf16x2(__uint_as_float(r[x][8 * u + 4]), __uint_as_float(r[x][8 * u + 5])),
                                    pack_bf16x2(__uint_as_float(r[x][8 * u + 6]), __uint_as_float(r[x][8 * u + 7]))));
        if (m0 + 32 <= rows) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d_hint(&maps.kv, box, h * 256 + 64 * c, m0, policy);
            bulk_commit();
          }
        } else {
          // the last rows: only those below the count are written, 8 lanes per row
          __syncwarp();
#pragma unroll 1
          for (int g = 0; g < 8; ++g) {
            const int rr = 4 * g + (lane >> 3), j = lane & 7;
            const uint4 v = ld_shared_v4(box + rr * 128 + ((uint32_t)(j ^ (rr & 7)) << 4));
            if (m0 + rr < rows)
              *reinterpret_cast<uint4*>(a.kv + ((size_t)(m0 + rr) * a.heads + h) * 256 + 64 * c + 8 * j) = v;
          }
        }
      }
    }
    if (lane == 0) bulk_wait_read();  // shared memory is read before the CTA can exit
    __syncwarp();
  }

  tc_fence_before();
  cluster_sync();  // neither CTA leaves while the other may still reach its shared memory or TMEM
  tc_fence_after();
  if (warp == 4) tmem_dealloc_pair(tmem, 512);
}

// SMs of the current device, the kernel's shared memory opted into (once per
// device); 0 on a CUDA error.
int expand_sms() {
  static std::mutex mu;
  static int sms[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    cudaGetLastError();
    return 0;
  }
  std::lock_guard<std::mutex> lock(mu);
  if (sms[dev] == 0) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaFuncSetAttribute((const void*)mla_expand_kv_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kExpSmem) != cudaSuccess) {
      cudaGetLastError();
      return 0;
    }
    sms[dev] = n;
  }
  return sms[dev];
}

mla_status_t expand(const mlap_expand_desc_t* d, const void* rows, const void* wkv_b, const int32_t* row_count,
                    void* kv, uint32_t* error, cudaStream_t stream) {
  if (!d) return MLA_ERR_INVALID_ARG;
  if (d->num_rows < 0 || d->num_heads < 1 || d->row_stride < kDLatent) return MLA_ERR_INVALID_ARG;
  if (d->num_heads > kMaxHeads || d->d_nope != 128 || d->d_v != 128 || d->d_latent != kDLatent ||
      d->row_stride % 8 != 0 || d->num_rows > 0x7fffffff - 256)
    return MLA_ERR_UNSUPPORTED;
  if (d->num_rows == 0) return MLA_OK;
  if (!rows || !wkv_b || !kv) return MLA_ERR_INVALID_ARG;
  const auto off = [](const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) != 0; };
  if (off(rows, 16) || off(wkv_b, 16) || off(kv, 16) || off(row_count, 4) || off(error, 4)) return MLA_ERR_INVALID_ARG;
  const int sms = expand_sms();
  if (sms == 0) return MLA_ERR_CUDA;
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) return MLA_ERR_CUDA;
  const auto encode = [&](CUtensorMap* m, const void* p, long long cols, long long n, long long stride, int box_rows) {
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)n}, strides[1] = {(cuuint64_t)stride * 2};
    cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, elem[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(p), dims, strides, box, elem,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  ExpandMaps maps;
  const long long width = (long long)d->num_heads * 256;
  if (!encode(&maps.rows, rows, kDLatent, d->num_rows, d->row_stride, 128) ||
      !encode(&maps.w, wkv_b, kDLatent, width, kDLatent, 128) || !encode(&maps.kv, kv, width, d->num_rows, width, 32))
    return MLA_ERR_CUDA;
  ExpandArgs a{row_count, static_cast<__nv_bfloat16*>(kv), error, d->num_rows, d->num_heads};
  const long long tiles = (long long)((d->num_rows + kExpRows - 1) / kExpRows) * d->num_heads;
  const int pairs = (int)(tiles < sms / 2 ? tiles : (sms < 2 ? 1 : sms / 2));
  return launch_dependent(mla_expand_kv_kernel, dim3(2 * pairs), kExpThreads, kExpSmem, stream, maps, a) == cudaSuccess
             ? MLA_OK
             : MLA_ERR_CUDA;
}

}  // namespace prefill
}  // namespace mla

extern "C" MLA_API mla_status_t mlap_expand_kv(const mlap_expand_desc_t* desc, const void* rows, const void* wkv_b,
                                               const int32_t* row_count, void* kv, uint32_t* error_word,
                                               mla_stream_t stream) {
  return mla::prefill::expand(desc, rows, wkv_b, row_count, kv, error_word, (cudaStream_t)stream);
}
