// Key / value expansion: per-head keys and values of cached rows, the product
// of the latents with the model's kv up-projection,
//
//   kv[t, h, j] = sum_c wkv_b[h, j, c] * rows[t, c]     t < rows, j < 256, c < 512
//
// one GEMM of M = rows, N = H * 256, K = 512 on tcgen05. A tile is 128 rows x
// one head (128 x 256, float32 accumulator of 256 TMEM columns, two of them, so
// that one tile is written while the next is computed); tiles are dealt to one
// persistent CTA per SM in runs, heads fastest, so that a CTA's row tile stays
// the same for a whole run of heads.
//
// Per row and head 262144 operations and 512 bytes written: compute bound for
// all but a few rows.
//
// Per CTA (192 threads): warps 0-3 epilogue (TMEM -> bf16 -> shared memory ->
// TMA store of 64-column boxes), warp 4 issues the MMAs, warp 5 loads (TMA).
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include "mla.h"
#include "mla_prefill.h"
#include "prefill.cuh"

namespace mla {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

namespace prefill {

constexpr int kExpThreads = 192;
constexpr int kExpStages = 4;
constexpr int kExpStageBytes = 3 * kBox;   // 128 rows and one head's 256 weight rows x 64 columns
constexpr int kExpSmem = 1024 + kExpStages * kExpStageBytes + 2 * kBox;
constexpr int kKBlocks = kDLatent / 64;

struct ExpandMaps {
  CUtensorMap rows;  // [num_rows, 512 of row_stride]
  CUtensorMap w;     // [H * 256, 512]
  CUtensorMap kv;    // [num_rows, H * 256]
};

struct ExpandArgs {
  const int32_t* row_count;  // device or nullptr
  __nv_bfloat16* kv;
  uint32_t* error;
  int num_rows, heads;
};

struct ExpandBars {
  uint64_t full[kExpStages], empty[kExpStages];
  uint64_t t_full[2], t_empty[2];
  uint64_t done;
  uint32_t tmem;
  uint32_t abort_flag;
};

MLA_DEV void epilogue_barrier() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
// The same, and whether every epilogue warp came with `ok`: after a wait that
// ran out they leave together, none left at a barrier.
MLA_DEV bool epilogue_all(bool ok) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.and.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(all)
      : "r"((uint32_t)ok)
      : "memory");
  return all != 0;
}

__global__ void __launch_bounds__(kExpThreads, 1)
    mla_expand_kv_kernel(const __grid_constant__ ExpandMaps maps, const ExpandArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ ExpandBars bars;
  const uint32_t ring = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t stage_out = ring + kExpStages * kExpStageBytes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Waiter W{&bars.abort_flag, a.error};
  const int rows = a.row_count ? min(max(__ldg(a.row_count), 0), a.num_rows) : a.num_rows;
  const long long tiles = (long long)((rows + 127) / 128) * a.heads;
  const long long per = (tiles + gridDim.x - 1) / gridDim.x;
  const long long i0 = min(blockIdx.x * per, tiles), i1 = min(i0 + per, tiles);
  if (i0 >= i1) return;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kExpStages; ++s) {
      mbar_init(smem_addr(&bars.full[s]), 1);
      mbar_init(smem_addr(&bars.empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_addr(&bars.t_full[b]), 1);
      mbar_init(smem_addr(&bars.t_empty[b]), 4);
    }
    mbar_init(smem_addr(&bars.done), 1);
    bars.abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == 4) {
    tmem_alloc(smem_addr(&bars.tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars.tmem;

  if (warp == 5) {
    if (lane == 0) {
      int n = 0;
      bool ok = true;
      for (long long i = i0; i < i1 && ok; ++i) {
        const int m0 = (int)(i / a.heads) * 128, h = (int)(i % a.heads);
        for (int k = 0; k < kKBlocks; ++k, ++n) {
          const int s = n % kExpStages;
          if (!(ok = W.wait(&bars.empty[s], ((n / kExpStages) & 1) ^ 1))) break;
          const uint32_t full = smem_addr(&bars.full[s]), st = ring + s * kExpStageBytes;
          mbar_arrive_expect_tx(full, kExpStageBytes);
          tma_load_2d(st, &maps.rows, 64 * k, m0, full);
          tma_load_2d(st + kBox, &maps.w, 64 * k, h * 256, full);
          tma_load_2d(st + 2 * kBox, &maps.w, 64 * k, h * 256 + 128, full);
        }
      }
      for (int d = max(0, n - kExpStages); d < n; ++d) W.wait(&bars.full[d % kExpStages], (d / kExpStages) & 1, true);
    }
    __syncwarp();
  } else if (warp == 4) {
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_bf16_f32(128, 256, 0, 0);
      int n = 0, nt = 0;
      bool ok = true;
      for (long long i = i0; i < i1 && ok; ++i, ++nt) {
        const int b = nt & 1;
        if (!(ok = W.wait(&bars.t_empty[b], ((nt >> 1) & 1) ^ 1))) break;
        for (int k = 0; k < kKBlocks; ++k, ++n) {
          const int s = n % kExpStages;
          if (!(ok = W.wait(&bars.full[s], (n / kExpStages) & 1))) break;
          tc_fence_after();
          const uint32_t st = ring + s * kExpStageBytes;
#pragma unroll
          for (int u = 0; u < 4; ++u)
            mma_ss(tmem + 256 * b, smem_desc_sw128(st + 32 * u, 16, 1024), smem_desc_sw128(st + kBox + 32 * u, 16, 1024),
                   idesc, (k > 0 || u > 0) ? 1u : 0u);
          mma_commit(smem_addr(&bars.empty[s]));
        }
        if (ok) mma_commit(smem_addr(&bars.t_full[b]));
      }
      mma_commit(smem_addr(&bars.done));
      W.wait(&bars.done, 0, true);
    }
    __syncwarp();
  } else {
    const int row = 32 * warp + lane;  // row of the tile = TMEM lane
    int nt = 0, nbox = 0;
    for (long long i = i0; i < i1; ++i, ++nt) {
      const int m0 = (int)(i / a.heads) * 128, h = (int)(i % a.heads), b = nt & 1;
      const bool full_tile = m0 + 128 <= rows;
      if (!epilogue_all(W.wait_warp(&bars.t_full[b], (nt >> 1) & 1))) break;
      tc_fence_after();
      const uint32_t acc = tmem + ((uint32_t)(32 * warp) << 16) + 256 * b;
#pragma unroll 1
      for (int c = 0; c < 4; ++c, ++nbox) {
        uint32_t r[2][32];
        tmem_ld_32x32b_32(acc + 64 * c, r[0]);
        tmem_ld_32x32b_32(acc + 64 * c + 32, r[1]);
        tmem_wait_ld();
        if (c == 3) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&bars.t_empty[b]));
        }
        const uint32_t box = stage_out + (nbox & 1) * kBox;
        // the store that read this box two boxes ago is done with it
        if (threadIdx.x == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
        epilogue_barrier();
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int u = 0; u < 4; ++u)
            st_shared_v4(box + row * 128 + (((uint32_t)(4 * x + u) ^ (uint32_t)(row & 7)) << 4),
                         make_uint4(pack_bf16x2(__uint_as_float(r[x][8 * u + 0]), __uint_as_float(r[x][8 * u + 1])),
                                    pack_bf16x2(__uint_as_float(r[x][8 * u + 2]), __uint_as_float(r[x][8 * u + 3])),
                                    pack_bf16x2(__uint_as_float(r[x][8 * u + 4]), __uint_as_float(r[x][8 * u + 5])),
                                    pack_bf16x2(__uint_as_float(r[x][8 * u + 6]), __uint_as_float(r[x][8 * u + 7]))));
        if (full_tile) {
          fence_proxy_async_smem();
          epilogue_barrier();
          if (threadIdx.x == 0) {
            tma_store_2d(&maps.kv, box, h * 256 + 64 * c, m0);
            bulk_commit();
          }
        } else {
          // the last rows: only those below the count are written, 8 lanes per row
          __syncwarp();
#pragma unroll 1
          for (int g = 0; g < 8; ++g) {
            const int rr = 32 * warp + 4 * g + (lane >> 3), j = lane & 7;
            const uint4 v = ld_shared_v4(box + rr * 128 + ((uint32_t)(j ^ (rr & 7)) << 4));
            if (m0 + rr < rows)
              *reinterpret_cast<uint4*>(a.kv + ((size_t)(m0 + rr) * a.heads + h) * 256 + 64 * c + 8 * j) = v;
          }
        }
      }
    }
    if (threadIdx.x == 0) bulk_wait_read();  // shared memory is read before the CTA can exit
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 4) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
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
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return MLA_ERR_CUDA;
  }
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) return MLA_ERR_CUDA;
  const auto encode = [&](CUtensorMap* m, const void* p, long long cols, long long n, long long stride) {
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)n}, strides[1] = {(cuuint64_t)stride * 2};
    cuuint32_t box[2] = {64, 128}, elem[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(p), dims, strides, box, elem,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  ExpandMaps maps;
  const long long width = (long long)d->num_heads * 256;
  if (!encode(&maps.rows, rows, kDLatent, d->num_rows, d->row_stride) ||
      !encode(&maps.w, wkv_b, kDLatent, width, kDLatent) || !encode(&maps.kv, kv, width, d->num_rows, width))
    return MLA_ERR_CUDA;
  if (cudaFuncSetAttribute((const void*)mla_expand_kv_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kExpSmem) !=
      cudaSuccess)
    return MLA_ERR_CUDA;
  ExpandArgs a{row_count, static_cast<__nv_bfloat16*>(kv), error, d->num_rows, d->num_heads};
  const long long tiles = (long long)((d->num_rows + 127) / 128) * d->num_heads;
  mla_expand_kv_kernel<<<(int)(tiles < sms ? tiles : sms), kExpThreads, kExpSmem, stream>>>(maps, a);
  return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // namespace prefill
}  // namespace mla

extern "C" MLA_API mla_status_t mlap_expand_kv(const mlap_expand_desc_t* desc, const void* rows, const void* wkv_b,
                                               const int32_t* row_count, void* kv, uint32_t* error_word,
                                               mla_stream_t stream) {
  return mla::prefill::expand(desc, rows, wkv_b, row_count, kv, error_word, (cudaStream_t)stream);
}
