// Ragged attention of new tokens over expanded per-head keys (128 + 64 rope)
// and values (128), as one persistent tcgen05 kernel and a merge of split rows.
//
// For a sequence's query i, key t and head h, with the exponentials taken
// relative to a running maximum m of the row:
//   s_t = scale * q . k_t,  p_t = exp(s_t - m),  l = sum_t p_t,  o = sum_t p_t v_t
//   out = o / l,  lse = m + ln l
// one pass over the keys; when m grows, o and l are scaled by exp(m_old - m).
//
// Work. An item is (sequence, block of 256 queries, head); its units are its
// visible 128-key tiles. All units are laid end to end (sequence, block, head,
// tile) and cut into one equal run per SM, so that every SM gets the same work
// whatever the lengths. With blocks before heads, SMs that work on different
// blocks of one sequence reach the same head, and so the same keys, at about
// the same time and share them in L2. An item cut by a run boundary leaves
// float32 partials with their own lse, merged by the second kernel.
//
// Per CTA (320 threads), two query tiles of 128 rows share each key tile:
//   warps 0-3, 4-7  softmax of query tile 0 / 1, one thread per row: S from
//                   TMEM, mask, maximum, exponentials, P (bf16) back over S in
//                   TMEM; rescales O when the maximum grew by more than 2^8;
//                   writes the finished rows
//   warp 8          tcgen05 issuer: S_t = Q_t K^T (M 128, N 128, K 192, both from
//                   shared memory), O_t += P_t V (P from TMEM, V read MN-major)
//   warp 9          producer: Q tiles and K / V boxes by TMA; a ring of eight
//                   16 KB boxes (128 rows x 64 columns): a key tile is K (two
//                   boxes), k_pe (one), V (two)
// The issuer alternates P_0 V, S_0, P_1 V, S_1, so that one tile's softmax runs
// under the other's products. TMEM: S_0 S_1 (128 columns each, P in the lower
// 64), O_0 O_1 (128 each): all 512 columns.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <math.h>

#include "mla.h"
#include "mla_prefill.h"
#include "prefill.cuh"

namespace mla {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

namespace prefill {

constexpr int kAttnThreads = 320;
constexpr int kTile = 128;                 // rows of a query tile, keys of a key tile
constexpr int kBlockQ = 2 * kTile;         // queries of an item
constexpr int kRing = 8;
constexpr int kQBoxes = 6;
constexpr int kAttnSmem = 1024 + (kQBoxes + kRing) * kBox;
constexpr uint32_t kTmemS = 0, kTmemO = 256, kTmemAll = 512;
constexpr float kGrowth = 8.0f;            // log2: O is rescaled when a row's maximum grew by more (p stays below 2^8)
constexpr float kLn2 = 0.6931471805599453f;

// What the merge kernel needs about the item that run w starts and does not
// finish: the number of runs it spans (0: none), its first query row, rows, head.
struct SplitInfo {
  int32_t pieces, row, rows, head;
};

struct AttnArgs {
  const int32_t* cu_q;
  const int32_t* cu_k;
  __nv_bfloat16* out;  // [num_q, H, 128]
  float* lse;          // [num_q, H]
  SplitInfo* info;     // [workers]
  float* part_lse;     // [2 * workers, 256]
  float* part_o;       // [2 * workers, 256, 128]
  uint32_t* error;
  int batch, heads, num_q, num_k, causal, workers;
  float scale, scale_log2;
};

struct AttnMaps {
  CUtensorMap q;   // [num_q, H * 192] boxes of 128 x 64
  CUtensorMap kv;  // [num_k, H * 256]
  CUtensorMap pe;  // [num_k, 64]
};

MLA_DEV int ceil_tiles(int keys) { return (keys + kTile - 1) >> 7; }  // also for negative counts

// One sequence: query rows [q0, q0 + n), key rows [k0, k0 + L).
struct Seq {
  int q0, n, k0, L;
  MLA_DEV void load(const AttnArgs& a, int b) {
    n = ragged_range(a.cu_q, b, a.num_q, &q0);
    L = ragged_range(a.cu_k, b, a.num_k, &k0);
  }
  MLA_DEV int blocks() const { return (n + kBlockQ - 1) / kBlockQ; }
  // keys visible to the last of the first `rows` queries
  MLA_DEV int visible(int rows, int causal) const {
    return causal ? max(min(L, L - n + min(n, rows)), 0) : L;
  }
  // key tiles worked on for queries below `rows`: at least one, so that rows
  // without keys are written too
  MLA_DEV int tiles(int rows, int causal) const { return max(1, ceil_tiles(visible(rows, causal))); }
  // tiles of the first m blocks of one head. Causal block x (from 1) short of
  // the last has max(1, c + 2x) tiles, c = ceil((L - n) / 128): the first
  // k = max(0, -c / 2) of them one each, the others an arithmetic series.
  MLA_DEV long long tiles_before(int m, int causal) const {
    if (m <= 0) return 0;
    const int last = tiles(n, causal);
    if (!causal) return (long long)m * last;
    const int full = m == blocks() ? m - 1 : m;
    const long long c = ceil_tiles(L - n);
    const long long k = min((long long)full, max(0ll, -c / 2));
    return k + (full - k) * c + ((long long)full * (full + 1) - k * (k + 1)) + (m == full ? 0 : last);
  }
};

// Position of a run in the list of items.
struct Cursor {
  long long u, end;  // next unit, end of the run
  Seq s;
  int b, qb, h, t0, tiles;
  MLA_DEV bool more() const { return u < end; }
  MLA_DEV int t1() const { return (int)min((long long)tiles, t0 + (end - u)); }
  MLA_DEV void next(const AttnArgs& a) {
    u += t1() - t0;
    t0 = 0;
    if (!more()) return;
    if (++h < a.heads) return;
    h = 0;
    if (++qb >= s.blocks()) {
      qb = 0;
      do {
        ++b;
        s.load(a, b);
      } while (s.n == 0 && b + 1 < a.batch);
    }
    tiles = s.tiles((qb + 1) * kBlockQ, a.causal);
  }
};

// Run `w`: called by a whole warp. Two passes over the sequences, 32 at a time.
MLA_DEV long long run_start(const AttnArgs& a, int w, Cursor* cur) {
  const int lane = threadIdx.x & 31;
  long long total = 0;
  bool bad = false;
  for (int b = lane; b < a.batch; b += 32) {
    Seq s;
    s.load(a, b);
    total += s.tiles_before(s.blocks(), a.causal) * a.heads;
    const int oq = __ldg(a.cu_q + b), ok = __ldg(a.cu_k + b);
    bad |= oq != s.q0 || ok != s.k0 || __ldg(a.cu_q + b + 1) != s.q0 + s.n || __ldg(a.cu_k + b + 1) != s.k0 + s.L;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(~0u, total, o);
  if (w == 0 && bad) set_error(a.error, kErrSeqLen);
  const long long quota = max(1ll, (total + a.workers - 1) / a.workers);
  cur->u = min((long long)w * quota, total);
  cur->end = min(cur->u + quota, total);
  cur->s = Seq{0, 0, 0, 0};
  cur->b = cur->qb = cur->h = cur->t0 = 0;
  cur->tiles = 1;
  if (!cur->more()) return quota;
  long long before = 0;
  for (int b0 = 0; b0 < a.batch; b0 += 32) {
    Seq s{0, 0, 0, 0};
    const int b = b0 + lane;
    if (b < a.batch) s.load(a, b);
    const long long own = s.tiles_before(s.blocks(), a.causal) * a.heads;
    long long incl = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(~0u, incl, o);
      if (lane >= o) incl += y;
    }
    const unsigned beyond = __ballot_sync(~0u, before + incl > cur->u);
    if (beyond) {
      const int src = __ffs(beyond) - 1;
      cur->b = b0 + src;
      cur->s.q0 = __shfl_sync(~0u, s.q0, src);
      cur->s.n = __shfl_sync(~0u, s.n, src);
      cur->s.k0 = __shfl_sync(~0u, s.k0, src);
      cur->s.L = __shfl_sync(~0u, s.L, src);
      const long long rest = cur->u - before - __shfl_sync(~0u, incl - own, src);
      int lo = 0, hi = cur->s.blocks() - 1;  // the last block that starts at or before `rest`
      while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (cur->s.tiles_before(mid, a.causal) * a.heads <= rest) lo = mid;
        else hi = mid - 1;
      }
      cur->qb = lo;
      cur->tiles = cur->s.tiles((lo + 1) * kBlockQ, a.causal);
      const long long in_block = rest - cur->s.tiles_before(lo, a.causal) * a.heads;
      cur->h = (int)(in_block / cur->tiles);
      cur->t0 = (int)(in_block % cur->tiles);
      return quota;
    }
    before += __shfl_sync(~0u, incl, 31);
  }
  cur->end = cur->u;  // not reached: the units add up to the total
  return quota;
}

struct AttnBars {
  uint64_t full[kRing], empty[kRing];
  uint64_t q_full, q_empty;
  uint64_t s_full[2], p_full[2], o_full[2];
  uint64_t done;
  Cursor start;
  long long quota;
  uint32_t tmem;
  uint32_t abort_flag;
};

MLA_DEV float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

__global__ void __launch_bounds__(kAttnThreads, 1)
    mla_prefill_attention_kernel(const __grid_constant__ AttnMaps maps, const AttnArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ AttnBars bars;
  const uint32_t qbuf = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t ring = qbuf + kQBoxes * kBox;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Waiter W{&bars.abort_flag, a.error};

  if (threadIdx.x == 0) {
    for (int s = 0; s < kRing; ++s) {
      mbar_init(smem_addr(&bars.full[s]), 1);
      mbar_init(smem_addr(&bars.empty[s]), 1);
    }
    mbar_init(smem_addr(&bars.q_full), 1);
    mbar_init(smem_addr(&bars.q_empty), 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(smem_addr(&bars.s_full[t]), 1);
      mbar_init(smem_addr(&bars.p_full[t]), 4);  // the four softmax warps of the tile
      mbar_init(smem_addr(&bars.o_full[t]), 1);
    }
    mbar_init(smem_addr(&bars.done), 1);
    bars.abort_flag = 0u;
    fence_mbar_init();
    a.info[blockIdx.x].pieces = 0;
  }
  if (warp == 8) {
    tmem_alloc(smem_addr(&bars.tmem), kTmemAll);
    tmem_relinquish();
  }
  if (warp == 9) {
    Cursor c;
    const long long quota = run_start(a, blockIdx.x, &c);
    if (lane == 0) {
      bars.start = c;
      bars.quota = quota;
      prefetch_tmap(&maps.q);
      prefetch_tmap(&maps.kv);
      prefetch_tmap(&maps.pe);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars.tmem;
  Cursor cur = bars.start;

  if (warp == 9) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      int nb = 0, nq = 0;  // boxes and query blocks whose loads were issued
      bool ok = true;
      for (; cur.more() && ok; cur.next(a)) {
        const int rows = cur.s.n - cur.qb * kBlockQ;
        if (!W.wait(&bars.q_empty, (nq & 1) ^ 1)) break;
        const int boxes = rows > kTile ? 6 : 3;
        mbar_arrive_expect_tx(smem_addr(&bars.q_full), boxes * kBox);
        for (int x = 0; x < boxes; ++x)
          tma_load_2d(qbuf + x * kBox, &maps.q, cur.h * 192 + 64 * (x % 3),
                      cur.s.q0 + cur.qb * kBlockQ + kTile * (x / 3), smem_addr(&bars.q_full));
        ++nq;
        const int t1 = cur.t1();
        for (int j = cur.t0; j < t1 && ok; ++j) {
          const int row = cur.s.k0 + j * kTile;
          for (int x = 0; x < 5; ++x) {  // K, K, k_pe, V, V
            const int s = nb % kRing;
            if (!(ok = W.wait(&bars.empty[s], ((nb / kRing) & 1) ^ 1))) break;
            const uint32_t full = smem_addr(&bars.full[s]);
            mbar_arrive_expect_tx(full, kBox);
            if (x == 2) tma_load_2d(ring + s * kBox, &maps.pe, 0, row, full);
            else tma_load_2d(ring + s * kBox, &maps.kv, cur.h * 256 + 64 * (x < 2 ? x : x - 1), row, full);
            ++nb;
          }
        }
      }
      // every issued copy lands before the CTA can exit
      for (int i = max(0, nb - kRing); i < nb; ++i) W.wait(&bars.full[i % kRing], (i / kRing) & 1, true);
      if (nq > 0) W.wait(&bars.q_full, (nq - 1) & 1, true);
    }
    __syncwarp();
  } else if (warp == 8) {
    // ------------------------------------------------------------ MMA issuer
    // The whole warp walks the loop (it clears value rows together); lane 0 issues.
    constexpr uint32_t idesc_s = idesc_bf16_f32(128, 128, 0, 0);
    constexpr uint32_t idesc_o = idesc_bf16_f32(128, 128, 0, 1);
    constexpr uint32_t idesc_half = idesc_bf16_f32(128, 64, 0, 1);
    int nb = 0, nq = 0;        // boxes and query blocks consumed
    int np[2] = {0, 0};        // P tiles consumed
    bool ok = true;
    const auto box = [&](int i) { return ring + (uint32_t)(i % kRing) * kBox; };
    const auto wait_boxes = [&](int first, int count) {
      bool good = true;
      for (int i = first; i < first + count && good; ++i) good = W.wait_warp(&bars.full[i % kRing], (i / kRing) & 1);
      return good;
    };
    const auto scores = [&](int t, int k) {  // S_t = Q_t K^T, K in boxes k .. k + 2
      if (lane == 0) {
#pragma unroll
        for (int u = 0; u < 12; ++u)
          mma_ss(tmem + kTmemS + 128 * t, smem_desc_sw128(qbuf + (3 * t + (u >> 2)) * kBox + (u & 3) * 32, 16, 1024),
                 smem_desc_sw128(box(k + (u >> 2)) + (u & 3) * 32, 16, 1024), idesc_s, u > 0 ? 1u : 0u);
        mma_commit(smem_addr(&bars.s_full[t]));
      }
    };
    const auto release = [&](int first, int count) {
      if (lane == 0)
        for (int i = first; i < first + count; ++i) mma_commit(smem_addr(&bars.empty[i % kRing]));
    };
    for (; cur.more() && ok; cur.next(a)) {
      const int t1 = cur.t1(), r0 = cur.qb * kBlockQ;
      int e[2];
      e[0] = min(t1, cur.s.tiles(r0 + kTile, a.causal));
      e[1] = cur.s.n > r0 + kTile ? t1 : 0;
      if (!(ok = W.wait_warp(&bars.q_full, nq & 1))) break;
      ++nq;
      if (!(ok = wait_boxes(nb, 3))) break;
      tc_fence_after();
      for (int t = 0; t < 2; ++t)
        if (cur.t0 < e[t]) scores(t, nb);
      release(nb, 3);
      for (int j = cur.t0; j < t1 && ok; ++j) {
        const int v = nb + 3, k_next = nb + 5;  // this tile's V boxes, the next tile's K boxes
        bool v_ready = false, k_ready = false;
        for (int t = 0; t < 2 && ok; ++t) {
          if (j < e[t]) {
            if (!v_ready) {
              if (!(ok = wait_boxes(v, 2))) break;
              const int valid = cur.s.L - j * kTile;
              if (valid < kTile) {
                // value rows behind the sequence's end: 0 * NaN is NaN, so they are cleared
                for (int i = max(valid, 0) * 8 + lane; i < kTile * 8; i += 32) {
                  st_shared_v4(box(v) + 16 * i, make_uint4(0, 0, 0, 0));
                  st_shared_v4(box(v + 1) + 16 * i, make_uint4(0, 0, 0, 0));
                }
                fence_proxy_async_smem();
                __syncwarp();
              }
              v_ready = true;
            }
            if (!(ok = W.wait_warp(&bars.p_full[t], np[t] & 1))) break;
            ++np[t];
            tc_fence_after();
            if (lane == 0) {
              const uint32_t o = tmem + kTmemO + 128 * t, p = tmem + kTmemS + 128 * t;
              if (v % kRing != kRing - 1) {
#pragma unroll
                for (int u = 0; u < 8; ++u)
                  mma_tmem_a(o, p + 8 * u, smem_desc_sw128(box(v) + 2048 * u, kBox, 1024), idesc_o,
                             (j > cur.t0 || u > 0) ? 1u : 0u);
              } else {  // the two boxes are the ring's last and first: one half at a time
#pragma unroll
                for (int u = 0; u < 8; ++u)
#pragma unroll
                  for (int x = 0; x < 2; ++x)
                    mma_tmem_a(o + 64 * x, p + 8 * u, smem_desc_sw128(box(v + x) + 2048 * u, kBox, 1024), idesc_half,
                               (j > cur.t0 || u > 0) ? 1u : 0u);
              }
              mma_commit(smem_addr(&bars.o_full[t]));
            }
          }
          if (t == 1) release(v, 2);
          if (j + 1 < e[t]) {
            if (!k_ready) {
              if (!(ok = wait_boxes(k_next, 3))) break;
              tc_fence_after();
              k_ready = true;
            }
            scores(t, k_next);
          }
        }
        if (ok && j + 1 < t1) release(k_next, 3);
        nb += 5;
      }
      if (ok && lane == 0) mma_commit(smem_addr(&bars.q_empty));
    }
    if (lane == 0) {
      mma_commit(smem_addr(&bars.done));
      W.wait(&bars.done, 0, true);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax
    const int t = warp >> 2;                           // query tile
    const int row = (warp & 3) * 32 + lane;            // row of the tile = TMEM lane
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t st = tmem + lanes + kTmemS + 128 * t, ot = tmem + lanes + kTmemO + 128 * t;
    int ns = 0;                                        // S tiles consumed = P tiles made
    bool ok = true;
    for (; cur.more() && ok; cur.next(a)) {
      const int t1 = cur.t1(), r0 = cur.qb * kBlockQ + kTile * t;
      if (threadIdx.x == 0 && cur.t0 == 0 && t1 < cur.tiles) {
        // the item goes on in the following runs
        const long long last = (cur.u + cur.tiles - 1) / bars.quota;
        a.info[blockIdx.x] = SplitInfo{(int)(last - blockIdx.x) + 1, cur.s.q0 + cur.qb * kBlockQ,
                                       min(cur.s.n - cur.qb * kBlockQ, kBlockQ), cur.h};
      }
      if (r0 >= cur.s.n) continue;
      const int e = min(t1, cur.s.tiles(r0 + kTile, a.causal));
      const int i = r0 + row;                          // query of the sequence
      const int limit = a.causal ? min(cur.s.L, cur.s.L - cur.s.n + i + 1) : cur.s.L;  // keys it sees
      float m = -INFINITY, l = 0.f;                    // reference maximum (raw scores), sum of exponentials
      for (int j = cur.t0; j < e; ++j) {
        if (!(ok = W.wait_warp(&bars.s_full[t], ns & 1))) break;
        tc_fence_after();
        uint32_t s[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld_32x32b_32(st + 32 * c, s[c]);
        tmem_wait_ld();
        const int seen = limit - j * kTile;
        if (!__all_sync(~0u, seen >= kTile)) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int x = 0; x < 32; ++x)
              if (32 * c + x >= seen) s[c][x] = 0xff800000u;  // -inf
        }
        float mx[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          mx[c] = __uint_as_float(s[c][0]);
#pragma unroll
          for (int x = 1; x < 31; x += 2) mx[c] = max3(mx[c], __uint_as_float(s[c][x]), __uint_as_float(s[c][x + 1]));
          mx[c] = fmaxf(mx[c], __uint_as_float(s[c][31]));
        }
        const float top = fmaxf(fmaxf(m, fmaxf(mx[0], mx[1])), fmaxf(mx[2], mx[3]));
        const bool grow = j > cur.t0 && (top - m) * a.scale_log2 > kGrowth;  // false while both are -inf (NaN)
        if (j == cur.t0) {
          m = top;
        } else if (__any_sync(~0u, grow)) {
          const float f = grow ? ex2((m - top) * a.scale_log2) : 1.f;
          if (!(ok = W.wait_warp(&bars.o_full[t], (ns - 1) & 1))) break;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t o[32];
            tmem_ld_32x32b_32(ot + 32 * c, o);
            tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
            tmem_st_32(ot + 32 * c, o);
          }
          l *= f;
          if (grow) m = top;
        }
        const float shift = m == -INFINITY ? 0.f : -m * a.scale_log2;
        const float2 k2 = make_float2(a.scale_log2, a.scale_log2), b2 = make_float2(shift, shift);
        float2 sum[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          sum[c] = make_float2(0.f, 0.f);
#pragma unroll
          for (int x = 0; x < 32; x += 2) {
            const float2 y = fma2_rn(make_float2(__uint_as_float(s[c][x]), __uint_as_float(s[c][x + 1])), k2, b2);
            const float2 p = make_float2(ex2(y.x), ex2(y.y));
            sum[c] = add2_rn(sum[c], p);
            s[c >> 1][(c & 1) * 16 + x / 2] = pack_bf16x2(p.x, p.y);
          }
          if (c & 1) tmem_st_32(st + 32 * (c >> 1), s[c >> 1]);
        }
        const float2 s01 = add2_rn(add2_rn(sum[0], sum[1]), add2_rn(sum[2], sum[3]));
        l += s01.x + s01.y;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&bars.p_full[t]));
        ++ns;
      }
      if (!ok) break;
      // finished rows, or this run's part of them
      const bool whole = cur.t0 == 0 && t1 == cur.tiles;
      const bool valid = i < cur.s.n;
      const float inv = l > 0.f ? 1.f / l : 0.f;
      const float lse = l > 0.f ? m * a.scale + logf(l) : -INFINITY;
      const size_t slot = (size_t)2 * blockIdx.x + (cur.t0 == 0 ? 1 : 0);
      const int prow = kTile * t + row;
      __nv_bfloat16* dst = a.out + ((size_t)(cur.s.q0 + i) * a.heads + cur.h) * 128;
      float* part = a.part_o + (slot * kBlockQ + prow) * 128;
      if (cur.t0 < e) {
        if (!(ok = W.wait_warp(&bars.o_full[t], (ns - 1) & 1))) break;
        tc_fence_after();
      }
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t o[32];
        if (cur.t0 < e) {
          tmem_ld_32x32b_32(ot + 32 * c, o);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int x = 0; x < 32; ++x) o[x] = 0u;
        }
        if (!valid) continue;
        // a row without keys: its products are all 0 * v
        if (whole) {
          uint4* d4 = reinterpret_cast<uint4*>(dst + 32 * c);
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            uint32_t w[4];
#pragma unroll
            for (int x = 0; x < 4; ++x)
              w[x] = pack_bf16x2(__uint_as_float(o[8 * u + 2 * x]) * inv, __uint_as_float(o[8 * u + 2 * x + 1]) * inv);
            d4[u] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        } else {
          float4* d4 = reinterpret_cast<float4*>(part + 32 * c);
#pragma unroll
          for (int u = 0; u < 8; ++u)
            d4[u] = make_float4(__uint_as_float(o[4 * u]) * inv, __uint_as_float(o[4 * u + 1]) * inv,
                                __uint_as_float(o[4 * u + 2]) * inv, __uint_as_float(o[4 * u + 3]) * inv);
        }
      }
      if (valid) {
        if (whole) a.lse[(size_t)(cur.s.q0 + i) * a.heads + cur.h] = lse;
        else a.part_lse[slot * kBlockQ + prow] = lse;
      }
    }
    __syncwarp();
  }

  allow_dependents();  // the merge kernel's blocks may take SMs as these CTAs finish
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemAll);
  }
}

// Merge of split items: block (w, g) joins 16 rows of the item that run w
// starts and does not finish. Its parts are run w's second slot and the first
// slots of the following runs; a thread holds 16 of a row's 128 columns.
constexpr int kMergeRows = 16;
__global__ void __launch_bounds__(128) mla_prefill_merge_kernel(const AttnArgs a) {
  grid_dependency_wait();
  const int w = blockIdx.x;
  const SplitInfo it = a.info[w];
  const int row = blockIdx.y * kMergeRows + (threadIdx.x >> 3), col = (threadIdx.x & 7) * 16;
  const int pieces = min(it.pieces, a.workers - w);
  if (pieces < 1 || row >= it.rows) return;
  const auto slot = [&](int p) { return (size_t)(p == 0 ? 2 * w + 1 : 2 * (w + p)) * kBlockQ + row; };
  float m = -INFINITY;
  for (int p = 0; p < pieces; ++p) m = fmaxf(m, a.part_lse[slot(p)]);
  float acc[16], sum = 0.f;
#pragma unroll
  for (int x = 0; x < 16; ++x) acc[x] = 0.f;
  if (m != -INFINITY) {
    for (int p = 0; p < pieces; ++p) {
      const size_t at = slot(p);
      const float lse = a.part_lse[at];
      if (lse == -INFINITY) continue;
      const float f = expf(lse - m);
      sum += f;
      const float4* src = reinterpret_cast<const float4*>(a.part_o + at * 128 + col);
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float4 v = src[x];
        acc[4 * x] += f * v.x;
        acc[4 * x + 1] += f * v.y;
        acc[4 * x + 2] += f * v.z;
        acc[4 * x + 3] += f * v.w;
      }
    }
  }
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  const size_t r = (size_t)(it.row + row) * a.heads + it.head;
  uint4* dst = reinterpret_cast<uint4*>(a.out + r * 128 + col);
#pragma unroll
  for (int x = 0; x < 2; ++x)
    dst[x] = make_uint4(pack_bf16x2(acc[8 * x] * inv, acc[8 * x + 1] * inv),
                        pack_bf16x2(acc[8 * x + 2] * inv, acc[8 * x + 3] * inv),
                        pack_bf16x2(acc[8 * x + 4] * inv, acc[8 * x + 5] * inv),
                        pack_bf16x2(acc[8 * x + 6] * inv, acc[8 * x + 7] * inv));
  if (col == 0) a.lse[r] = sum > 0.f ? m + logf(sum) : -INFINITY;
}

mla_status_t check_attention(const mlap_attention_desc_t* d) {
  if (!d) return MLA_ERR_INVALID_ARG;
  if (d->batch < 0 || d->num_heads < 1 || d->num_q < 0 || d->num_k < 0 || (d->causal != 0 && d->causal != 1) ||
      d->num_sms < 0 || d->pe_stride < kDRope || !(d->softmax_scale > 0.f) || !isfinite(d->softmax_scale))
    return MLA_ERR_INVALID_ARG;
  if (d->num_heads > kMaxHeads || d->d_nope != 128 || d->d_rope != kDRope || d->d_v != 128 || d->pe_stride % 8 != 0)
    return MLA_ERR_UNSUPPORTED;
  // row indexes and tile counts are 32-bit
  if (d->num_q > 0x7fffffff - kBlockQ || d->num_k > 0x7fffffff - kTile) return MLA_ERR_UNSUPPORTED;
  return MLA_OK;
}

// Workers (one per SM) of the current device for this descriptor; 0 on a CUDA error.
int attention_workers(const mlap_attention_desc_t* d) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return d->num_sms > 0 && d->num_sms < sms ? d->num_sms : sms;
}

// Workspace: [SplitInfo | part_lse | part_o], each a multiple of 256 bytes.
size_t info_bytes(int workers) { return ((size_t)workers * sizeof(SplitInfo) + 255) & ~(size_t)255; }
size_t part_lse_bytes(int workers) { return (size_t)2 * workers * kBlockQ * sizeof(float); }
size_t workspace_bytes(int workers) {
  return info_bytes(workers) + part_lse_bytes(workers) + (size_t)2 * workers * kBlockQ * 128 * sizeof(float);
}

bool encode_rows(CUtensorMap* m, const void* p, long long cols, long long rows, long long stride) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)stride * 2};
  cuuint32_t box[2] = {64, kTile}, elem[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(p), dims, strides, box, elem,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

mla_status_t attention(const mlap_attention_desc_t* d, const void* q, const void* kv, const void* k_pe,
                       const int32_t* cu_q, const int32_t* cu_k, void* out, float* lse, void* workspace,
                       size_t ws_bytes, uint32_t* error, cudaStream_t stream) {
  const mla_status_t st = check_attention(d);
  if (st != MLA_OK) return st;
  if (d->batch == 0 || d->num_q == 0) return MLA_OK;
  if (!q || !cu_q || !cu_k || !out || !lse || !workspace || (d->num_k > 0 && (!kv || !k_pe))) return MLA_ERR_INVALID_ARG;
  const auto off = [](const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) != 0; };
  if (off(q, 16) || off(kv, 16) || off(k_pe, 16) || off(out, 16) || off(workspace, 16) || off(cu_q, 4) ||
      off(cu_k, 4) || off(lse, 4) || off(error, 4))
    return MLA_ERR_INVALID_ARG;
  const int workers = attention_workers(d);
  if (workers == 0) return MLA_ERR_CUDA;
  if (ws_bytes < workspace_bytes(workers)) return MLA_ERR_WORKSPACE_TOO_SMALL;
  AttnMaps maps;
  // without keys the boxes still load (all masked): any valid memory does
  const bool keys = d->num_k > 0;
  if (!encode_rows(&maps.q, q, (long long)d->num_heads * 192, d->num_q, (long long)d->num_heads * 192) ||
      !encode_rows(&maps.kv, keys ? kv : q, keys ? (long long)d->num_heads * 256 : 64, keys ? d->num_k : 1,
                   keys ? (long long)d->num_heads * 256 : 64) ||
      !encode_rows(&maps.pe, keys ? k_pe : q, 64, keys ? d->num_k : 1, keys ? d->pe_stride : 64))
    return MLA_ERR_CUDA;
  AttnArgs a;
  a.cu_q = cu_q;
  a.cu_k = cu_k;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.info = reinterpret_cast<SplitInfo*>(ws);
  a.part_lse = reinterpret_cast<float*>(ws + info_bytes(workers));
  a.part_o = reinterpret_cast<float*>(ws + info_bytes(workers) + part_lse_bytes(workers));
  a.error = error;
  a.batch = d->batch;
  a.heads = d->num_heads;
  a.num_q = d->num_q;
  a.num_k = d->num_k;
  a.causal = d->causal;
  a.workers = workers;
  a.scale = d->softmax_scale;
  a.scale_log2 = d->softmax_scale * 1.4426950408889634f;
  if (cudaFuncSetAttribute((const void*)mla_prefill_attention_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           kAttnSmem) != cudaSuccess)
    return MLA_ERR_CUDA;
  mla_prefill_attention_kernel<<<workers, kAttnThreads, kAttnSmem, stream>>>(maps, a);
  if (cudaGetLastError() != cudaSuccess) return MLA_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(workers, kBlockQ / kMergeRows, 1);
  cfg.blockDim = dim3(128, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, mla_prefill_merge_kernel, a) == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // namespace prefill
}  // namespace mla

extern "C" MLA_API size_t mlap_attention_workspace_bytes(const mlap_attention_desc_t* desc) {
  using namespace mla::prefill;
  if (check_attention(desc) != MLA_OK) return 0;
  const int workers = attention_workers(desc);
  return workers > 0 ? workspace_bytes(workers) : 0;
}

extern "C" MLA_API mla_status_t mlap_attention(const mlap_attention_desc_t* desc, const void* q, const void* kv,
                                               const void* k_pe, const int32_t* cu_q, const int32_t* cu_k, void* out,
                                               float* lse, void* workspace, size_t workspace_bytes,
                                               uint32_t* error_word, mla_stream_t stream) {
  return mla::prefill::attention(desc, q, kv, k_pe, cu_q, cu_k, out, lse, workspace, workspace_bytes, error_word,
                                 (cudaStream_t)stream);
}
