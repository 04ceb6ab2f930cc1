// Ragged attention of new tokens over expanded per-head keys (128 + 64 rope)
// and values (128), as one persistent tcgen05 kernel and a merge of split rows.
//
// For a sequence's query i, key t and head h, with the exponentials taken
// relative to a running maximum m of the row:
//   s_t = scale * q . k_t,  p_t = exp(s_t - m),  l = sum_t p_t,  o = sum_t p_t v_t
//   out = o / l,  lse = m + ln l
// one pass over the keys; when m grows, o and l are scaled by exp(m_old - m).
// A row without a key has l = 0: out = 0, lse = -inf. A NaN or an infinity in q
// makes l NaN, or 0 where every score is -inf: out = NaN, lse = NaN. Hence l is
// compared with 0 and never tested for being above it, and a row with l = 0 is
// taken for one without keys only if none is visible to it (`blind`).
//
// Work. An item is (sequence, block of 256 queries, head); its units are its
// visible 128-key tiles, and kItemUnits more for what an item costs beside its
// tiles (Q, filling the pipeline, its rows; without them the runs of six prompts
// of 645 to 1491 tokens, 16 heads, took from 52 to 93 us, and the call 90 us
// instead of 78). All units are laid end to end and cut into one equal run per
// CTA pair, so that every SM gets the same work whatever the lengths. The order
// is (sequence, group of heads, block, head of the group, tile), with groups of
// about as many heads as a run has items: pairs then work on the different
// blocks of one sequence with the same heads, and so the same keys, at about the
// same time, and share them in L2 (128 heads, 2048 queries over 16384 keys, without
// the rounds below: 2.05 ms, 2.14 with all heads in one group). An item cut by a run
// boundary leaves float32 partials with their own lse, merged by the second kernel.
// Where keys and values are many, whole items are dealt in rounds before the runs
// (rounds_of), which keeps the pairs in step: the same call reads 1.8 GB from HBM
// instead of 5.9, for 1.2 GB of inputs, and takes 1.89 ms instead of 2.05; 16
// heads, 16384 new tokens: 0.99 ms instead of 1.08; 32 heads, 2048 queries over
// 8192 keys: 239 us instead of 257. (Times of this comment, unless it says more:
// replayed graphs in bursts of 20 ms, at 1965 MHz. Under the power cap, 2 s of
// replays, these three take 2.17 for 2.42 ms, 1.13 for 1.25 ms, 275 for 301 us.)
//
// Where rounds begin, measured on both sides, causal unless said otherwise:
// - 64 MiB of keys and values. Below: 32 MiB (4096 new tokens, 16 heads) 86.9 us in
//   rounds, 85.0 in runs; 55 MiB (2048 over 3500, 32 heads) 101.9 and 102.1. Eight
//   calls at 64 MiB, 16 to 128 heads: 0.1 to 2.5 % less time in rounds (4096, 32
//   heads 156.8 for 160.8 us; 8192, 16 heads 274.0 for 280.6; 1024 over 2048, 64
//   heads 73.2 for 73.3), four from 70 to 128 MiB 1 to 5 % less. A measured size, not
//   L2's (126 MB).
// - four blocks. 1024 queries over 8192 keys, 128 heads: 508 us for 512, not causal
//   530 for 532. Two or three blocks go either way: 512 over 1024, 128 heads, 52.9
//   us in rounds for 51.6 in runs, 300 over 2000 81.6 for 80.0, four sequences of
//   512 over 4096 565 for 556; but 600 over 7000 335 for 337, 512 over 8192 285 for
//   296. They stay in runs.
// The host picks the kernel that knows rounds by num_q and num_k, which may be a
// capacity; on many short sequences, which have none, it costs 3 % (400 prompts of
// 300 tokens, 16 heads, 915 us for 888), from 1000 keys a sequence on nothing.
//
// A CTA pair (cta_group::2) works on a block: S = Q K^T and O += P V with M 256,
// 128 rows in each CTA. Each CTA loads half of every key tile (64 keys of K,
// 64 columns of V), so that a tile costs the pair's SMs 40 KB each and three
// tiles fit beside two Q buffers. TMEM of a CTA: O (128 columns), two S buffers
// of 128 and two P buffers (bf16) of 64. The two softmax warpgroups of a CTA take
// alternate tiles, one S and one P buffer each. A warpgroup frees its S as soon as
// it holds the scores in registers, so that the tensor cores make its next S
// while it works on this one, and P V follows when it comes: neither waits for
// the other's latency. (With P over S and three S buffers the loop S, softmax,
// P V, S bound: 1800 cycles a tile for 1280 of products. One CTA with two query
// tiles of one S each: 4400 cycles per 2560.)
//
// Per CTA (384 threads):
//   warps 0-3, 4-7  softmax of the even / odd key tiles, one thread per row: S
//                   from TMEM, mask, maximum, exponentials, P; O is rescaled when
//                   the row's maximum grew by more than 2^8 since its reference
//                   (which the two warpgroups hand on tile by tile); each writes
//                   half of the finished columns
//   warps 8, 11     (even CTA) tcgen05 issuers, one thread each: scores; values.
//                   The tensor core's queue is short, an issuer is held up while
//                   its products run: with one issuer its own waits and address
//                   arithmetic then left the tensor cores idle
//   warp 9          producer by TMA: Q, V of tile i, K of tile i + 3; walks the run
//                   and hands every item on to the other warps
//   warp 10         clears the value rows behind a sequence's end
//
// Bound by the tensor cores and the softmax behind them: 1280 cycles of products
// a tile, about 1650 taken (a warpgroup needs 2900 for its tile, 1024 of them
// exponentials, every second tile is its). 2048 queries over 16384 keys, 128
// heads, causal: 1.89 ms, 1.36 PFLOP/s; 2.17 ms, 1.19 PFLOP/s at 1.40 GHz under
// the power cap. 2048 over 8192 keys, 32 heads: 239 us, 1.26 PFLOP/s, tensor pipe
// 71 % active.
//
// Roundings: scores, maxima, sums, O and split partials are float32. P is rounded
// to bf16 because the tensor cores take both factors of P V in one type and V is
// bf16; l sums the unrounded p. Random in sign, that adds to the rounding of out
// an error of its size (2-norm relative to float64 0.0023; 0.0016 in float32
// throughout with out rounded once).
// Two ideas are published ones: rescaling O only when the maximum has grown by
// more than a bound, and two softmax warpgroups on alternate tiles.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <math.h>
#include <mutex>

#include "mla.h"
#include "mla_prefill.h"
#include "prefill.cuh"

namespace mla {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

namespace prefill {

constexpr int kAttnThreads = 384;
constexpr int kTile = 128;                 // query rows of a CTA, keys of a key tile
constexpr int kBlockQ = 2 * kTile;         // queries of an item
constexpr int kStages = 3;                 // key tiles in shared memory
constexpr int kQBytes = 3 * kBox;          // 128 rows x 192
constexpr int kHalfBox = kBox / 2;         // 64 rows x 64 columns
constexpr int kKBytes = 3 * kHalfBox;      // 64 keys x 192 (two column blocks of K, k_pe)
constexpr int kVBytes = kBox;              // 128 keys x 64
constexpr int kStageBytes = kKBytes + kVBytes;
constexpr int kAttnSmem = 1024 + 2 * kQBytes + kStages * kStageBytes;
constexpr uint32_t kTmemO = 0, kTmemP = 128, kTmemS = 256, kTmemAll = 512;
constexpr float kGrowth = 8.0f;            // log2: O is rescaled when a row's maximum grew by more (p stays below 2^8)
constexpr int kItems = 8;                  // items handed on and not yet finished by every warp
constexpr long long kShareBytes = 64ll << 20;  // keys and values of a sequence from which rounds pay (see above)
constexpr int kShareBlocks = 4;            // and the blocks that read them
constexpr int kKeyBytes = 512;             // of a head's key and value
constexpr int kItemUnits = 3;              // cost of an item beside its tiles, in tiles
// Registers a thread after the split: the softmax warpgroups hold a row of
// scores each. 256 * 200 + 128 * 104 = 64512 = the 384 * 168 launched.
constexpr int kSoftmaxRegs = 200, kOtherRegs = 104;

// What the merge kernel needs about the item that run w starts and does not
// finish: the number of runs it spans (0: none), its first query row, rows, head,
// and how many of its rows, the first ones, see no key.
struct SplitInfo {
  int32_t pieces, row, rows, head, blind;
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
  // [64 columns, rows, 64-column blocks] of bf16; boxes:
  CUtensorMap q;   // 128 rows, 3 blocks (a head)
  CUtensorMap k;   // 64 rows, 2 blocks
  CUtensorMap v;   // 128 rows, 1 block
  CUtensorMap pe;  // 64 rows, 1 block
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
  // units of the first m blocks of one head. Causal block x (from 1) short of
  // the last has max(1, c + 2x) tiles, c = ceil((L - n) / 128): the first
  // k = max(0, -c / 2) of them one each, the others an arithmetic series.
  MLA_DEV long long units_before(int m, int causal) const {
    return tiles_before(m, causal) + (long long)m * kItemUnits;
  }
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

// A sequence with many keys and values (kShareBytes, kShareBlocks) goes to the
// workers in rounds first, as long as there are items for all of them: heads
// 2x and 2x + 1 give one turn for each block m, blocks m of the first and
// blocks - 1 - m of the second, so that causal turns cost the same, and worker w
// takes turn w of a round. Neighbours then read a head's keys at the same time.
// Returns the number of rounds; the items left over are dealt in runs. kRounds is
// false in the kernel for calls in which no sequence can have rounds.
template <bool kRounds>
MLA_DEV int rounds_of(const AttnArgs& a, const Seq& s) {
  if (!kRounds || s.blocks() < kShareBlocks || (long long)s.L * a.heads * kKeyBytes < kShareBytes) return 0;
  return a.heads / 2 * s.blocks() / a.workers;
}

// What the rounds leave of a sequence: the items from block qb of head h on, in
// the order head, block, without those of head `gap_h` from block `gap_qb` on.
template <bool kRounds>
struct Rest {
  int h, qb, gap_h, gap_qb;
  long long skipped, gap;  // units before the first of them, and of the gap
  MLA_DEV Rest(const AttnArgs& a, const Seq& s) : h(0), qb(0), gap_h(-1), gap_qb(0), skipped(0), gap(0) {
    const int rounds = rounds_of<kRounds>(a, s);
    if (rounds == 0) return;
    const int turns = rounds * a.workers, nb = s.blocks();
    const long long per_head = s.units_before(nb, a.causal);
    h = turns / nb * 2;
    qb = turns % nb;
    skipped = per_head * h + s.units_before(qb, a.causal);
    if (qb > 0) {
      gap_h = h + 1;
      gap_qb = nb - qb;
      gap = per_head - s.units_before(gap_qb, a.causal);
    }
  }
  MLA_DEV long long units(const AttnArgs& a, const Seq& s) const {
    return s.units_before(s.blocks(), a.causal) * a.heads - skipped - gap;
  }
};

// A run's part of an item, as the producer hands it to the other warps.
struct Item {
  int t0, t1;         // key tiles; t1 = 0: the run's end
  int q, rows;        // first query row of the block, its rows
  int h;
  int L, k0;          // the sequence's keys, the first one's row
  int sees;           // keys that the query before the block's first sees, when causal
  int part;           // all of the item's keys: -1; else the slot of its partials (0, 1)
  // rows of the block, its first ones, that see no key
  MLA_DEV int blind(int causal) const { return causal ? min(max(-sees, 0), kBlockQ) : L > 0 ? 0 : kBlockQ; }
};

// Position of a run in the list of items. An item takes kItemUnits + tiles units
// from `item` on; a run that begins or ends in the first kItemUnits begins with,
// or ends before, the item's first tile.
template <bool kRounds>
struct Cursor {
  long long item, end;  // the item's first unit, the run's end
  long long quota;      // units of a run
  Seq s;
  int b, qb, h, t0, tiles;
  int group;            // heads of a group
  int gap_h, gap_qb;    // of Rest
  int round_b, round_end;  // from the first sequence with rounds to behind the last
  MLA_DEV int t1() const { return (int)max(0ll, min((long long)tiles, end - item - kItemUnits)); }
  MLA_DEV bool more() const { return t0 < t1(); }
  // Heads of a group: about a run's number of items of this sequence.
  MLA_DEV static int group_heads(const AttnArgs& a, const Seq& s, long long quota) {
    if (rounds_of<kRounds>(a, s) > 0) return 1;
    const long long per_head = s.units_before(s.blocks(), a.causal);
    return (int)min((long long)a.heads, max(1ll, quotient(quota * s.blocks() + per_head / 2, max(per_head, 1ll))));
  }
  MLA_DEV void next(const AttnArgs& a) {
    item += kItemUnits + tiles;
    t0 = 0;
    if (item + kItemUnits >= end) {  // the run ends before this item's first tile
      tiles = 0;
      return;
    }
    const int g0 = h - h % group;
    if (++h < min(g0 + group, a.heads)) return;
    if (++qb < (g0 == gap_h ? gap_qb : s.blocks())) {
      h = g0;
    } else {
      qb = 0;
      if (h >= a.heads) {  // the sequence's last group
        do {
          s.load(a, ++b);
          const Rest<kRounds> r(a, s);
          h = r.h;
          qb = r.qb;
          gap_h = r.gap_h;
          gap_qb = r.gap_qb;
        } while ((s.n == 0 || h == a.heads) && b + 1 < a.batch);
        group = group_heads(a, s, quota);
      }
    }
    tiles = s.tiles((qb + 1) * kBlockQ, a.causal);
  }
};

// Run `w`: called by a whole warp. Two passes over the sequences, 32 at a time.
template <bool kRounds>
MLA_DEV void run_start(const AttnArgs& a, int w, Cursor<kRounds>* cur) {
  const int lane = threadIdx.x & 31;
  long long total = 0, first_units = 0;
  Seq first{0, 0, 0, 0};  // this lane's sequence of the first 32
  int round_b = a.batch, round_end = 0;
  bool bad = false;
#pragma unroll 1
  for (int b = lane; b < a.batch; b += 32) {
    Seq s;
    s.load(a, b);
    const Rest<kRounds> left(a, s);
    const long long units = left.units(a, s);
    if (left.skipped > 0) {
      round_b = min(round_b, b);
      round_end = b + 1;
    }
    const int oq = __ldg(a.cu_q + b), ok = __ldg(a.cu_k + b);
    bad |= oq != s.q0 || ok != s.k0 || __ldg(a.cu_q + b + 1) != s.q0 + s.n || __ldg(a.cu_k + b + 1) != s.k0 + s.L;
    if (b == lane) {
      first = s;
      first_units = units;
    }
    total += units;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(~0u, total, o);
  if (w == 0 && bad) set_error(a.error, kErrSeqLen);
  const long long quota = max(1ll, quotient(total + a.workers - 1, a.workers));
  cur->quota = quota;
  const long long u = min((long long)w * quota, total);
  cur->item = u;
  cur->end = min(u + quota, total);
  cur->s = Seq{0, 0, 0, 0};
  cur->b = cur->qb = cur->h = cur->t0 = 0;
  cur->tiles = 0;
  cur->group = 1;
  cur->round_b = __reduce_min_sync(~0u, round_b);
  cur->round_end = __reduce_max_sync(~0u, round_end);
  cur->gap_h = -1;
  cur->gap_qb = 0;
  if (u >= total) return;
  long long before = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < a.batch; b0 += 32) {
    Seq s = first;
    long long own = first_units;
    if (b0 > 0) {
      s = Seq{0, 0, 0, 0};
      if (b0 + lane < a.batch) s.load(a, b0 + lane);
      own = Rest<kRounds>(a, s).units(a, s);
    }
    long long incl = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(~0u, incl, o);
      if (lane >= o) incl += y;
    }
    const unsigned beyond = __ballot_sync(~0u, before + incl > u);
    if (beyond) {
      const int src = __ffs(beyond) - 1;
      cur->b = b0 + src;
      cur->s.q0 = __shfl_sync(~0u, s.q0, src);
      cur->s.n = __shfl_sync(~0u, s.n, src);
      cur->s.k0 = __shfl_sync(~0u, s.k0, src);
      cur->s.L = __shfl_sync(~0u, s.L, src);
      cur->group = Cursor<kRounds>::group_heads(a, cur->s, quota);
      long long rest = u - before - __shfl_sync(~0u, incl - own, src);
      const long long per_head = cur->s.units_before(cur->s.blocks(), a.causal);
      const Rest<kRounds> left(a, cur->s);
      cur->gap_h = left.gap_h;
      cur->gap_qb = left.gap_qb;
      rest += left.skipped;
      if (rest >= per_head * (left.gap_h + 1) - left.gap) rest += left.gap;
      const int g0 = (int)quotient(rest, per_head * cur->group) * cur->group;  // the group's first head
      const int heads = min(cur->group, a.heads - g0);
      rest -= per_head * g0;
      int lo = 0, hi = cur->s.blocks() - 1;  // the last block that starts at or before `rest`
      while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (cur->s.units_before(mid, a.causal) * heads <= rest) lo = mid;
        else hi = mid - 1;
      }
      cur->qb = lo;
      cur->tiles = cur->s.tiles((lo + 1) * kBlockQ, a.causal);
      rest -= cur->s.units_before(lo, a.causal) * heads;
      const int units = cur->tiles + kItemUnits, items = (int)quotient(rest, units);
      const int in_item = (int)(rest - (long long)items * units);
      cur->h = g0 + items;
      cur->item = u - in_item;
      cur->t0 = max(0, in_item - kItemUnits);
      return;
    }
    before += __shfl_sync(~0u, incl, 31);
  }
}

// An item whose rows a softmax warp has still to write.
struct PendingRows {
  int q, rows, h;     // output row of the warp's lane 0, lanes with a row, head
  int blind;          // lanes, the first ones, whose row sees no key
  int live, whole;    // rows of this CTA at all; all of the item's keys (not a part)
  long long part;     // else: row of the partials
};

struct AttnShared {
  // Key tile i uses entry i % 3 of the first four, i % 2 of the next three.
  // "even": only the even CTA's is used, by both CTAs; "both": each CTA's own.
  uint64_t k_full[kStages], v_full[kStages];   // even: both CTAs' halves have landed
  uint64_t k_empty[kStages];                   // both: Q K(i) done
  uint64_t pv_done[kStages];                   // both: P(i) V(i) done
  uint64_t s_full[2];                          // both: Q K(i) done
  uint64_t s_free[2], p_full[2];               // even: scores read, probabilities written by both CTAs
  uint64_t q_full[2], q_empty[2];              // q_full: even CTA
  uint64_t o_done;                             // both: an item's last P V is done
  uint64_t o_empty;                            // even CTA: both CTAs have read an item's O
  uint64_t v_landed[kStages];                  // V of a sequence's last tile, before its rows are cleared
  uint64_t m_ready[4], fin[4];                 // per 32 rows: reference maximum of a tile, sums of an item
  uint64_t done;
  uint64_t item_full[kItems], item_free[kItems];  // entry of item[], read by all other warps
  Item item[kItems];
  PendingRows pending[8];
  Cursor<true> run;                            // the producer's run while it is in rounds
  float m[2][kTile];                           // reference maximum after tile n, entry n % 2
  float fin_m[2][2][kTile], fin_l[2][2][kTile];  // [item % 2][warpgroup]
  uint32_t tmem;
  uint32_t abort_flag;
};

// Entry and phase of a ring of kStages.
struct RingPos {
  int s = 0;
  uint32_t phase = 0;
  MLA_DEV void next() {
    if (++s == kStages) {
      s = 0;
      phase ^= 1u;
    }
  }
  MLA_DEV void advance(int n) {
    s += n;
    phase ^= (uint32_t)(s / kStages) & 1u;
    s %= kStages;
  }
};

// 32 bytes to global memory, 32-byte aligned.
MLA_DEV void st_global_v8(void* dst, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

MLA_DEV float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

template <bool kRounds>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kAttnThreads, 1)
    mla_prefill_attention_kernel(const __grid_constant__ AttnMaps maps, const AttnArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ AttnShared sh;
  // both CTAs' layouts are the same: the pair's instructions use one set of offsets
  const uint32_t qbuf = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t stages = qbuf + 2 * kQBytes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_ctarank(), worker = (int)cluster_id_x();
  Waiter W{&sh.abort_flag, a.error};

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_addr(&sh.k_full[s]), 2);  // both producers, or both clearing warps
      mbar_init(smem_addr(&sh.v_full[s]), 2);
      mbar_init(smem_addr(&sh.k_empty[s]), 1);
      mbar_init(smem_addr(&sh.pv_done[s]), 1);
      mbar_init(smem_addr(&sh.v_landed[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_addr(&sh.s_full[b]), 1);
      mbar_init(smem_addr(&sh.s_free[b]), 8);  // four softmax warps of either CTA
      mbar_init(smem_addr(&sh.p_full[b]), 8);
      mbar_init(smem_addr(&sh.q_full[b]), 2);
      mbar_init(smem_addr(&sh.q_empty[b]), 1);
    }
    mbar_init(smem_addr(&sh.o_done), 1);
    mbar_init(smem_addr(&sh.o_empty), 16);     // all softmax warps of both CTAs
    for (int x = 0; x < 4; ++x) {
      mbar_init(smem_addr(&sh.m_ready[x]), 1);
      mbar_init(smem_addr(&sh.fin[x]), 2);     // the two softmax warps of the rows
    }
    for (int x = 0; x < kItems; ++x) {
      mbar_init(smem_addr(&sh.item_full[x]), 1);
      mbar_init(smem_addr(&sh.item_free[x]), rank == 0 ? 11 : 9);  // softmax, clearing, (even CTA) issuers
    }
    mbar_init(smem_addr(&sh.done), 2);         // the two issuers
    sh.abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == 8) {
    tmem_alloc_pair(smem_addr(&sh.tmem), kTmemAll);
    tmem_relinquish_pair();
  }
  if (warp == 9 && elect_one()) {
    prefetch_tmap(&maps.q);
    prefetch_tmap(&maps.k);
    prefetch_tmap(&maps.v);
    prefetch_tmap(&maps.pe);
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  grid_dependency_wait();  // every thread, for its own accesses
  const uint32_t tmem = sh.tmem;
  // an entry of the even CTA's barriers, for both CTAs
  const auto leader = [&](uint64_t* bar) { return map_to_rank(smem_addr(bar), 0); };
  // tile j reaches behind the sequence's end
  const auto tail = [](const Item& it, int j) { return it.L < (j + 1) * kTile; };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
  }
  if (warp == 9) {
    // ------------------------------------------------------------ producer
    Cursor<kRounds> cur;
    run_start(a, worker, &cur);
    if (elect_one()) {
      // Rounds come first: the cursor is at one of their items, an item's end its
      // run's end, and the run's start waits in shared memory.
      int rb = cur.round_b - 1, rk = 0, halves = 0;  // sequence, half turn, half turns
      const int round_end = cur.round_end;
      bool in_rounds = kRounds && cur.round_b < round_end;
      const auto next_turn = [&]() {
        if constexpr (kRounds) {
#pragma unroll 1
          while (rk == halves) {
            if (++rb >= round_end) {
              cur = sh.run;
              return false;
            }
            cur.s.load(a, rb);
            halves = 2 * rounds_of<kRounds>(a, cur.s);
            rk = 0;
          }
          const int turn = (rk >> 1) * a.workers + worker, nb = cur.s.blocks();
          cur.h = turn / nb * 2 + (rk & 1);
          cur.qb = (rk & 1) ? nb - 1 - turn % nb : turn % nb;
          cur.tiles = cur.s.tiles((cur.qb + 1) * kBlockQ, a.causal);
          cur.t0 = 0;
          cur.item = 0;
          cur.end = cur.tiles + kItemUnits;
          ++rk;
        }
        return true;
      };
      if constexpr (kRounds) {
        if (in_rounds) {
          sh.run = cur;
          in_rounds = next_turn();
        }
      }
      if (rank == 0) a.info[worker].pieces = 0;
      RingPos pk, pv;
      int nk = 0, nv = 0;           // items handed on, items of V begun
      int jk = 0, k_end = 0, jv = 0, v_end = 0;  // tiles of the items at hand
      int left = 0;                 // tiles whose K was loaded and V not yet
      bool ok = true, more = true;
      // turn x: V of tile x - 3, K of tile x
#pragma unroll 1
      for (int x = 0; ok; ++x) {
        if (x >= kStages) {
          if (left == 0) break;
          if (jv == v_end) {
            const Item& next = sh.item[nv++ % kItems];
            jv = next.t0;
            v_end = next.t1;
          }
          const Item& it = sh.item[(nv - 1) % kItems];
          if (!(ok = W.wait(&sh.pv_done[pv.s], pv.phase ^ 1))) break;  // V of three tiles ago is done with
          const uint32_t vs = stages + pv.s * kStageBytes + kKBytes;
          const int row = it.k0 + jv * kTile;
          if (tail(it, jv)) {
            const uint32_t vl = smem_addr(&sh.v_landed[pv.s]);
            mbar_arrive_expect_tx(vl, kVBytes);
            tma_load_3d(vs, &maps.v, 0, row, 4 * it.h + 2 + rank, vl);
          } else {
            const uint32_t vf = leader(&sh.v_full[pv.s]);
            mbar_arrive_expect_tx_cluster(vf, kVBytes);
            tma_load_3d_pair(vs, &maps.v, 0, row, 4 * it.h + 2 + rank, vf);
          }
          pv.next();
          ++jv;
          --left;
        }
        if (more && jk == k_end) {  // the next item, or the run's end, for all warps
          const int e = nk % kItems, b = nk & 1;
          if (!(ok = W.wait(&sh.item_free[e], ((nk / kItems) & 1) ^ 1))) break;
          Item& it = sh.item[e];
          const int t1 = cur.t1(), r0 = cur.qb * kBlockQ;
          jk = cur.t0;
          more = cur.more();
          it = Item{jk, more ? t1 : 0, cur.s.q0 + r0, min(cur.s.n - r0, kBlockQ), cur.h, cur.s.L, cur.s.k0,
                    cur.s.L - cur.s.n + r0, jk > 0 ? 0 : t1 < cur.tiles ? 1 : -1};
          mbar_arrive(smem_addr(&sh.item_full[e]));
          if (more) {
            k_end = t1;
            if (rank == 0 && it.part == 1)  // the item goes on in the following runs
              a.info[worker] = SplitInfo{
                  (int)(quotient(cur.item + kItemUnits + cur.tiles - 1, cur.quota) - worker) + 1, it.q, it.rows, it.h,
                  it.blind(a.causal)};
            if (!(ok = W.wait(&sh.q_empty[b], ((nk >> 1) & 1) ^ 1))) break;
            mbar_arrive_expect_tx_cluster(leader(&sh.q_full[b]), kQBytes);
            tma_load_3d_pair(qbuf + b * kQBytes, &maps.q, 0, it.q + rank * kTile, 3 * it.h, leader(&sh.q_full[b]));
            ++nk;
            if (in_rounds) in_rounds = next_turn();
            else cur.next(a);
          }
        }
        if (more) {
          const Item& it = sh.item[(nk - 1) % kItems];
          if (!(ok = W.wait(&sh.k_empty[pk.s], pk.phase ^ 1))) break;  // K of three tiles ago is done with
          const uint32_t kf = leader(&sh.k_full[pk.s]), ks = stages + pk.s * kStageBytes;
          const int row = it.k0 + jk * kTile + 64 * rank;
          mbar_arrive_expect_tx_cluster(kf, kKBytes);
          tma_load_3d_pair(ks, &maps.k, 0, row, 4 * it.h, kf);
          tma_load_3d_pair(ks + 2 * kHalfBox, &maps.pe, 0, row, 0, kf);
          pk.next();
          ++jk;
          ++left;
        }
      }
      // Every load was waited for by its reader, unless a wait ran out: then
      // the copies in flight get ample time before the CTA exits.
      if (W.aborted()) {
        const uint64_t t = global_timer_ns();
        while (global_timer_ns() - t < 10000000ull) {}
      }
    }
    __syncwarp();
  } else if (warp == 8) {
    // ------------------------------------------------------------ MMA issuer: scores
    if (rank == 0 && elect_one()) {
      constexpr uint32_t idesc = idesc_bf16_f32(256, 128, 0, 0);
      RingPos p;
      int nq = 0, i = 0;  // items, tiles
      bool ok = true;
#pragma unroll 1
      for (; ok; ++nq) {
        if (!W.wait(&sh.item_full[nq % kItems], (nq / kItems) & 1)) break;
        const int t0 = sh.item[nq % kItems].t0, t1 = sh.item[nq % kItems].t1, b = nq & 1;
        if (t1 == 0) break;
        mbar_arrive(smem_addr(&sh.item_free[nq % kItems]));
        if (!W.wait(&sh.q_full[b], (nq >> 1) & 1)) break;
        const uint64_t qd = smem_desc_sw128(qbuf + b * kQBytes, 16, 1024);
#pragma unroll 1
        for (int j = t0; j < t1; ++j, p.next(), ++i) {
          if (!(ok = W.wait(&sh.k_full[p.s], p.phase))) break;
          if (!(ok = W.wait(&sh.s_free[i & 1], ((i >> 1) & 1) ^ 1))) break;
          tc_fence_after();
          // S = Q K^T; 16 columns are 32 bytes of a swizzled row
          const uint64_t kd = smem_desc_sw128(stages + p.s * kStageBytes, 16, 1024);
          const uint32_t st = tmem + kTmemS + 128 * (i & 1);
#pragma unroll
          for (int u = 0; u < 12; ++u)
            mma_ss_pair(st, qd + (u >> 2) * (kBox >> 4) + 2 * (u & 3), kd + (u >> 2) * (kHalfBox >> 4) + 2 * (u & 3),
                        idesc, u > 0 ? 1u : 0u);
          mma_commit_pair(smem_addr(&sh.s_full[i & 1]));
          mma_commit_pair(smem_addr(&sh.k_empty[p.s]));
        }
        if (ok) mma_commit_pair(smem_addr(&sh.q_empty[b]));
      }
      mma_commit_pair(smem_addr(&sh.done));
      W.wait(&sh.done, 0, true);
    }
    __syncwarp();
  } else if (warp == 11) {
    // ------------------------------------------------------------ MMA issuer: values
    if (rank == 0 && elect_one()) {
      constexpr uint32_t idesc = idesc_bf16_f32(256, 128, 0, 1);
      RingPos p;
      int no = 0, i = 0;  // items, tiles
      bool ok = true;
#pragma unroll 1
      for (; ok; ++no) {
        if (!W.wait(&sh.item_full[no % kItems], (no / kItems) & 1)) break;
        const Item& it = sh.item[no % kItems];
        const int t0 = it.t0, t1 = it.t1, last_tail = tail(it, t1 - 1) ? t1 - 1 : -1;
        if (t1 == 0) break;
        mbar_arrive(smem_addr(&sh.item_free[no % kItems]));
        if (!W.wait(&sh.o_empty, (no & 1) ^ 1)) break;
#pragma unroll 1
        for (int j = t0; j < t1; ++j, p.next(), ++i) {
          // the rows cleared by the other CTA's threads want the wider acquire
          if (!(ok = j == last_tail ? W.wait_cluster(&sh.v_full[p.s], p.phase) : W.wait(&sh.v_full[p.s], p.phase))) break;
          if (!(ok = W.wait(&sh.p_full[i & 1], (i >> 1) & 1))) break;
          tc_fence_after();
          const uint64_t vd = smem_desc_sw128(stages + p.s * kStageBytes + kKBytes, kBox, 1024);
          const uint32_t pt = tmem + kTmemP + 64 * (i & 1);
#pragma unroll
          for (int u = 0; u < 8; ++u)  // 16 keys: 8 columns of P, 16 rows of V
            mma_tmem_a_pair(tmem + kTmemO, pt + 8 * u, vd + 128 * u, idesc, (u > 0 || j > t0) ? 1u : 0u);
          mma_commit_pair(smem_addr(&sh.pv_done[p.s]));
        }
        if (ok) mma_commit_pair(smem_addr(&sh.o_done));
      }
      mma_commit_pair(smem_addr(&sh.done));
      W.wait(&sh.done, 0, true);
    }
    __syncwarp();
  } else if (warp == 10) {
    // ------------------------------------------------------------ value rows behind a sequence's end
    // Their probabilities are 0, but 0 * NaN is NaN: whatever lies there is cleared.
    RingPos p;
    uint32_t phases = 0;  // of the entries of v_landed, which only some tiles use
    int ahead = 0;        // tiles of the item before: this warp waits for an item's end, not tile by tile
#pragma unroll 1
    for (int n = 0;; ++n) {
      if (!W.wait_warp_tiles(&sh.item_full[n % kItems], (n / kItems) & 1, ahead)) break;
      const Item it = sh.item[n % kItems];
      const int t1 = it.t1;
      if (t1 == 0) break;
      ahead = t1 - it.t0;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&sh.item_free[n % kItems]));
#pragma unroll 1
      for (int j = it.t0; j < t1 - 1; ++j) p.next();  // only an item's last tile can be its sequence's last
      if (tail(it, t1 - 1)) {
        if (!W.wait_warp_tiles(&sh.v_landed[p.s], (phases >> p.s) & 1, ahead)) break;
        phases ^= 1u << p.s;
        const uint32_t vs = stages + p.s * kStageBytes + kKBytes;
        for (int x = max(it.L - (t1 - 1) * kTile, 0) * 8 + lane; x < kTile * 8; x += 32)
          st_shared_v4(vs + 16 * x, make_uint4(0, 0, 0, 0));
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_release_cluster(leader(&sh.v_full[p.s]));
      }
      p.next();
    }
    __syncwarp();
  } else if (warp < 8) {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int g = warp >> 2, quad = warp & 3;          // warpgroup, 32-row quadrant
    const int row = quad * 32 + lane;                  // row of the CTA = TMEM lane
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
    const uint32_t st = lanes + kTmemS + 128 * g, pt = lanes + kTmemP + 64 * g;
    RingPos first;                                     // entry of the item's first tile
    RingPos mine;                                      // entry of this warpgroup's last tile
    int turn = 0;                                      // tiles before the item, mod 2
    int ns = 0;                                        // tiles of this warpgroup
    int ne = 0;                                        // items
    int nm = 0, nf = 0, ni = 0;                        // tiles with shared maxima; written items with live rows, all items
    bool ok = true;
    bool pending = false;                              // an item's rows are still to be written
    // The rows of an item, or this run's part of them: 64 columns for each
    // warpgroup. The last P V is normally long done when this is called.
    const auto write_rows = [&]() {
      pending = false;
      const PendingRows& pr = sh.pending[warp];
      if (!W.wait_warp(&sh.o_done, ni & 1)) return false;
      ++ni;
      tc_fence_after();
      if (!pr.live) {
        if (lane == 0) mbar_arrive_cluster(leader(&sh.o_empty));
        return true;
      }
      const bool valid = lane < pr.rows;
      const size_t r = (size_t)(pr.q + lane) * a.heads + pr.h, prow = (size_t)pr.part + lane;
      __nv_bfloat16* dst = a.out + r * 128 + 64 * g;
      float* part = a.part_o + prow * 128 + 64 * g;
      uint32_t o[64];
      tmem_ld_32x32b_32(lanes + kTmemO + 64 * g, *reinterpret_cast<uint32_t(*)[32]>(&o[0]));
      tmem_ld_32x32b_32(lanes + kTmemO + 64 * g + 32, *reinterpret_cast<uint32_t(*)[32]>(&o[32]));
      tmem_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(leader(&sh.o_empty));
      if (!W.wait_warp(&sh.fin[quad], nf & 1)) return false;
      const float m0 = sh.fin_m[nf & 1][0][row], m1 = sh.fin_m[nf & 1][1][row], mm = fmaxf(m0, m1);
      const float l0 = sh.fin_l[nf & 1][0][row], l1 = sh.fin_l[nf & 1][1][row];
      ++nf;
      float l = l0 != 0.f ? l0 * ex2((m0 - mm) * a.scale_log2) : 0.f;
      if (l1 != 0.f) l += l1 * ex2((m1 - mm) * a.scale_log2);
      // l = 0: no keys (the products are all 0 * v), or nothing but -inf scores; of
      // a part only the merge knows which, it writes (0, -inf)
      const float none = pr.whole && lane >= pr.blind ? NAN : 0.f;
      const float inv = l != 0.f ? 1.f / l : none;
      const float lse = l != 0.f ? mm * a.scale + logf(l) : none - INFINITY;
      if (valid) {
#pragma unroll
        for (int x = 0; x < 64; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * inv);
        uint32_t w[8];
        if (pr.whole) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
#pragma unroll
            for (int x = 0; x < 8; ++x)
              w[x] = pack_bf16x2(__uint_as_float(o[16 * c + 2 * x]), __uint_as_float(o[16 * c + 2 * x + 1]));
            st_global_v8(dst + 16 * c, w);
          }
        } else {
#pragma unroll
          for (int c = 0; c < 8; ++c) st_global_v8(part + 8 * c, *reinterpret_cast<uint32_t(*)[8]>(&o[8 * c]));
        }
      }
      if (valid && g == 0) {
        if (pr.whole) a.lse[r] = lse;
        else a.part_lse[prow] = lse;
      }
      return true;
    };
#pragma unroll 1
    while (true) {
      if (!(ok = W.wait_warp(&sh.item_full[ne % kItems], (ne / kItems) & 1))) break;
      const Item& it = sh.item[ne % kItems];
      const int t0 = it.t0, t1 = it.t1;
      const bool more = t1 > 0;
      if (!more && !pending) break;
      // keys this row sees
      const int limit = a.causal ? min(it.L, it.sees + kTile * rank + row + 1) : it.L;
      // key tiles that all of the warp's rows see whole (the first row sees least)
      const int whole_tiles = __shfl_sync(~0u, limit, 0) >> 7;
      const bool live = kTile * rank < it.rows;        // without live rows only the hand-shakes remain
      float m = -INFINITY, l = 0.f;                    // this warpgroup's reference maximum (raw scores) and sum
      // This warpgroup's tiles, every second one, and one turn behind the last.
      // The rows of the item before are written when the item's first tile is
      // under way: its softmax does not need O, but any other tile may have to
      // rescale O, which the tensor cores start on only when it has been read.
      RingPos now = first;
      if (turn != g) now.next();
#pragma unroll 1
      for (int j = t0 + (turn ^ g);; j += 2) {
        if (pending && (j > t0 || !more) && !(ok = write_rows())) break;
        if (j >= t1) break;
        if (!(ok = W.wait_warp(&sh.s_full[g], ns & 1))) break;
        tc_fence_after();
        if (live) {
          uint32_t s[4][32];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld_32x32b_32(st + 32 * c, s[c]);
          // the reference after the previous tile
          const int nt = nm + j - t0;                  // tiles with shared maxima before this one
          if (nt > 0 && !(ok = W.wait_warp(&sh.m_ready[quad], (nt - 1) & 1))) break;
          float m_prev = sh.m[(nt & 1) ^ 1][row];
          tmem_wait_ld();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(leader(&sh.s_free[g]));
          if (j >= whole_tiles) {
            const int seen = limit - j * kTile;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int n = min(max(seen - 32 * c, 0), 32);
              const uint32_t hidden = n < 32 ? ~0u << n : 0u;  // bit x: column 32 c + x is not seen
#pragma unroll
              for (int x = 0; x < 32; ++x)
                if ((hidden >> x) & 1u) s[c][x] = 0xff800000u;  // -inf
            }
          }
          float mx[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            mx[c] = __uint_as_float(s[c][0]);
#pragma unroll
            for (int x = 1; x < 31; x += 2) mx[c] = max3(mx[c], __uint_as_float(s[c][x]), __uint_as_float(s[c][x + 1]));
            mx[c] = fmaxf(mx[c], __uint_as_float(s[c][31]));
          }
          const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
          if (j == t0) m_prev = top;
          const bool grow = (top - m_prev) * a.scale_log2 > kGrowth;  // false while both are -inf (NaN)
          const float m_new = grow ? top : m_prev;
          sh.m[nt & 1][row] = m_new;
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&sh.m_ready[quad]));
          if (m_new != m) {
            l *= ex2((m - m_new) * a.scale_log2);      // 0 * ex2(-inf) at the first
            m = m_new;
          }
          if (__any_sync(~0u, grow)) {
            const float f = grow ? ex2((m_prev - m_new) * a.scale_log2) : 1.f;
            RingPos prev = now;                        // the previous tile's entry is two further in the ring of three
            prev.next();
            prev.next();
            if (!(ok = W.wait_warp(&sh.pv_done[prev.s], prev.phase ^ 1))) break;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
              uint32_t o[16];
              tmem_ld_32x32b_16(lanes + kTmemO + 16 * c, o);
              tmem_wait_ld();
#pragma unroll
              for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
              tmem_st_16(lanes + kTmemO + 16 * c, o);
            }
          }
          const float shift = m == -INFINITY ? 0.f : -m * a.scale_log2;
          const float2 k2 = make_float2(a.scale_log2, a.scale_log2), b2 = make_float2(shift, shift);
          float2 sum[4];
          uint32_t p0[32], p1[32];
          const auto exponentials = [&](const uint32_t(&x)[32], uint32_t* out, float2& total) {
            total = make_float2(0.f, 0.f);
#pragma unroll
            for (int u = 0; u < 32; u += 2) {
              const float2 y = fma2_rn(make_float2(__uint_as_float(x[u]), __uint_as_float(x[u + 1])), k2, b2);
              const float2 e2 = make_float2(ex2(y.x), ex2(y.y));
              total = add2_rn(total, e2);
              out[u / 2] = pack_bf16x2(e2.x, e2.y);
            }
          };
          exponentials(s[0], p0, sum[0]);
          exponentials(s[1], p0 + 16, sum[1]);
          // P V of this warpgroup's last tile has read its P
          if (ns > 0 && !(ok = W.wait_warp(&sh.pv_done[mine.s], mine.phase))) break;
          tc_fence_after();
          tmem_st_32(pt, p0);
          exponentials(s[2], p1, sum[2]);
          exponentials(s[3], p1 + 16, sum[3]);
          tmem_st_32(pt + 32, p1);
          const float2 s01 = add2_rn(add2_rn(sum[0], sum[1]), add2_rn(sum[2], sum[3]));
          l += s01.x + s01.y;
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
        } else {
          if (lane == 0) mbar_arrive_cluster(leader(&sh.s_free[g]));
          if (ns > 0 && !(ok = W.wait_warp(&sh.pv_done[mine.s], mine.phase))) break;
        }
        if (lane == 0) mbar_arrive_cluster(leader(&sh.p_full[g]));
        mine = now;
        ++ns;
        now.next();
        now.next();
      }
      if (!ok || !more) break;
      first.advance(t1 - t0);
      turn ^= (t1 - t0) & 1;
      if (live) nm += t1 - t0;
      pending = true;
      __syncwarp();
      if (live) {
        sh.fin_m[nf & 1][g][row] = m;  // the item before is written: this is item nf
        sh.fin_l[nf & 1][g][row] = l;
      }
      if (lane == 0) {
        const int r0 = kTile * rank + quad * 32;
        sh.pending[warp] = PendingRows{it.q + r0, it.rows - r0, it.h, it.blind(a.causal) - r0, live, it.part < 0,
                                       (2ll * worker + it.part) * kBlockQ + r0};
        mbar_arrive(smem_addr(&sh.item_free[ne % kItems]));
      }
      ++ne;
      __syncwarp();
      if (live && lane == 0) mbar_arrive(smem_addr(&sh.fin[quad]));
    }
    __syncwarp();
  }

  allow_dependents();  // the merge kernel's blocks may take SMs as these CTAs finish
  tc_fence_before();
  cluster_sync();      // neither CTA leaves while the other may still reach its shared memory or TMEM
  tc_fence_after();
  if (warp == 8) tmem_dealloc_pair(tmem, kTmemAll);
}

// Merge of split items: block (w, g) joins 8 rows of the item that run w starts
// and does not finish, a warp each, four columns to a lane. The parts are run w's
// second slot and the first slots of the following runs; lane p holds the lse of
// part p (of p + 32, ... in turn for a longer list).
constexpr int kMergeRows = 8;
__global__ void __launch_bounds__(32 * kMergeRows) mla_prefill_merge_kernel(const AttnArgs a) {
  grid_dependency_wait();
  const int w = blockIdx.x, lane = threadIdx.x & 31;
  const SplitInfo it = a.info[w];
  const int row = blockIdx.y * kMergeRows + (threadIdx.x >> 5);
  const int pieces = min(it.pieces, a.workers - w);
  if (pieces < 1 || row >= it.rows) return;
  const auto slot = [&](int p) { return (size_t)(p == 0 ? 2 * w + 1 : 2 * (w + p)) * kBlockQ + row; };
  float m = -INFINITY;
  for (int p = lane; p < pieces; p += 32) m = fmaxf(m, a.part_lse[slot(p)]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f;
  for (int p0 = 0; p0 < pieces; p0 += 32) {
    const int mine = p0 + lane;
    const float lse = mine < pieces ? a.part_lse[slot(mine)] : -INFINITY;
    const float weight = lse == -INFINITY ? 0.f : expf(lse - m);
    const int count = min(32, pieces - p0);
#pragma unroll 4
    for (int p = 0; p < count; ++p) {
      const float f = __shfl_sync(~0u, weight, p);
      const float4 v = reinterpret_cast<const float4*>(a.part_o + slot(p0 + p) * 128)[lane];
      sum += f;
      if (f != 0.f) {  // a part without keys counts for nothing, whatever its rows hold
        acc.x = fmaf(f, v.x, acc.x);
        acc.y = fmaf(f, v.y, acc.y);
        acc.z = fmaf(f, v.z, acc.z);
        acc.w = fmaf(f, v.w, acc.w);
      }
    }
  }
  const float none = row >= it.blind ? NAN : 0.f;  // keys, and nothing but -inf scores: NaN
  const float inv = sum != 0.f ? 1.f / sum : none;
  const size_t r = (size_t)(it.row + row) * a.heads + it.head;
  reinterpret_cast<uint2*>(a.out + r * 128)[lane] =
      make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  if (lane == 0) a.lse[r] = sum != 0.f ? m + logf(sum) : none - INFINITY;
}

mla_status_t check_attention(const mlap_attention_desc_t* d) {
  if (!d) return MLA_ERR_INVALID_ARG;
  if (d->batch < 0 || d->num_heads < 1 || d->num_q < 0 || d->num_k < 0 || (d->causal != 0 && d->causal != 1) ||
      d->num_sms < 0 || d->pe_stride < kDRope || !(d->softmax_scale > 0.f) || !isfinite(d->softmax_scale))
    return MLA_ERR_INVALID_ARG;
  if (d->num_heads > kMaxHeads || d->batch > kMaxBatch || d->d_nope != 128 || d->d_rope != kDRope || d->d_v != 128 || d->pe_stride % 8 != 0)
    return MLA_ERR_UNSUPPORTED;
  // row indexes and tile counts are 32-bit
  if (d->num_q > 0x7fffffff - kBlockQ || d->num_k > 0x7fffffff - kTile) return MLA_ERR_UNSUPPORTED;
  return MLA_OK;
}

// SMs of the current device, the kernel's shared memory opted into (once per
// device); 0 on a CUDA error.
int device_sms() {
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
        cudaFuncSetAttribute((const void*)mla_prefill_attention_kernel<false>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, kAttnSmem) != cudaSuccess ||
        cudaFuncSetAttribute((const void*)mla_prefill_attention_kernel<true>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, kAttnSmem) != cudaSuccess) {
      cudaGetLastError();
      return 0;
    }
    sms[dev] = n;
  }
  return sms[dev];
}

// Workers (CTA pairs) of the current device for this descriptor; 0 on a CUDA error.
int attention_workers(const mlap_attention_desc_t* d) {
  int sms = device_sms();
  if (sms == 0) return 0;
  if (d->num_sms > 0 && d->num_sms < sms) sms = d->num_sms;
  return sms < 2 ? 1 : sms / 2;
}

// Workspace: [SplitInfo | part_lse | part_o], each a multiple of 256 bytes.
size_t info_bytes(int workers) { return ((size_t)workers * sizeof(SplitInfo) + 255) & ~(size_t)255; }
size_t part_lse_bytes(int workers) { return (size_t)2 * workers * kBlockQ * sizeof(float); }
size_t workspace_bytes(int workers) {
  return info_bytes(workers) + part_lse_bytes(workers) + (size_t)2 * workers * kBlockQ * 128 * sizeof(float);
}

// A row-major bf16 matrix as [64 columns, rows, 64-column blocks]; a box's
// blocks lie one after the other, rows 128-byte swizzled.
bool encode_blocks(CUtensorMap* m, const void* p, long long blocks, long long rows, long long stride, int box_rows,
                   int box_blocks) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[3] = {64, (cuuint64_t)rows, (cuuint64_t)blocks};
  cuuint64_t strides[2] = {(cuuint64_t)stride * 2, 128};
  cuuint32_t box[3] = {64, (cuuint32_t)box_rows, (cuuint32_t)box_blocks}, elem[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), dims, strides, box, elem,
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
  if (off(q, 16) || off(kv, 16) || off(k_pe, 16) || off(out, 32) || off(workspace, 32) || off(cu_q, 4) ||
      off(cu_k, 4) || off(lse, 4) || off(error, 4))
    return MLA_ERR_INVALID_ARG;
  const int workers = attention_workers(d);
  if (workers == 0) return MLA_ERR_CUDA;
  if (ws_bytes < workspace_bytes(workers)) return MLA_ERR_WORKSPACE_TOO_SMALL;
  AttnMaps maps;
  // without keys the boxes still load (all masked): any valid memory does
  const bool keys = d->num_k > 0;
  const void* kvp = keys ? kv : q;
  const long long kv_blocks = keys ? 4ll * d->num_heads : 1, nk = keys ? d->num_k : 1;
  if (!encode_blocks(&maps.q, q, 3ll * d->num_heads, d->num_q, 192ll * d->num_heads, kTile, 3) ||
      !encode_blocks(&maps.k, kvp, kv_blocks, nk, 64 * kv_blocks, kTile / 2, 2) ||
      !encode_blocks(&maps.v, kvp, kv_blocks, nk, 64 * kv_blocks, kTile, 1) ||
      !encode_blocks(&maps.pe, keys ? k_pe : q, 1, nk, keys ? d->pe_stride : 64, kTile / 2, 1))
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
  // whether rounds_of can be above 0 for a sequence of these rows
  const int blocks = (a.num_q + kBlockQ - 1) / kBlockQ;
  const bool rounds = (long long)a.num_k * a.heads * kKeyBytes >= kShareBytes && blocks >= kShareBlocks &&
                      (long long)(a.heads / 2) * blocks >= workers;
  if (launch_dependent(rounds ? mla_prefill_attention_kernel<true> : mla_prefill_attention_kernel<false>, dim3(2 * workers), kAttnThreads, kAttnSmem, stream, maps, a) !=
      cudaSuccess)
    return MLA_ERR_CUDA;
  return launch_dependent(mla_prefill_merge_kernel, dim3(workers, kBlockQ / kMergeRows), 32 * kMergeRows, 0, stream, a) ==
                 cudaSuccess
             ? MLA_OK
             : MLA_ERR_CUDA;
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
