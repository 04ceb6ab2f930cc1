// Definitions shared by the prefill kernels: bounded pipeline waits and the
// error bits they report.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "prefill_ptx.cuh"

namespace mla {
namespace prefill {

constexpr uint32_t kErrPosition = 0x10u;       // MLA_DEVERR_POSITION
constexpr uint64_t kWaitNs = 2000000000ull;    // a pipeline wait gives up after 2 s: only a broken device gets there
constexpr uint64_t kTileNs = 20000;            // more for a wait that lasts as long as a tile of 128 keys
// Sequences of a call: indexes that step over them stay in 32 bits, and a worker
// passes a run of empty ones within the waits of the warps that it feeds (84 ns
// each: 2^20 between two sequences 88 ms, 2^22 0.35 s, 0.6 s at the lowest clocks).
constexpr int kMaxBatch = 1 << 22;
constexpr int kBox = 128 * 128;                // bytes of a 128-row x 64-column bf16 box (128-byte swizzle rows)

MLA_DEV void set_error(uint32_t* word, uint32_t bits) {
  if (word) atomicOr(word, bits);
}

// Bounded waits of one CTA: a wait that runs out raises the CTA's abort flag
// and the caller's error word; every later wait then returns at once, except
// the draining ones, which let copies and MMAs in flight finish.
struct Waiter {
  uint32_t* abort_flag;  // shared memory
  uint32_t* err;         // device word or nullptr
  MLA_DEV bool aborted() const { return *reinterpret_cast<volatile uint32_t*>(abort_flag) != 0; }
  MLA_DEV void fail() {
    *reinterpret_cast<volatile uint32_t*>(abort_flag) = 1u;
    set_error(err, kErrTimeout);
  }
  template <bool kCluster>
  MLA_DEV bool wait_impl(uint64_t* bar, uint32_t parity, bool drain, uint64_t limit = kWaitNs) {
    const uint32_t a = smem_addr(bar);
    if (kCluster ? mbar_try_wait_cluster(a, parity) : mbar_try_wait(a, parity)) return true;
    const uint64_t t0 = global_timer_ns();
#pragma unroll 1
    while (true) {
      if (kCluster ? mbar_try_wait_cluster(a, parity) : mbar_try_wait(a, parity)) return true;
      if (!drain && aborted()) return false;
      if (global_timer_ns() - t0 > limit) {
        fail();
        return false;
      }
    }
  }
  MLA_DEV bool wait(uint64_t* bar, uint32_t parity, bool drain = false) { return wait_impl<false>(bar, parity, drain); }
  // For phases completed by the other CTA of a pair.
  MLA_DEV bool wait_cluster(uint64_t* bar, uint32_t parity, bool drain = false) {
    return wait_impl<true>(bar, parity, drain);
  }
  // Every lane waits; the outcome is made warp-uniform so that no lane leaves
  // a loop its warp-mates stay in.
  MLA_DEV bool wait_warp(uint64_t* bar, uint32_t parity) { return __all_sync(~0u, wait(bar, parity)); }
  // As wait_warp, for what comes behind `tiles` key tiles of work at a microsecond or two each.
  MLA_DEV bool wait_warp_tiles(uint64_t* bar, uint32_t parity, int tiles) {
    return __all_sync(~0u, wait_impl<false>(bar, parity, false, kWaitNs + (uint64_t)tiles * kTileNs));
  }
};

// a / b for a >= 0, b > 0: one 32-bit division where both fit, else bit by bit
// (a call that long runs for a minute).
MLA_DEV long long quotient(long long a, long long b) {
  if (((unsigned long long)a | (unsigned long long)b) >> 32 == 0) return (uint32_t)a / (uint32_t)b;
  unsigned long long q = 0, r = 0;
#pragma unroll 1
  for (int i = 62; i >= 0; --i) {
    r = (r << 1) | (((unsigned long long)a >> i) & 1u);
    q <<= 1;
    if (r >= (unsigned long long)b) {
      r -= (unsigned long long)b;
      q |= 1u;
    }
  }
  return (long long)q;
}

// Range [*first, *first + return) of sequence b in ragged rows [0, rows):
// offsets outside [0, rows] or out of order are clipped into it, so that no
// caller's offsets make an access leave the rows.
MLA_DEV int ragged_range(const int32_t* offsets, int b, int rows, int* first) {
  const int o0 = __ldg(offsets + b), o1 = __ldg(offsets + b + 1);
  const int a0 = min(max(o0, 0), rows);
  *first = a0;
  return min(max(o1, a0), rows) - a0;
}

// Launch with programmatic stream serialization: the kernel may be set up while
// the one before it in the stream still runs, and reads and writes global memory
// only behind grid_dependency_wait().
template <typename Kernel, typename... Args>
inline cudaError_t launch_dependent(Kernel kernel, dim3 grid, int threads, int smem, cudaStream_t stream,
                                    const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return reported(cudaLaunchKernelEx(&cfg, kernel, args...));
}

}  // namespace prefill
}  // namespace mla
