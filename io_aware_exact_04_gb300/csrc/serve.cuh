// What the serving kernels (prompts, drafted trees, the cache in pages) share.
#pragma once
#include <cstdint>

#include "common.cuh"

namespace fa {

// Check sites recorded with FA_ERR_DEVICE_CHECK by the serving kernels.
enum { SITE_S_OFFSETS = 50, SITE_S_LENGTH, SITE_S_PAGE, SITE_S_ROW, SITE_S_PARENT, SITE_S_WORDS, SITE_S_SLOT,
       SITE_S_SMEM };

// Bounded waits of the serving kernels, by a whole warp. They give up after kWaitLimitNs, as the
// other kernels' do, and when another CTA has; not when a check was recorded, as these kernels
// carry on past the values that they check. The waiting part is out of line: a warp that mostly
// finds its phase complete then runs through less code, and the issuing warps' own time bounds
// the steps of these kernels.
__device__ __noinline__ inline bool wait_slow(uint32_t bar, uint32_t parity, DevStatus st, int site) {
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t spins = 1;; ++spins) {
    if (__all_sync(0xffffffffu, mbar_try_wait_sleep(bar, parity, 20000u))) return true;
    if ((spins & 7u) != 0) continue;
    bool give_up = *(volatile int*)st.abort_smem != 0;
    if (!give_up && *(volatile int*)st.word == FA_ERR_TIMEOUT) {
      *(volatile int*)st.abort_smem = 1;
      give_up = true;
    }
    if (!give_up && globaltimer_ns() - t0 > kWaitLimitNs) {
      record_error(st, FA_ERR_TIMEOUT, site);
      give_up = true;
    }
    if (__any_sync(0xffffffffu, give_up)) return false;
  }
}
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, DevStatus st, int site) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return wait_slow(bar, parity, st, site);
}

// The tokens [lo, hi) of sequence b, cut to [0, T): offsets are the caller's device data.
struct SeqRange {
  int lo, hi;
};
__device__ __forceinline__ SeqRange seq_range(const int* cu, int b, int T, int* status) {
  const int lo = cu[b], hi = cu[b + 1];
  SeqRange r;
  r.lo = min(max(lo, 0), T);
  r.hi = min(max(hi, r.lo), T);
  if (r.lo != lo || r.hi != hi) record_check(status, SITE_S_OFFSETS);
  return r;
}

// The sequence of token t by a whole warp: the last b with cu[b] <= t (the offsets do not
// decrease), 32 candidates a step; -1 where t lies before the first or behind the last one.
__device__ __forceinline__ int find_sequence(const int* cu, int B, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = B + 1;  // the answer's candidates: [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int i = lo + min(lane * step, n - 1);
    const unsigned below = __ballot_sync(0xffffffffu, cu[i] <= t);
    if (below == 0) return -1;
    const int k = 31 - __clz(below);
    const int at = min(k * step, n - 1);
    n = min(step, n - at);
    lo += at;
  }
  return (lo < B && cu[lo] <= t) ? lo : -1;
}

// All offsets, by one block: kernels with a block or warp for each token never meet a sequence
// that no token lies in.
__device__ __forceinline__ void check_offsets(const int* cu, int B, int T, int* status) {
  for (int b = threadIdx.x; b < B; b += blockDim.x) seq_range(cu, b, T, status);
}

}  // namespace fa
