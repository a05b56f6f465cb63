// What the serving kernels (prompts, drafted trees, the cache in pages) share.
#pragma once
#include <cstdint>

#include "common.cuh"

namespace fa {

// Check sites recorded with FA_ERR_DEVICE_CHECK by the serving kernels.
enum { SITE_S_OFFSETS = 40, SITE_S_LENGTH, SITE_S_PAGE, SITE_S_ROW, SITE_S_PARENT, SITE_S_WORDS, SITE_S_SLOT };

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
