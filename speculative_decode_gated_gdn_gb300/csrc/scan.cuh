// scan.cuh -- prefix sums of one CTA, for the bookkeeping kernels.
#pragma once

#include "gdn_common.cuh"

namespace gdn {

constexpr int kScanThreads = 1024;

// Inclusive scan of v over the CTA; *total gets the sum of all threads.
__device__ __forceinline__ long long block_scan(long long v, long long *s_warp, long long *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  sync_cta();  // s_warp may still be read by an earlier scan
  if (lane == 31) s_warp[warp] = v;
  sync_cta();
  if (warp == 0) {
    long long w = s_warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += u;
    }
    s_warp[lane] = w;
  }
  sync_cta();
  *total = s_warp[31];
  return v + (warp ? s_warp[warp - 1] : 0);
}

// First index i in [0, n) with ends[i] > x (ends ascending, ends[n - 1] > x).
__device__ __forceinline__ int find_row(const int *ends, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int m = (lo + hi) >> 1;
    if (ends[m] > x) hi = m;
    else lo = m + 1;
  }
  return lo;
}

}  // namespace gdn
