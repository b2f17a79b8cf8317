// Finding a token's request and its row of the paged pool, shared by the
// kernels that write and read cache pages.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "common.cuh"

namespace msa {

// The request of token t: the number of requests b with cu[b + 1] <= t,
// found by a whole warp, 32 probes a step (B <= 32: one step, B <= 1024:
// two).  All lanes get the result, in [0, B]; B when no request holds t.
// Any contents of cu give an index in range.
__device__ __forceinline__ int warp_request_of(const int32_t* __restrict__ cu, int B, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = B;  // the answer lies in [lo, lo + n]
  while (n > 0) {
    const int step = (n + 31) / 32;
    const int i = lo + (lane + 1) * step;  // probe cu[i], the end of request i - 1
    const bool below = i <= lo + n && __ldg(cu + i) <= t;
    const int k = __popc(__ballot_sync(0xffffffffu, below));
    // cu[lo + k * step] <= t < cu[lo + (k + 1) * step] (or past the end)
    lo += k * step;
    n = step == 1 ? 0 : min(step - 1, n - k * step);
  }
  return lo;
}

// The same for 32 consecutive tokens at once, lane i's being `first + i`: the
// first one's request by the search above; lanes whose token lies behind it
// search on from there.
__device__ __forceinline__ int lane_request_of(const int32_t* __restrict__ cu, int B, int first) {
  const int t = first + (int)(threadIdx.x & 31);
  int lo = warp_request_of(cu, B, first);
  if (lo < B && __ldg(cu + lo + 1) <= t) {
    int hi = B;  // the answer lies in (lo, hi]
    ++lo;
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (__ldg(cu + mid + 1) <= t) lo = mid + 1; else hi = mid;
    }
  }
  return lo;
}

// The row of the pool (page * 128 + offset) that position `pos` of request b
// lies in, or -1 with a status bit in *bad.
__device__ __forceinline__ int64_t pool_row(const int32_t* __restrict__ block_table,
                                            int64_t bt_stride, int64_t num_pages, int b,
                                            int64_t pos, uint32_t* bad) {
  if (pos < 0 || pos / kPage >= bt_stride) {
    *bad |= MSA_STATUS_BAD_SEQLENS;
    return -1;
  }
  const int page = __ldg(block_table + b * bt_stride + pos / kPage);
  if (page < 0 || page >= num_pages) {
    *bad |= MSA_STATUS_BAD_BLOCK;
    return -1;
  }
  return (int64_t)page * kPage + pos % kPage;
}

}  // namespace msa
