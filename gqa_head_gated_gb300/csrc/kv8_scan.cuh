// Prefix sums that the block planning kernels (kv8_plan.cu, kv8_pages.cu) share.
#pragma once

#include <cuda_runtime.h>

namespace gqa {
namespace {

// Exclusive prefix sums of two arrays of n counts in place; returns both totals.
template <int kThreads>
__device__ int2 scan2(int* a, int* b, int n, int2* part) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (n + kThreads - 1) / kThreads;
  const int lo = min(tid * per, n), hi = min(lo + per, n);
  int2 s = make_int2(0, 0);
  for (int i = lo; i < hi; ++i) {
    s.x += a[i];
    s.y += b[i];
  }
  int2 v = s;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, v.x, o), y = __shfl_up_sync(0xffffffffu, v.y, o);
    if (lane >= o) {
      v.x += x;
      v.y += y;
    }
  }
  if (lane == 31) part[warp] = v;
  __syncthreads();
  int2 before = make_int2(0, 0), total = make_int2(0, 0);
  for (int w = 0; w < kThreads / 32; ++w) {
    const int2 p = part[w];
    if (w < warp) {
      before.x += p.x;
      before.y += p.y;
    }
    total.x += p.x;
    total.y += p.y;
  }
  int2 run = make_int2(before.x + v.x - s.x, before.y + v.y - s.y);
  for (int i = lo; i < hi; ++i) {
    const int x = a[i], y = b[i];
    a[i] = run.x;
    b[i] = run.y;
    run.x += x;
    run.y += y;
  }
  __syncthreads();
  return total;
}

// The last index whose first rank (exclusive sum) is at most k: the one that has rank k.
__device__ __forceinline__ int owner_of(const int* sums, int n, int k) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (sums[mid] <= k) lo = mid; else hi = mid - 1;
  }
  return lo;
}

}  // namespace
}  // namespace gqa
