// What the kernels that go through rows and block ids of the pool share (one block of 1024
// threads, or a cluster of them): a prefix sum and a search.
#pragma once

#include "device_common.cuh"

namespace pkv {
namespace pool {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;

// Inclusive sum over the block's threads; *total gets the sum of all. scratch: kWarps words that
// neither the call before nor the one behind uses.
template <typename T>
__device__ __forceinline__ T block_sum(T v, T* total, T* scratch) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  if (lane == 31) scratch[w] = v;
  __syncthreads();
  T upto = scratch[lane];   // every warp sums the warps' sums for itself
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  *total = __shfl_sync(0xffffffffu, upto, kWarps - 1);
  const T before = __shfl_sync(0xffffffffu, upto, w > 0 ? w - 1 : 0);
  return w > 0 ? v + before : v;
}

// first index i of the ascending a[0, n) with a[i] > x (n when there is none)
__device__ __forceinline__ int first_above(const int* a, int n, int x) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] > x)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

}  // namespace pool
}  // namespace pkv
