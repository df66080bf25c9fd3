// Attention of ragged queries over an encoder's states in a paged cache
// (pkv_cross_attention): out = softmax(scale q k^T) v over the n_b states of the row's
// sequence, lse = ln sum e^{scale q k}. Scores are held in log2 units (scale * log2 e).
//
// First form: one warp per (token, query head), lanes across the head; the running maximum
// and sum of the softmax in registers.
#include <cuda_bf16.h>
#include <math.h>

#include "device_common.cuh"
#include "internal.h"
#include "step_ops.h"

namespace pkv {
namespace {

constexpr int kThreads = 128;

template <typename T>
struct Num;
template <>
struct Num<__half> {
  static __device__ __forceinline__ float to(__half x) { return __half2float(x); }
  static __device__ __forceinline__ __half from(float x) { return __float2half_rn(x); }
};
template <>
struct Num<__nv_bfloat16> {
  static __device__ __forceinline__ float to(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ __forceinline__ __nv_bfloat16 from(float x) { return __float2bfloat16_rn(x); }
};

// sequence of token i: the last b with cu[b] <= i, or -1
__device__ __forceinline__ int sequence_of(const CrossParams& p, int i) {
  int lo = 0, hi = p.B - 1, b = -1;
  while (lo <= hi) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(p.cu + mid) <= i) {
      b = mid;
      lo = mid + 1;
    } else {
      hi = mid - 1;
    }
  }
  return b;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) cross_rows_kernel(CrossParams p) {
  constexpr int V = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t w = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5;
  if (blockIdx.x == 0) {   // sequences that take no part or are cut
    int seen = 0;
    for (int b = threadIdx.x; b < p.B; b += kThreads) {
      const int lo = __ldg(p.cu + b), hi = __ldg(p.cu + b + 1), n = __ldg(p.klen + b);
      if (lo < 0 || hi < lo || hi > p.T || hi - lo > p.max_q || n < 0)
        seen |= PKV_DEV_BAD_SEQUENCE;
      else if (hi > lo && n > p.MB * p.BS)
        seen |= PKV_DEV_BAD_BLOCK;
    }
    if (seen) flag_status(p.status, seen);
  }
  if (w >= (int64_t)p.T * p.Hq) return;
  const int i = (int)(w / p.Hq), hq = (int)(w % p.Hq), h = hq / p.G;
  const int b = sequence_of(p, i);
  int n = 0, flags = 0;
  if (b >= 0) {
    const int lo = __ldg(p.cu + b), hi = __ldg(p.cu + b + 1);
    n = __ldg(p.klen + b);
    if (lo < 0 || hi < lo || hi > p.T || hi - lo > p.max_q || n < 0) {
      flags = PKV_DEV_BAD_SEQUENCE;
      n = 0;
    } else if (i >= hi) {
      n = 0;
    } else if (n > p.MB * p.BS) {
      flags = PKV_DEV_BAD_BLOCK;
      n = p.MB * p.BS;
    }
  }
  const T* q = static_cast<const T*>(p.q) + ((int64_t)i * p.Hq + hq) * D;
  float qv[V], o[V];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    qv[k] = Num<T>::to(q[lane * V + k]);
    o[k] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j < n; ++j) {
    const int col = p.bs_shift >= 0 ? j >> p.bs_shift : j / p.BS;
    const int blk = __ldg(p.table + (int64_t)b * p.MB + col);
    if (blk < 0 || blk >= p.NB) {
      flags |= PKV_DEV_BAD_BLOCK;
      continue;
    }
    const int64_t row = (((int64_t)blk * p.BS + (j - col * p.BS)) * p.Hkv + h) * D + lane * V;
    const T* k_ = static_cast<const T*>(p.kc) + row;
    const T* v_ = static_cast<const T*>(p.vc) + row;
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < V; ++k) s += qv[k] * Num<T>::to(k_[k]);
    s = warp_sum(s) * p.scale_log2;
    const float mn = fmaxf(m, s);
    const float base = mn == -INFINITY ? 0.f : mn;   // scores of -inf weigh nothing
    const float a = ex2(m - base), e = ex2(s - base);
    m = mn;
    l = l * a + e;
#pragma unroll
    for (int k = 0; k < V; ++k) o[k] = o[k] * a + e * Num<T>::to(v_[k]);
  }
  T* out = static_cast<T*>(p.out) + ((int64_t)i * p.Hq + hq) * D + lane * V;
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int k = 0; k < V; ++k) out[k] = Num<T>::from(o[k] * inv);
  if (lane == 0) {
    if (p.lse) p.lse[(int64_t)i * p.Hq + hq] = l > 0.f ? m * kLn2 + logf(l) : -INFINITY;
    if (flags) flag_status(p.status, flags);
  }
}

}  // namespace

size_t cross_workspace_bytes(const CrossParams& p) {
  (void)p;
  return 256;
}

cudaError_t launch_cross(const CrossParams& p, void* workspace, cudaStream_t s) {
  (void)workspace;
  ProfScope ps("cross_decode", s);
  const unsigned grid = (unsigned)(((int64_t)p.T * p.Hq * 32 + kThreads - 1) / kThreads);
  if (p.bf16) {
    if (p.D == 64)
      cross_rows_kernel<__nv_bfloat16, 64><<<grid, kThreads, 0, s>>>(p);
    else
      cross_rows_kernel<__nv_bfloat16, 128><<<grid, kThreads, 0, s>>>(p);
  } else {
    if (p.D == 64)
      cross_rows_kernel<__half, 64><<<grid, kThreads, 0, s>>>(p);
    else
      cross_rows_kernel<__half, 128><<<grid, kThreads, 0, s>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace pkv
