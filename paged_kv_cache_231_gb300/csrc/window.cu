// Causal attention over the paged cache with a sliding window (pkv_paged_window_attention) and
// behind a shared prefix (pkv_paged_prefix_attention): a row at position t sees keys j <= t with
// j > t - window or j < sinks; out = sum_j e^{s_j - lse} v_j, lse = ln sum_j e^{s_j}.
// The simplest form: a warp for a query row and head, one key after the other, all in fp32.
#include <cmath>

#include "cross_dev.cuh"

namespace pkv {
namespace {

using namespace cross;

template <typename T>
__device__ __forceinline__ float wide(T x);
template <>
__device__ __forceinline__ float wide(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float wide(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T, int D>
__global__ void __launch_bounds__(256) window_rows_kernel(CrossParams p) {
  constexpr int V = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (unit >= (int64_t)p.T * p.Hq) return;
  const int row = (int)(unit / p.Hq), h = (int)(unit - (int64_t)row * p.Hq), kv = h / p.G;
  int flags = 0, seq = 0;
  int64_t pos = -1;
  const int limit = p.MB * p.BS;
  for (int b = 0; b < p.B; ++b) {
    const int lo = __ldg(p.cu + b), hi = __ldg(p.cu + b + 1), past = __ldg(p.past + b);
    if (lo < 0 || hi < lo || hi > p.T || hi - lo > p.max_q || past < 0) {
      flags |= PKV_DEV_BAD_SEQUENCE;
    } else if (row >= lo && row < hi) {
      pos = (int64_t)past + row - lo;
      seq = b;
    }
  }
  float q[V], o[V], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    q[v] = wide(static_cast<const T*>(p.q)[unit * D + v * 32 + lane]) * p.scale_log2;
    o[v] = 0.f;
  }
  if (pos >= limit) flags |= PKV_DEV_BAD_BLOCK;
  const int end = (int)min(pos + 1, (int64_t)limit);
  for (int j = 0; j < end; ++j) {
    if (p.window > 0 && j <= pos - p.window && j >= p.sinks) continue;
    const int col = j / p.BS, blk = __ldg(p.table + (int64_t)seq * p.MB + col);
    if (blk < 0 || blk >= p.NB) {
      flags |= PKV_DEV_BAD_BLOCK;
      continue;
    }
    const int64_t at = (((int64_t)blk * p.BS + (j - col * p.BS)) * p.Hkv + kv) * D + lane;
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) s += q[v] * wide(static_cast<const T*>(p.kc)[at + v * 32]);
    s = warp_sum(s);
    const float top = fmaxf(m, s), base = top == -INFINITY ? 0.f : top;
    const float old = ex2(m - base), w = ex2(s - base);
    m = top;
    l = l * old + w;
#pragma unroll
    for (int v = 0; v < V; ++v)
      o[v] = o[v] * old + w * wide(static_cast<const T*>(p.vc)[at + v * 32]);
  }
  const float inv = inverse_of(l);
#pragma unroll
  for (int v = 0; v < V; ++v)
    static_cast<T*>(p.out)[unit * D + v * 32 + lane] = static_cast<T>(o[v] * inv);
  if (p.lse && lane == 0) p.lse[unit] = lse_of(m, l);
  if (flags && lane == 0) flag_status(p.status, flags);
}

template <typename T>
void launch_typed(const CrossParams& p, cudaStream_t s) {
  const unsigned grid = (unsigned)(((int64_t)p.T * p.Hq + 7) / 8);
  if (p.D == 64)
    window_rows_kernel<T, 64><<<grid, 256, 0, s>>>(p);
  else
    window_rows_kernel<T, 128><<<grid, 256, 0, s>>>(p);
}

}  // namespace

cudaError_t launch_window(const CrossParams& p, cudaStream_t s) {
  ProfScope ps("window_decode", s);
  if (p.bf16)
    launch_typed<__nv_bfloat16>(p, s);
  else
    launch_typed<__half>(p, s);
  return cudaGetLastError();
}

}  // namespace pkv
