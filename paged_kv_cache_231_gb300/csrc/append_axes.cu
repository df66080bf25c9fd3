// K and V of new tokens into the paged cache, with rotary positions of several axes
// (pkv_paged_append_rotary_axes).
//
// Pair j of a head turns by the angle of table row pos[axis(j)][token], column j:
//   lead' = lead * cos - trail * sin,   trail' = trail * cos + lead * sin
// in fp32, rounded once. Every element is read once and written once: the operator is bound
// by HBM, 4 * (Hq + 2 Hkv) * D bytes per token.
#include <cuda_bf16.h>

#include "device_common.cuh"
#include "internal.h"
#include "step_ops.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;

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
template <>
struct Num<float> {
  static __device__ __forceinline__ float to(float x) { return x; }
};

// One block per token; a thread moves chunks of 8 elements.
template <typename T, typename TT>
__global__ void __launch_bounds__(kThreads) append_axes_kernel(AxesParams p) {
  const int t = blockIdx.x;
  const int slot = __ldg(p.slots + t);
  if (slot < 0) return;
  bool known = true;   // every axis in use has a table row
  for (int a = 0; a < p.axes; ++a)
    if ((p.used_axes >> a) & 1u) {
      const int x = __ldg(p.pos + (int64_t)a * p.T + t);
      known = known && x >= 0 && x < p.P;
    }
  const bool fits = slot < p.pool_rows;
  if (threadIdx.x == 0 && (!known || !fits))
    flag_status(p.status, (known ? 0 : PKV_DEV_BAD_POSITION) | (fits ? 0 : PKV_DEV_BAD_SLOT));
  const bool write_kv = known && fits;
  const int cpr = p.D / 8, half = p.R / 2;
  const TT* cs = static_cast<const TT*>(p.cos);
  const TT* sn = static_cast<const TT*>(p.sin);
  const int heads = p.Hq + 2 * p.Hkv;
  for (int u = threadIdx.x; u < heads * cpr; u += kThreads) {
    const int h = u / cpr, c = u % cpr;
    const bool isq = h < p.Hq, isv = h >= p.Hq + p.Hkv;
    if (!isq && !write_kv) continue;
    const int kh = isv ? h - p.Hq - p.Hkv : h - p.Hq;
    const T* src = isq ? static_cast<const T*>(p.q) + (int64_t)t * p.q_stride + (int64_t)h * p.D
                       : static_cast<const T*>(isv ? p.v : p.k) + (int64_t)t * p.kv_stride + (int64_t)kh * p.D;
    T* dst = isq ? static_cast<T*>(p.q_out) + ((int64_t)t * p.Hq + h) * p.D
                 : static_cast<T*>(isv ? p.vc : p.kc) + ((int64_t)slot * p.Hkv + kh) * p.D;
    __align__(16) T x[8];
    *reinterpret_cast<uint4*>(x) = *reinterpret_cast<const uint4*>(src + c * 8);
    if (!isv && known) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int i = c * 8 + e;
        if (i >= p.R) break;
        const int j = p.interleaved ? i >> 1 : (i < half ? i : i - half);
        const bool lead = p.interleaved ? (i & 1) == 0 : i < half;
        const int other = p.interleaved ? i ^ 1 : (lead ? i + half : i - half);
        const int64_t at = (int64_t)__ldg(p.pos + (int64_t)p.pair_axis[j] * p.T + t) * half + j;
        const float co = Num<TT>::to(cs[at]), si = Num<TT>::to(sn[at]);
        const float own = Num<T>::to(src[i]), mate = Num<T>::to(src[other]);
        x[e] = Num<T>::from(lead ? own * co - mate * si : own * co + mate * si);
      }
    }
    *reinterpret_cast<uint4*>(dst + c * 8) = *reinterpret_cast<const uint4*>(x);
  }
}

template <typename T>
void launch_typed(const AxesParams& p, cudaStream_t s) {
  if (p.table_f32)
    append_axes_kernel<T, float><<<p.T, kThreads, 0, s>>>(p);
  else
    append_axes_kernel<T, T><<<p.T, kThreads, 0, s>>>(p);
}

}  // namespace

cudaError_t launch_append_axes(const AxesParams& p, cudaStream_t s) {
  ProfScope ps("append_axes", s);
  if (p.bf16)
    launch_typed<__nv_bfloat16>(p, s);
  else
    launch_typed<__half>(p, s);
  return cudaGetLastError();
}

}  // namespace pkv
