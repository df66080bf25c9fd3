// K and V of new tokens into the paged cache, with rotary positions of several axes
// (pkv_paged_append_rotary_axes).
//
// Pair j of a head turns by the angle of table row pos[axis(j)][token], column j:
//   lead' = lead * cos - trail * sin,   trail' = trail * cos + lead * sin
// in fp32, rounded once. Every element is read once and written once: the operator is bound
// by HBM, 4 * (Hq + 2 Hkv) * D bytes per token.
//
// A thread moves one item: 16 elements of a rotated head (8 pairs: two 16-byte chunks rotary_dim
// / 2 apart, or side by side), or two chunks that are only copied. The token's cos and sin, one
// of each a pair, are gathered once into shared memory, whatever the axes' order, while the
// item's own loads are under way, and so are the token's slot and whether it may be written. A
// block is one token's items, or several tokens' where a token has few. Rotary dimensions that are no multiple of 16 take a thread a chunk and read each
// partner by itself.
#include <cuda_bf16.h>

#include "device_common.cuh"
#include "internal.h"
#include "step_ops.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;      // of the second kernel; and what the first fills with tokens
constexpr int kMaxThreads = 512;

template <typename T>
struct Num;
template <>
struct Num<__half> {
  static __device__ __forceinline__ float to(__half x) { return __half2float(x); }
  static __device__ __forceinline__ __half from(float x) { return __float2half_rn(x); }
  static __device__ __forceinline__ float2 to2(uint32_t x) {
    return __half22float2(*reinterpret_cast<const __half2*>(&x));
  }
  static __device__ __forceinline__ uint32_t from2(float a, float b) { return pack_half2(a, b); }
};
template <>
struct Num<__nv_bfloat16> {
  static __device__ __forceinline__ float to(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ __forceinline__ __nv_bfloat16 from(float x) { return __float2bfloat16_rn(x); }
  static __device__ __forceinline__ float2 to2(uint32_t x) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&x));
  }
  static __device__ __forceinline__ uint32_t from2(float a, float b) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&x);
  }
};
template <>
struct Num<float> {
  static __device__ __forceinline__ float to(float x) { return x; }
};

// What stops a token's key and value rows; reported by one thread.
struct Token {
  int slot;
  bool known, fits;   // every axis in use has a table row; the slot lies in the pool
};
__device__ __forceinline__ Token read_token(const AxesParams& p, int t) {
  Token k;
  k.slot = __ldg(p.slots + t);
  k.known = true;
  for (int a = 0; a < p.axes; ++a)
    if ((p.used_axes >> a) & 1u) {
      const int x = __ldg(p.pos + (int64_t)a * p.T + t);
      k.known = k.known && x >= 0 && x < p.P;
    }
  k.fits = k.slot < p.pool_rows;
  return k;
}
__device__ __forceinline__ void report(const AxesParams& p, const Token& k) {
  if (k.slot >= 0 && (!k.known || !k.fits))
    flag_status(p.status, (k.known ? 0 : PKV_DEV_BAD_POSITION) | (k.fits ? 0 : PKV_DEV_BAD_SLOT));
}

// items: items of a token; tokens: tokens that a block holds side by side (1 when a token has
// more items than threads). A thread does the same item of N tokens, `tokens` apart.
template <typename T, typename TT, bool kSide, int N>
__global__ void __launch_bounds__(kMaxThreads)
    append_axes_items_kernel(const __grid_constant__ AxesParams p, int items, int tokens) {
  // [N * tokens][4][R / 16] (cos, cos, sin, sin) of pairs 2 y and 2 y + 1 of item c at [y][c], so
  // that neighbouring threads read neighbouring words; then (slot, flags) of each token
  extern __shared__ __align__(16) float4 turn[];
  const int half = p.R / 2, cpr = p.D / 8;
  const int per_head = p.R / 16, rotated = (p.Hq + p.Hkv) * per_head;
  const int plain = cpr - 2 * per_head;            // chunks of a rotated head behind rotary_dim
  const int t0 = blockIdx.x * tokens * N;
  const int mine = tokens > 1 ? threadIdx.x / items : 0;
  const bool there = mine < tokens;
  const int step = tokens > 1 ? items : blockDim.x;
  int i = tokens > 1 ? threadIdx.x - mine * items : threadIdx.x;
  int2* about = reinterpret_cast<int2*>(turn + N * tokens * per_head * 4);

  // the two chunks of item i: where they are read and written from token 0 (slot 0) on, and what
  // they are (0 query, 1 key, 2 value, 3 nothing)
  const T* src[2];
  T* dst[2];
  int kind[2];
  const int q_row = p.Hq * p.D, kv_row = p.Hkv * p.D;
  const auto place = [&](int i) {
    int h[2], ch[2];
    if (i < rotated) {
      h[0] = h[1] = i / per_head;
      const int c = i - h[0] * per_head;
      ch[0] = kSide ? 2 * c : c;
      ch[1] = kSide ? 2 * c + 1 : c + per_head;
    } else {
      const int values = p.Hkv * cpr, all = values + (p.Hq + p.Hkv) * plain;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int n = 2 * (i - rotated) + x;
        h[x] = n < values ? p.Hq + p.Hkv + n / cpr : n < all ? (n - values) / plain : -1;
        ch[x] = n < values ? n % cpr : n < all ? 2 * per_head + (n - values) % plain : 0;
      }
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      kind[x] = h[x] < 0 ? 3 : h[x] < p.Hq ? 0 : h[x] < p.Hq + p.Hkv ? 1 : 2;
      const int hh = kind[x] == 0 ? h[x] : kind[x] == 1 ? h[x] - p.Hq : h[x] - p.Hq - p.Hkv;
      const int e = hh * p.D + ch[x] * 8;
      src[x] = static_cast<const T*>(kind[x] == 0 ? p.q : kind[x] == 1 ? p.k : p.v) + e;
      dst[x] = static_cast<T*>(kind[x] == 0 ? p.q_out : kind[x] == 1 ? p.kc : p.vc) + e;
    }
  };
  uint4 x[N][2];
  const auto load = [&]() {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int t = t0 + mine + n * tokens;
#pragma unroll
      for (int y = 0; y < 2; ++y)
        if (t < p.T && kind[y] < 3)
          x[n][y] = __ldcs(reinterpret_cast<const uint4*>(
              src[y] + (int64_t)t * (kind[y] == 0 ? p.q_stride : p.kv_stride)));
    }
  };
  const bool any = there && i < items;
  if (any) {
    place(i);
    load();
  }
  if (threadIdx.x < N * tokens && t0 + threadIdx.x < p.T) {
    const Token k = read_token(p, t0 + threadIdx.x);
    report(p, k);
    about[threadIdx.x] = make_int2(k.slot, (k.known ? 1 : 0) | (k.known && k.fits ? 2 : 0));
  }
  for (int n = threadIdx.x; n < N * tokens * half; n += blockDim.x) {
    const int w = n / half, j = n - w * half;
    if (t0 + w >= p.T) break;
    const int r = __ldg(p.pos + (int64_t)p.pair_axis[j] * p.T + t0 + w);
    if (r >= 0 && r < p.P) {
      const int64_t at = (int64_t)r * half + j;
      float* z = reinterpret_cast<float*>(turn + (w * 4 + (j & 7) / 2) * per_head + j / 8) + (j & 1);
      z[0] = Num<TT>::to(static_cast<const TT*>(p.cos)[at]);
      z[2] = Num<TT>::to(static_cast<const TT*>(p.sin)[at]);
    }
  }
  __syncthreads();
  while (any) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int w = mine + n * tokens;
      if (t0 + w >= p.T) break;
      const int2 k = about[w];
      if (k.x < 0) continue;
      if (i < rotated && (k.y & 1)) {
        const float4* cs = turn + w * 4 * per_head + i % per_head;
        uint32_t* a = reinterpret_cast<uint32_t*>(&x[n][0]);
        uint32_t* b = reinterpret_cast<uint32_t*>(&x[n][1]);
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const float4 c = cs[y * per_head];
          if constexpr (kSide) {        // a pair is one 32-bit word
            uint32_t* z = y < 2 ? a + 2 * y : b + 2 * (y - 2);
            const float2 u = Num<T>::to2(z[0]), v = Num<T>::to2(z[1]);
            z[0] = Num<T>::from2(u.x * c.x - u.y * c.z, u.y * c.x + u.x * c.z);
            z[1] = Num<T>::from2(v.x * c.y - v.y * c.w, v.y * c.y + v.x * c.w);
          } else {
            const float2 u = Num<T>::to2(a[y]), v = Num<T>::to2(b[y]);
            a[y] = Num<T>::from2(u.x * c.x - v.x * c.z, u.y * c.y - v.y * c.w);
            b[y] = Num<T>::from2(v.x * c.x + u.x * c.z, v.y * c.y + u.y * c.w);
          }
        }
      }
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        if (kind[y] == 0)
          *reinterpret_cast<uint4*>(dst[y] + (int64_t)(t0 + w) * q_row) = x[n][y];
        else if (kind[y] < 3 && (k.y & 2))
          *reinterpret_cast<uint4*>(dst[y] + (int64_t)k.x * kv_row) = x[n][y];
      }
    }
    i += step;
    if (tokens > 1 || i >= items) break;
    place(i);
    load();
  }
}

// Any rotary_dim: one block per token, a thread moves chunks of 8 elements.
template <typename T, typename TT>
__global__ void __launch_bounds__(kThreads)
    append_axes_chunks_kernel(const __grid_constant__ AxesParams p) {
  const int t = blockIdx.x;
  const Token k = read_token(p, t);
  if (k.slot < 0) return;
  if (threadIdx.x == 0) report(p, k);
  const bool write_kv = k.known && k.fits;
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
                 : static_cast<T*>(isv ? p.vc : p.kc) + ((int64_t)k.slot * p.Hkv + kh) * p.D;
    __align__(16) T x[8];
    *reinterpret_cast<uint4*>(x) = *reinterpret_cast<const uint4*>(src + c * 8);
    if (!isv && k.known) {
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

template <typename T, typename TT, int N>
void launch_items(const AxesParams& p, int items, int tokens, int threads, cudaStream_t s) {
  const unsigned grid = (unsigned)((p.T + tokens * N - 1) / (tokens * N));
  const size_t smem = (size_t)tokens * N * (sizeof(float4) * (p.R / 4) + sizeof(int2));
  if (p.interleaved)
    append_axes_items_kernel<T, TT, true, N><<<grid, threads, smem, s>>>(p, items, tokens);
  else
    append_axes_items_kernel<T, TT, false, N><<<grid, threads, smem, s>>>(p, items, tokens);
}

template <typename T, typename TT>
void launch_typed(const AxesParams& p, cudaStream_t s) {
  if (p.R % 16 != 0) {
    append_axes_chunks_kernel<T, TT><<<p.T, kThreads, 0, s>>>(p);
    return;
  }
  const int cpr = p.D / 8, per_head = p.R / 16;
  const int copied = p.Hkv * cpr + (p.Hq + p.Hkv) * (cpr - 2 * per_head);
  const int items = (p.Hq + p.Hkv) * per_head + (copied + 1) / 2;
  const int tokens = items * 2 <= kThreads ? kThreads / items : 1;
  const int threads = tokens > 1 ? (tokens * items + 31) / 32 * 32
                                 : (items < kMaxThreads ? (items + 31) / 32 * 32 : kMaxThreads);
  // Many tokens: four to a thread, so that enough of their loads are under way at once; few: one,
  // so that they are spread over the SMs. MEASURED
  if (p.T >= 4 * tokens * 2 * device_sms())
    launch_items<T, TT, 4>(p, items, tokens, threads, s);
  else
    launch_items<T, TT, 1>(p, items, tokens, threads, s);
}

}  // namespace

cudaError_t launch_append_axes(const AxesParams& p, cudaStream_t s) {
  ProfScope ps("append_axes", s);
  if (p.bf16) {
    if (p.table_f32)
      launch_typed<__nv_bfloat16, float>(p, s);
    else
      launch_typed<__nv_bfloat16, __nv_bfloat16>(p, s);
  } else {
    if (p.table_f32)
      launch_typed<__half, float>(p, s);
    else
      launch_typed<__half, __half>(p, s);
  }
  return cudaGetLastError();
}

}  // namespace pkv
