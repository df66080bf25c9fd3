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
// block is one token's items, or several tokens' where a token has few. Rotary dimensions that
// are no multiple of 16 take a thread a chunk and read each partner by itself.
// Measured (32 + 2 x 8 heads of 128): 64 tokens 3.6 us, which is latency; 32768 tokens 134 us.
#include "append_dev.cuh"

namespace pkv {
namespace {

using append::Token;
using append::read_token;
using append::report;
using elem::Num;

constexpr int kThreads = 256;      // of the second kernel; and what the first fills with tokens
constexpr int kMaxThreads = 512;

// The two chunks of item i of a token: where they are read and written from token 0 (slot 0) on.
template <typename T>
struct Item {
  const T* src[2];
  T* dst[2];
  int kind[2];   // 0 query, 1 key, 2 value, 3 nothing
  template <bool kSide>
  __device__ __forceinline__ void place(const AxesParams& p, int i) {
    const int cpr = p.D / 8, per_head = p.R / 16, rotated = (p.Hq + p.Hkv) * per_head;
    const int plain = cpr - 2 * per_head;   // chunks of a rotated head behind rotary_dim
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
  }
  __device__ __forceinline__ void load(const AxesParams& p, int t, uint4 (&x)[2]) const {
#pragma unroll
    for (int y = 0; y < 2; ++y)
      if (kind[y] < 3)
        x[y] = __ldcs(reinterpret_cast<const uint4*>(
            src[y] + (int64_t)t * (kind[y] == 0 ? p.q_stride : p.kv_stride)));
  }
  // about: the token's slot, and 1 for known | 2 for known and inside the pool
  __device__ __forceinline__ void store(const AxesParams& p, int t, int2 about,
                                        const uint4 (&x)[2]) const {
    const int q_row = p.Hq * p.D, kv_row = p.Hkv * p.D;
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      if (kind[y] == 0)
        *reinterpret_cast<uint4*>(dst[y] + (int64_t)t * q_row) = x[y];
      else if (kind[y] < 3 && (about.y & 2))
        *reinterpret_cast<uint4*>(dst[y] + (int64_t)about.x * kv_row) = x[y];
    }
  }
};

// Turns the 8 pairs of an item; cs[y * apart]: (cos, cos, sin, sin) of pairs 2 y and 2 y + 1.
template <typename T, bool kSide>
__device__ __forceinline__ void turn_item(uint4 (&x)[2], const float4* cs, int apart) {
  uint32_t* a = reinterpret_cast<uint32_t*>(&x[0]);
  uint32_t* b = reinterpret_cast<uint32_t*>(&x[1]);
#pragma unroll
  for (int y = 0; y < 4; ++y) {
    const float4 c = cs[y * apart];
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

// Many tokens of many items: a block stays and goes through groups of two tokens. While one group
// is turned and written, the next one's rows and table entries are on their way and the slots and
// positions of the one behind it, so that loads are under way all the time.
constexpr int kPair = 2;
constexpr int kStreamFrom = 3;   // tokens an SM
template <typename T, typename TT, bool kSide>
__global__ void __launch_bounds__(kMaxThreads)
    append_axes_stream_kernel(const __grid_constant__ AxesParams p, int items) {
  extern __shared__ __align__(16) float4 turn[];   // [2][kPair][4][R / 16], as below; then about
  const int half = p.R / 2, per_head = p.R / 16, rotated = (p.Hq + p.Hkv) * per_head;
  const int words = kPair * per_head * 4;          // of a group
  int2* about = reinterpret_cast<int2*>(turn + 2 * words);   // [2][kPair]
  const int i = threadIdx.x, groups = (p.T + kPair - 1) / kPair;
  const bool mine = i < items;
  Item<T> it;
  if (mine) it.template place<kSide>(p, i);
  // this thread's share of the gathering: pair gj of token gw of a group; the first threads look
  // after the tokens themselves
  const bool gathers = i < kPair * half;
  const int gw = gathers ? i / half : 0, gj = gathers ? i - gw * half : 0;
  const int* gpos = gathers ? p.pos + (int64_t)p.pair_axis[gj] * p.T : nullptr;
  float* const put =
      reinterpret_cast<float*>(turn + (gw * 4 + (gj & 7) / 2) * per_head + gj / 8) + (gj & 1);
  const int tw = i;                                // token of the group that this thread reports

  const auto row_of = [&](int g) {                 // table row of this thread's pair, -1: none
    const int t = g * kPair + gw;
    return gathers && g < groups && t < p.T ? __ldg(gpos + t) : -1;
  };
  const auto fetch = [&](int r, float& c, float& s) {
    if (r >= 0 && r < p.P) {
      const int64_t at = (int64_t)r * half + gj;
      c = Num<TT>::to(__ldg(static_cast<const TT*>(p.cos) + at));
      s = Num<TT>::to(__ldg(static_cast<const TT*>(p.sin) + at));
    }
  };
  uint4 x[kPair][2], ahead[kPair][2];
  const auto load = [&](int g, uint4 (&v)[kPair][2]) {
#pragma unroll
    for (int n = 0; n < kPair; ++n)
      if (mine && g < groups && g * kPair + n < p.T) it.load(p, g * kPair + n, v[n]);
  };
  const auto token = [&](int g, int buf) {
    const int t = g * kPair + tw;
    if (tw < kPair && g < groups && t < p.T) {
      const Token k = read_token(p, t);
      report(p, k);
      about[buf * kPair + tw] = make_int2(k.slot, (k.known ? 1 : 0) | (k.known && k.fits ? 2 : 0));
    }
  };

  int g = blockIdx.x;
  const int apart = gridDim.x;
  float c = 0.f, s = 0.f;
  load(g, x);
  fetch(row_of(g), c, s);
  int row = row_of(g + apart);
  token(g, 0);
  if (gathers) {
    put[0] = c;
    put[2] = s;
  }
  __syncthreads();
  for (int buf = 0; g < groups; g += apart, buf ^= 1) {
    load(g + apart, ahead);
    fetch(row, c, s);
    row = row_of(g + 2 * apart);
    token(g + apart, buf ^ 1);
#pragma unroll
    for (int n = 0; n < kPair; ++n) {
      const int t = g * kPair + n;
      if (!mine || t >= p.T) break;
      const int2 k = about[buf * kPair + n];
      if (k.x < 0) continue;
      if (i < rotated && (k.y & 1))
        turn_item<T, kSide>(x[n], turn + buf * words + n * 4 * per_head + i % per_head, per_head);
      it.store(p, t, k, x[n]);
    }
    if (gathers) {
      put[(buf ^ 1) * words * 4] = c;
      put[(buf ^ 1) * words * 4 + 2] = s;
    }
#pragma unroll
    for (int n = 0; n < kPair; ++n)
#pragma unroll
      for (int y = 0; y < 2; ++y) x[n][y] = ahead[n][y];
    __syncthreads();
  }
}

// items: items of a token; tokens: tokens that a block holds side by side (1 when a token has
// more items than threads). A thread does the same item of N tokens, `tokens` apart.
template <typename T, typename TT, bool kSide, int N>
__global__ void __launch_bounds__(kMaxThreads)
    append_axes_items_kernel(const __grid_constant__ AxesParams p, int items, int tokens) {
  // [N * tokens][4][R / 16] (cos, cos, sin, sin) of pairs 2 y and 2 y + 1 of item c at [y][c], so
  // that neighbouring threads read neighbouring words; then (slot, flags) of each token
  extern __shared__ __align__(16) float4 turn[];
  const int half = p.R / 2, per_head = p.R / 16, rotated = (p.Hq + p.Hkv) * per_head;
  const int t0 = blockIdx.x * tokens * N;
  const int mine = tokens > 1 ? threadIdx.x / items : 0;
  const bool there = mine < tokens;
  const int step = tokens > 1 ? items : blockDim.x;
  int i = tokens > 1 ? threadIdx.x - mine * items : threadIdx.x;
  int2* about = reinterpret_cast<int2*>(turn + N * tokens * per_head * 4);

  Item<T> it;
  uint4 x[N][2];
  const bool any = there && i < items;
  const auto load = [&]() {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int t = t0 + mine + n * tokens;
      if (t < p.T) it.load(p, t, x[n]);
    }
  };
  if (any) {
    it.template place<kSide>(p, i);
    load();
  }
  // a block may hold more tokens than threads (tokens of three items or fewer)
  for (int w = threadIdx.x; w < N * tokens && t0 + w < p.T; w += blockDim.x) {
    const Token k = read_token(p, t0 + w);
    report(p, k);
    about[w] = make_int2(k.slot, (k.known ? 1 : 0) | (k.known && k.fits ? 2 : 0));
  }
  for (int n = threadIdx.x; n < N * tokens * half; n += blockDim.x) {
    const int w = n / half, j = n - w * half;
    if (t0 + w >= p.T) break;
    const int r = __ldg(p.pos + (int64_t)p.pair_axis[j] * p.T + t0 + w);
    if (r >= 0 && r < p.P) {
      const int64_t at = (int64_t)r * half + j;
      float* z =
          reinterpret_cast<float*>(turn + (w * 4 + (j & 7) / 2) * per_head + j / 8) + (j & 1);
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
      if (i < rotated && (k.y & 1))
        turn_item<T, kSide>(x[n], turn + w * 4 * per_head + i % per_head, per_head);
      it.store(p, t0 + w, k, x[n]);
    }
    i += step;
    if (tokens > 1 || i >= items) break;
    it.template place<kSide>(p, i);
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
                       : static_cast<const T*>(isv ? p.v : p.k) + (int64_t)t * p.kv_stride +
                             (int64_t)kh * p.D;
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
  const int sms = device_sms();
  if (tokens == 1 && items <= kMaxThreads && p.T >= kStreamFrom * sms &&
      p.R <= kMaxThreads / kPair * 2) {
    // Many tokens of many items stay with the blocks that fit the SMs (80 registers a thread):
    // 32768 tokens of 384 items take 133 us (6182 GB/s, 91 % of measured copy bandwidth), 152 us
    // with a block for four tokens, 272 us with one for each. From three tokens an SM on: 512
    // tokens take 4.9 us, 6.3 us with a block each; 320 tokens 4.9 us and 4.5 us.
    int block = items > p.R ? items : p.R;   // R: kPair * R / 2 gathering threads
    block = (block + 31) / 32 * 32;
    const int per_sm = 65536 / (block * 80) > 1 ? 65536 / (block * 80) : 1;
    const size_t smem = 2 * (sizeof(float4) * kPair * (p.R / 4) + sizeof(int2) * kPair);
    if (p.interleaved)
      append_axes_stream_kernel<T, TT, true><<<per_sm * sms, block, smem, s>>>(p, items);
    else
      append_axes_stream_kernel<T, TT, false><<<per_sm * sms, block, smem, s>>>(p, items);
    return;
  }
  // Tokens of a thread (one, two, four: 56, 64, 80 registers): as few as one wave of blocks takes
  // them all with; else two, so that the last wave is no longer than it has to be, and four where
  // the waves are many. Tokens of 48 items, with 1, 2, 4: 4096 6.9, 5.9, 7.1 us; 8192 11.1, 10.2,
  // 8.8 us; 12000 15.0, 12.1, 14.4 us. Of 80 items, with 2, 4: 12000 17.4, 18.5 us; 65536 83, 74 us.
  // (Blocks that stay took 74 us for 65536 of 48 items, 57 us with four: they need more registers
  // where a thread gathers for several tokens.)
  const auto wave = [&](int n, int regs) {
    return (int64_t)(65536 / (threads * regs)) * n * tokens * sms;
  };
  if (p.T <= wave(1, 56))
    launch_items<T, TT, 1>(p, items, tokens, threads, s);
  else if (p.T > wave(2, 64) && (p.T <= wave(4, 80) || p.T > 3 * wave(4, 80)))
    launch_items<T, TT, 4>(p, items, tokens, threads, s);
  else
    launch_items<T, TT, 2>(p, items, tokens, threads, s);
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
