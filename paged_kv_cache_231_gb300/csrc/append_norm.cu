// K and V of new tokens into the paged cache, queries and keys normed for each head and rotated
// (pkv_paged_append_norm_rotary).
//
// For a head x of D elements: y_i = x_i * w_i / sqrt(sum_j x_j^2 / D + epsilon), then pair j turns
// by the angle of table row pos[axis(j)][token], column j:
//   lead' = lead * cos - trail * sin,   trail' = trail * cos + lead * sin
// in fp32, rounded once. Every element is read once and written once: the operator is bound by
// HBM, 4 * (Hq + 2 Hkv) * D bytes per token.
//
// D / 16 neighbouring lanes hold a head, 16 elements each: a lane has both members of its 8 pairs
// (two 16-byte chunks rotary_dim / 2 apart, or side by side) or two chunks behind rotary_dim, so
// the norm is log2(D / 16) shuffles and the rotation none. Cos and sin of a group of tokens are
// gathered once into shared memory, whatever the axes' order. Few tokens: a block for each group.
// Many: a block stays, and while a group is normed, turned and written, the next one's rows are on
// their way into a ring in shared memory and its table entries into registers, and so are the slots
// and positions of the one behind it. Other head sizes and rotary dimensions take a warp for a
// head, which passes the normed row on through shared memory.
// Measured (32 + 2 x 8 heads of 128): 64 tokens 3.6 us, which is latency; 32768 tokens 140 us with one
// axis and 146 us with three, 5.9 and 5.6 TB/s (87 and 83 % of measured copy bandwidth): barriers and
// the gathering, which an append without norms (134 us) has as well, behind a longer computation.
#include <type_traits>

#include "append_dev.cuh"

namespace pkv {
namespace {

using append::Token;
using append::read_token;
using append::report;
using elem::Num;

constexpr int kMaxThreads = 384;   // two blocks of 85 registers a thread to an SM
constexpr int kFill = 256;   // threads that tokens side by side fill
constexpr int kStages = 2;   // groups of tokens whose rows the ring holds

__device__ __forceinline__ float weight_at(const void* w, bool f32, bool bf16, int i) {
  return f32    ? __ldg(static_cast<const float*>(w) + i)
         : bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i])
                : __half2float(static_cast<const __half*>(w)[i]);
}

// tokens: tokens of a block side by side, N times as many a group; heads: heads of a token that
// this block works on (blockIdx.y: which).
// kRing: the block goes on to further groups, whose rows come through a ring in shared memory; else
// it has one.
template <typename T, typename TT, int D, bool kSide, int N, bool kRing>
__global__ void __launch_bounds__(kMaxThreads, 2)
    append_norm_kernel(const __grid_constant__ NormParams np, int tokens, int heads) {
  constexpr int kLanes = D / 16;
  const AxesParams& p = np.axes;
  // [2][N * tokens][4][R / 16] (cos, cos, sin, sin) of pairs 2 y and 2 y + 1 of item c at [y][c], so
  // that neighbouring lanes read neighbouring words; then (slot, flags) of each token, twice
  // Behind them the ring of rows: each thread copies what it will work on itself, so nothing but
  // its own copies is waited for; [kStages][N][2] 16 bytes of each thread.
  extern __shared__ __align__(16) float4 turn[];
  __shared__ __align__(16) float s_weight[2][D];   // of queries and of keys
  const int half = p.R / 2, per_head = p.R / 16, group = N * tokens;
  const int words = group * per_head * 4;
  int2* about = reinterpret_cast<int2*>(turn + 2 * words);
  uint4* const ring = reinterpret_cast<uint4*>(turn + 2 * words + group) + threadIdx.x;
  const int items = heads * kLanes, w = threadIdx.x / items, i = threadIdx.x - w * items;
  const int groups = (p.T + group - 1) / group;
  const int h = blockIdx.y * heads + i / kLanes, c = i % kLanes;
  const bool mine = w < tokens && h < p.Hq + 2 * p.Hkv;
  const int kind = h < p.Hq ? 0 : h < p.Hq + p.Hkv ? 1 : 2;   // query, key, value
  const bool turns = c < per_head && kind < 2;
  int chunk[2];
  chunk[0] = c >= per_head ? 2 * c : kSide ? 2 * c : c;
  chunk[1] = c >= per_head || kSide ? 2 * c + 1 : c + per_head;
  const int hh = kind == 0 ? h : kind == 1 ? h - p.Hq : h - p.Hq - p.Hkv;
  const T* const src = static_cast<const T*>(kind == 0 ? p.q : kind == 1 ? p.k : p.v) + hh * D;
  T* const dst = static_cast<T*>(kind == 0 ? p.q_out : kind == 1 ? p.kc : p.vc) + hh * D;
  const int64_t in_row = kind == 0 ? p.q_stride : p.kv_stride;
  const int out_row = (kind == 0 ? p.Hq : p.Hkv) * D;
  const void* const weight = kind == 0 ? np.qw : np.kw;
  const bool normed = kind < 2 && weight != nullptr;

  const auto slot_of = [&](int stage, int n, int y) {
    return ring + ((stage * N + n) * 2 + y) * blockDim.x;
  };
  uint4 alone[kRing ? 1 : N][2];
  const auto load = [&](int g, int stage) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int t = g * group + n * tokens + w;
      if (mine && g < groups && t < p.T) {
        const uint4* row = reinterpret_cast<const uint4*>(src + (int64_t)t * in_row);
        if constexpr (kRing) {
          cp_async_16(slot_of(stage, n, 0), row + chunk[0], 16);
          cp_async_16(slot_of(stage, n, 1), row + chunk[1], 16);
        } else {
          alone[n][0] = __ldcs(row + chunk[0]);
          alone[n][1] = __ldcs(row + chunk[1]);
        }
      } else if (!kRing) {
        alone[n][0] = alone[n][1] = make_uint4(0, 0, 0, 0);
      }
    }
    if constexpr (kRing) cp_async_commit();
  };
  // Cos and sin of pair j of token k of a group, one pair to a thread and round. The table rows of
  // a group are asked for a group before its entries are, and these a group before their use.
  const int pairs = group * half, apart = gridDim.x;
  const auto row_of = [&](int g, int k) {   // table row, -1: none
    if (k >= pairs || g >= groups) return -1;
    const int t = g * group + k / half;
    return t < p.T ? __ldg(p.pos + (int64_t)p.pair_axis[k % half] * p.T + t) : -1;
  };
  const auto fetch = [&](int row, int k, float& c, float& s) {
    if (row >= 0 && row < p.P) {
      const int64_t at = (int64_t)row * half + k % half;
      c = Num<TT>::to(__ldg(static_cast<const TT*>(p.cos) + at));
      s = Num<TT>::to(__ldg(static_cast<const TT*>(p.sin) + at));
    }
  };
  const auto put = [&](int buf, int k, float c, float s) {
    const int tok = k / half, j = k % half;
    float* z = reinterpret_cast<float*>(turn + buf * words) +
               4 * ((tok * 4 + (j & 7) / 2) * per_head + j / 8) + (j & 1);
    z[0] = c;
    z[2] = s;
  };
  const auto later = [&](int g, int buf) {   // pairs behind the first round, all at once
    for (int k = threadIdx.x + blockDim.x; k < pairs; k += blockDim.x) {
      float c = 0.f, s = 0.f;
      fetch(row_of(g, k), k, c, s);
      put(buf, k, c, s);
    }
  };
  // slot and flags of this thread's token of a group, asked for a group before they are put down
  const auto token = [&](int g) {
    const int t = g * group + (int)threadIdx.x;
    if ((int)threadIdx.x >= group || g >= groups || t >= p.T) return make_int2(-1, 0);
    const Token tk = read_token(p, t);
    if (blockIdx.y == 0) report(p, tk);
    return make_int2(tk.slot, (tk.known ? 1 : 0) | (tk.known && tk.fits ? 2 : 0));
  };
  const int first = threadIdx.x;
  const bool gathers = first < pairs;

  int g = blockIdx.x;
#pragma unroll
  for (int i = 0; i < (kRing ? kStages - 1 : 1); ++i) load(g + i * apart, i);
  for (int e = threadIdx.x; e < 2 * D; e += blockDim.x) {
    const void* from = e < D ? np.qw : np.kw;
    s_weight[e / D][e % D] = from ? weight_at(from, np.weight_f32, p.bf16, e % D) : 1.f;
  }
  float co = 0.f, si = 0.f;
  fetch(row_of(g, first), first, co, si);
  int row = kRing ? row_of(g + apart, first) : -1;
  int2 tok_about = token(g);
  later(g, 0);
  if (gathers) put(0, first, co, si);
  if (first < group) about[first] = tok_about;
  __syncthreads();
  for (int buf = 0, stage = 0; g < groups; g += apart, buf ^= 1, stage = (stage + 1) % kStages) {
    if constexpr (kRing) {
      cp_async_wait<kStages - 2>();
      load(g + (kStages - 1) * apart, (stage + kStages - 1) % kStages);
      fetch(row, first, co, si);
      row = row_of(g + 2 * apart, first);
      tok_about = token(g + apart);
      later(g + apart, buf ^ 1);
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int tok = n * tokens + w, t = g * group + tok;
      // the shuffles are the whole warp's; rows that are not there are not written
      float v[16], sum = 0.f;
      uint4 x[2];
#pragma unroll
      for (int y = 0; y < 2; ++y)
        if constexpr (kRing)
          x[y] = *slot_of(stage, n, y);
        else
          x[y] = alone[n][y];
      const uint32_t* u = reinterpret_cast<const uint32_t*>(x);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float2 f = Num<T>::to2(u[e]);
        v[2 * e] = f.x;
        v[2 * e + 1] = f.y;
        sum += f.x * f.x;
        sum += f.y * f.y;
      }
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (!mine || t >= p.T) continue;
      const int2 k = about[buf * group + tok];
      if (k.x < 0 || (kind > 0 && !(k.y & 2))) continue;
      if (kind < 2) {
        if (normed) {
          const float by = rsqrtf(sum * (1.f / D) + np.epsilon);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float4 w4 =
                *reinterpret_cast<const float4*>(s_weight[kind] + chunk[e / 2] * 8 + e % 2 * 4);
            v[4 * e] *= by * w4.x;
            v[4 * e + 1] *= by * w4.y;
            v[4 * e + 2] *= by * w4.z;
            v[4 * e + 3] *= by * w4.w;
          }
        }
        if (turns && (k.y & 1)) {
          const float4* cs = turn + buf * words + tok * 4 * per_head + c;
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const float4 a = cs[y * per_head];
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              const int lead = kSide ? 4 * y + 2 * z : 2 * y + z;
              const int trail = kSide ? lead + 1 : lead + 8;
              const float co = z ? a.y : a.x, si = z ? a.w : a.z, l = v[lead], r = v[trail];
              v[lead] = l * co - r * si;
              v[trail] = r * co + l * si;
            }
          }
        }
        uint32_t* q = reinterpret_cast<uint32_t*>(x);
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = Num<T>::from2(v[2 * e], v[2 * e + 1]);
      }
      uint4* row = reinterpret_cast<uint4*>(dst + (int64_t)(kind == 0 ? t : k.x) * out_row);
      row[chunk[0]] = x[0];
      row[chunk[1]] = x[1];
    }
    if (!kRing) break;
    if (gathers) put(buf ^ 1, first, co, si);
    if (first < group) about[(buf ^ 1) * group + first] = tok_about;
    __syncthreads();
  }
}

// Any head size and rotary dimension: a warp for a head of a token.
constexpr int kWarps = 8;
template <typename T, typename TT>
__global__ void __launch_bounds__(32 * kWarps)
    append_norm_heads_kernel(const __grid_constant__ NormParams np) {
  __shared__ float s_row[kWarps][256];
  const AxesParams& p = np.axes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, heads = p.Hq + 2 * p.Hkv;
  for (int64_t unit = (int64_t)blockIdx.x * kWarps + warp; unit < (int64_t)p.T * heads;
       unit += (int64_t)gridDim.x * kWarps) {
    const int t = (int)(unit / heads), h = (int)(unit - (int64_t)t * heads);
    const Token k = read_token(p, t);
    if (k.slot < 0) continue;
    if (h == 0 && lane == 0) report(p, k);
    const int kind = h < p.Hq ? 0 : h < p.Hq + p.Hkv ? 1 : 2;
    if (kind > 0 && !(k.known && k.fits)) continue;
    const int hh = kind == 0 ? h : kind == 1 ? h - p.Hq : h - p.Hq - p.Hkv, half = p.R / 2;
    const T* src = static_cast<const T*>(kind == 0 ? p.q : kind == 1 ? p.k : p.v) +
                   (int64_t)t * (kind == 0 ? p.q_stride : p.kv_stride) + (int64_t)hh * p.D;
    T* dst = kind == 0 ? static_cast<T*>(p.q_out) + ((int64_t)t * p.Hq + hh) * p.D
                       : static_cast<T*>(kind == 1 ? p.kc : p.vc) +
                             ((int64_t)k.slot * p.Hkv + hh) * p.D;
    const bool there = lane * 8 < p.D;
    __align__(16) T x[8];
    float sum = 0.f;
    if (there) {
      *reinterpret_cast<uint4*>(x) = *reinterpret_cast<const uint4*>(src + lane * 8);
  #pragma unroll
      for (int e = 0; e < 8; ++e) sum += Num<T>::to(x[e]) * Num<T>::to(x[e]);
    }
    if (kind < 2) {
      const void* weight = kind == 0 ? np.qw : np.kw;
      sum = warp_sum(sum);
      const float by = weight ? rsqrtf(sum / (float)p.D + np.epsilon) : 1.f;
      float* row = s_row[warp];
      if (there)
  #pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int i = lane * 8 + e;
          row[i] = Num<T>::to(x[e]) * by *
                   (weight ? weight_at(weight, np.weight_f32, p.bf16, i) : 1.f);
        }
      __syncwarp();
      if (there)
  #pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int i = lane * 8 + e;
          float y = row[i];
          if (i < p.R && k.known) {
            const int j = p.interleaved ? i >> 1 : (i < half ? i : i - half);
            const bool lead = p.interleaved ? (i & 1) == 0 : i < half;
            const int other = p.interleaved ? i ^ 1 : (lead ? i + half : i - half);
            const int64_t at = (int64_t)__ldg(p.pos + (int64_t)p.pair_axis[j] * p.T + t) * half + j;
            const float co = Num<TT>::to(static_cast<const TT*>(p.cos)[at]);
            const float si = Num<TT>::to(static_cast<const TT*>(p.sin)[at]);
            y = lead ? y * co - row[other] * si : y * co + row[other] * si;
          }
          x[e] = Num<T>::from(y);
        }
    }
    if (there) *reinterpret_cast<uint4*>(dst + lane * 8) = *reinterpret_cast<const uint4*>(x);
    __syncwarp();   // the row is read before the next one takes its place
  }
}

// Of the largest block: 384 threads of 8 tokens' rows, or 128 tokens (of two heads of 64) with the
// cos and sin of 32 pairs twice.
constexpr int kMostShared = 150 * 1024;

template <typename T, typename TT, int D, bool kSide>
cudaError_t launch_lanes(const NormParams& np, cudaStream_t s) {
  const AxesParams& p = np.axes;
  constexpr int kLanes = D / 16;
  const int all = p.Hq + 2 * p.Hkv;
  const int parts = (all * kLanes + kMaxThreads - 1) / kMaxThreads, heads = (all + parts - 1) / parts;
  const int items = heads * kLanes, tokens = items * 2 <= kFill ? kFill / items : 1;
  const int threads = (tokens * items + 31) / 32 * 32, sms = device_sms();
  const auto shared = [&](int n, bool ring) {   // turned pairs, tokens and rows
    return (size_t)n * tokens * (2 * sizeof(float4) * (p.R / 4) + sizeof(float4)) +
           (ring ? (size_t)threads * kStages * n * 32 : 0);
  };
  const auto run = [&](auto n, auto ring) {
    constexpr int N = decltype(n)::value;
    constexpr bool kRing = decltype(ring)::value;
    static std::atomic<uint64_t> configured{0};
    int dev = -1;
    if (needs_configure(configured, &dev)) {
      const cudaError_t e =
          cudaFuncSetAttribute(append_norm_kernel<T, TT, D, kSide, N, kRing>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, kMostShared);
      if (e != cudaSuccess) return e;
      mark_configured(configured, dev);
    }
    const size_t smem = shared(N, kRing);
    const int group = N * tokens, groups = (p.T + group - 1) / group;
    int most = groups;
    if (kRing) {   // blocks that the SMs take at once, by 80 registers a thread
      const int regs = 65536 / (threads * 80), by_smem = (int)(225 * 1024 / (smem + 1024 + 8 * D));
      most = (regs < by_smem ? regs : by_smem) * sms / parts;
      if (most < 1) most = 1;
    }
    const dim3 grid((unsigned)(groups < most ? groups : most), (unsigned)parts);
    append_norm_kernel<T, TT, D, kSide, N, kRing><<<grid, threads, smem, s>>>(np, tokens, heads);
    return cudaGetLastError();
  };
  // A block for each group of tokens while one wave of blocks takes them all, with as few tokens to
  // a thread as that needs: tokens of 384 items, with one, two, four to a thread and with the ring: 300
  // 4.1, 4.1, 5.0 and 5.7 us, 600 6.6, 5.0, 5.1 and 5.8 us, 1200 10.9, 9.3, 7.8 and 9.2 us. Behind that
  // blocks that stay and have the next rows on their way: 2500 22.7, 22.4, 19.9 and 18.3 us, 32768 258,
  // 245, 192 and 140 us. Where a block holds many tokens side by side it is the gathering that takes
  // the time, and the ring's registers and barriers cost more than they bring: 32768 tokens of 80 items
  // 63.7, 54.6, 42.9 and 41.2 us, of 48 items 51.8, 51.2, 44.3 and 51.9 us.
  const auto wave = [&](int n) { return (int64_t)(65536 / (threads * 80)) * n * tokens * sms / parts; };
  if (p.T <= wave(1)) return run(std::integral_constant<int, 1>(), std::false_type());
  if (p.T <= wave(2)) return run(std::integral_constant<int, 2>(), std::false_type());
  if (p.T <= wave(4) || tokens > 3)
    return run(std::integral_constant<int, 4>(), std::false_type());
  return run(std::integral_constant<int, 4>(), std::true_type());
}

template <typename T, typename TT>
cudaError_t launch_typed(const NormParams& np, cudaStream_t s) {
  const AxesParams& p = np.axes;
  const bool lanes = p.R % 16 == 0 && (p.D == 64 || p.D == 128 || p.D == 256);
  if (!lanes) {
    const int64_t blocks = ((int64_t)p.T * (p.Hq + 2 * p.Hkv) + kWarps - 1) / kWarps;
    const int64_t fit = (int64_t)64 * device_sms();   // 8 waves
    append_norm_heads_kernel<T, TT>
        <<<(unsigned)(blocks < fit ? blocks : fit), 32 * kWarps, 0, s>>>(np);
    return cudaGetLastError();
  }
  if (p.interleaved)
    return p.D == 64    ? launch_lanes<T, TT, 64, true>(np, s)
           : p.D == 128 ? launch_lanes<T, TT, 128, true>(np, s)
                        : launch_lanes<T, TT, 256, true>(np, s);
  return p.D == 64    ? launch_lanes<T, TT, 64, false>(np, s)
         : p.D == 128 ? launch_lanes<T, TT, 128, false>(np, s)
                      : launch_lanes<T, TT, 256, false>(np, s);
}

}  // namespace

cudaError_t launch_append_norm(const NormParams& p, cudaStream_t s) {
  ProfScope ps("append_norm", s);
  if (p.axes.bf16)
    return p.axes.table_f32 ? launch_typed<__nv_bfloat16, float>(p, s)
                            : launch_typed<__nv_bfloat16, __nv_bfloat16>(p, s);
  return p.axes.table_f32 ? launch_typed<__half, float>(p, s) : launch_typed<__half, __half>(p, s);
}

}  // namespace pkv
