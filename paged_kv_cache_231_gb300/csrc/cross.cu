// Attention of ragged queries over an encoder's states in a paged cache
// (pkv_cross_attention): out = softmax(scale q k^T) v over the n_b states of the row's
// sequence, lse = ln sum e^{scale q k}. Scores are held in log2 units (scale * log2 e).
//
// This file: the kernel for few query rows (sequences with at most 16 rows of a kv head:
// single tokens, drafts), the join of pieces and the launches. cross_tiles.cu: many rows.
//
// Few rows: bound by HBM, every key and value row is read once, 4 * D bytes a state and kv
// head. Each warp of a persistent grid runs through its steps of 4 KB of keys (16 or 32): rows
// go through the warp's own ring in shared memory by 16-byte asynchronous copies (two steps
// ahead; the block table a third), scores and products on mma.sync m16n8k16, whose 16 rows are
// the sequence's query rows x the heads that share the kv head. That is enough where memory is
// the bound: 64 single tokens over 512 to 8192 states, 8 kv heads of 128: 176 to 180 us, 6470 to
// 6630 GB/s (95 to 98 % of measured copy bandwidth).
// Sequences with more than 16 such rows go to the tiles of 256 rows: 64 x 4000 states, 4 heads of
// 128 a kv head, 1 or 4 tokens each: 161 and 169 us here, 203 us there (5 tokens).
// Few and short sequences take one launch (kSmall): 2 tokens over 400 states 5.2 us.
#include <cmath>

#include "cross_dev.cuh"

namespace pkv {
namespace {

using namespace cross;

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kLeastTile = 2;   // steps of a run of the other kernel, at least

template <int D>
__device__ __forceinline__ int chunk_at(int r, int c) {   // 16-byte chunk c of row r, swizzled
  return (r * (D / 8) + (c ^ (r & 7))) * 8;
}

// Lane r < few_keys(D): element offset of key r of step s of (sequence b, kv head h), -1 past
// the keys or where the block is unmapped.
template <int D>
__device__ __forceinline__ int64_t key_offset(const CrossParams& p, int b, int h, int s, int keys,
                                              int lane, int& flags) {
  constexpr int K = few_keys(D);
  const int j = s * K + lane;
  if (lane >= K || j >= keys) return -1;
  const int col = p.bs_shift >= 0 ? j >> p.bs_shift : j / p.BS;
  const int blk = __ldg(p.table + (int64_t)b * p.MB + col);
  if (blk < 0 || blk >= p.NB) {
    flags |= PKV_DEV_BAD_BLOCK;
    return -1;
  }
  return (((int64_t)blk * p.BS + (j - col * p.BS)) * p.Hkv + h) * p.D;
}

// Copies the key and value rows whose offsets the lanes hold; others are zeroed.
template <typename T, int D>
__device__ __forceinline__ void copy_step(const CrossParams& p, int64_t off, T* sk, T* sv,
                                          int lane) {
  constexpr int CPR = D / 8, RPI = 32 / CPR;
  const int c = lane % CPR;
#pragma unroll
  for (int i = 0; i < few_keys(D) / RPI; ++i) {
    const int r = i * RPI + lane / CPR;
    const long long o = __shfl_sync(0xffffffffu, (long long)off, r);
    const int64_t at = o >= 0 ? o + c * 8 : 0;
    cp_async_16(sk + chunk_at<D>(r, c), static_cast<const T*>(p.kc) + at, o >= 0 ? 16 : 0);
    cp_async_16(sv + chunk_at<D>(r, c), static_cast<const T*>(p.vc) + at, o >= 0 ? 16 : 0);
  }
}

template <typename T, int D>
__device__ __forceinline__ void load_queries(const CrossParams& p, const Cursor& c, int h,
                                             int lane, uint32_t (&qa)[D / 16][4]) {
  const int R = c.q.rows * p.G;
  const T* row[2];
  bool ok[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int r = (lane >> 2) + 8 * x;
    ok[x] = r < R;
    const int pos = ok[x] ? r / p.G : 0, g = ok[x] ? r % p.G : 0;
    row[x] = static_cast<const T*>(p.q) + ((int64_t)(c.q.cu0 + pos) * p.Hq + h * p.G + g) * D;
  }
#pragma unroll
  for (int ks = 0; ks < D / 16; ++ks) {
    const int e = ks * 16 + 2 * (lane & 3);
#pragma unroll
    for (int x = 0; x < 4; ++x)
      qa[ks][x] = ok[x & 1]
                      ? __ldg(reinterpret_cast<const unsigned*>(row[x & 1] + e + (x >> 1) * 8))
                      : 0u;
  }
}

// End of the unit's part of a range: the output if the range lies in the run, else a piece.
template <typename T, int D>
__device__ __forceinline__ void flush(const CrossParams& p, const Cursor& c, int h, int gw,
                                      bool whole, int slot, float (&m)[2], float (&l)[2],
                                      float (&o)[D / 8][4], int lane) {
  const int R = c.q.rows * p.G, t4 = lane & 3;
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
    l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
    const int r = (lane >> 2) + 8 * x;
    if (r >= R) continue;
    if (whole) {
      const float inv = inverse_of(l[x]);
      const int64_t row = (int64_t)(c.q.cu0 + r / p.G) * p.Hq + h * p.G + r % p.G;
      uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<T*>(p.out) + row * D) + t4;
#pragma unroll
      for (int d = 0; d < D / 8; ++d)
        out[d * 4] = Num<T>::pack(o[d][2 * x] * inv, o[d][2 * x + 1] * inv);
      if (p.lse && t4 == 0) p.lse[row] = lse_of(m[x], l[x]);
    } else {
      const int64_t row = (int64_t)(2 * gw + slot) * p.few_rows + r;
#pragma unroll
      for (int d = 0; d < D / 8; ++d)
        *reinterpret_cast<float2*>(p.few_o + row * D + d * 8 + 2 * t4) =
            make_float2(o[d][2 * x], o[d][2 * x + 1]);
      if (t4 == 0) {
        p.few_m[row] = m[x];
        p.few_l[row] = l[x];
      }
    }
  }
}

// Whether row i lies in sequence b and sees a key of it.
__device__ __forceinline__ bool holds_row(const CrossParams& p, int b, int i) {
  int f = 0;
  bool z = false;
  const Seq few = read_seq<false>(p, b, &f, &z), many = read_seq<true>(p, b, &f, &z);
  return few.ranges + many.ranges > 0 && i >= few.cu0 && i < few.cu0 + few.rows;
}

// Rows that no key is seen from, or that no sequence covers: output 0, lse -inf. Where the
// cumulative lengths ascend, only the last sequence that begins at or in front of a row can hold
// it. Where they do not (some sequence is bad), a later or an earlier one can: a row that the search
// does not find held is looked for in all of them.
// ordered: 1 they ascend, 0 they do not, -1 not known; then a warp looks when it has such a row.
template <typename T, int D>
__device__ void zero_rows(const CrossParams& p, int unit, int units, int lane, int ordered) {
  for (int64_t i0 = (int64_t)unit * 32; i0 < p.T; i0 += (int64_t)units * 32) {
    const int i = (int)min(i0 + lane, (int64_t)p.T - 1);
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
    const bool empty = b < 0 || !holds_row(p, b, i);
    uint32_t todo = __ballot_sync(0xffffffffu, empty && i0 + lane < p.T);
    if (todo && ordered < 0) {
      bool descends = false;
      for (int c = lane; c < p.B; c += 32) descends |= __ldg(p.cu + c + 1) < __ldg(p.cu + c);
      ordered = __any_sync(0xffffffffu, descends) ? 0 : 1;
    }
    for (; todo; todo &= todo - 1) {
      const int64_t row = i0 + __ffs(todo) - 1;
      bool held = false;
      for (int b0 = 0; ordered == 0 && !held && b0 < p.B; b0 += 32)
        held = __any_sync(0xffffffffu, b0 + lane < p.B && holds_row(p, b0 + lane, (int)row));
      if (held) continue;
      uint4* out = reinterpret_cast<uint4*>(static_cast<T*>(p.out) + row * p.Hq * D);
      for (int c = lane; c < p.Hq * D / 8; c += 32) out[c] = make_uint4(0, 0, 0, 0);
      if (p.lse)
        for (int h = lane; h < p.Hq; h += 32) p.lse[row * p.Hq + h] = -INFINITY;
    }
  }
}

// ---------------------------------------------------------------------------- join
// Over the pieces of a row: M = max m, out = sum 2^{m - M} o / sum 2^{m - M} l. What it waits for
// is memory, so a warp asks for kAhead pieces of a row at once, whether they weigh anything or
// not; a piece of no weight may hold anything.
constexpr int kJoinWarps = 8;
// pieces of a row that a warp asks for at once (8 lowered the occupancy: 64 tokens 16 us, not 12)
constexpr int kAhead = 4;
// rows of a tile's record that a block takes (records of many pieces: 12 us, with 64 18 us)
constexpr int kJoinRows = 16;

template <int D>
struct Joined {
  static constexpr int V = D / 32;   // columns of a lane
  float acc[V], M = -INFINITY, L = 0.f;
  // pieces from, from + share, ... of `pieces`: rows `apart` one from the other, the first one
  // `late` rows on
  __device__ __forceinline__ void add(const float* po, const float* pm, const float* pl, int row,
                                      int late, int apart, int pieces, int from, int share,
                                      int lane) {
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = 0.f;
    for (int q0 = from; q0 < pieces; q0 += kAhead * share) {
      float m[kAhead], l[kAhead], x[kAhead][V];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int q = min(q0 + k * share, pieces - 1);
        const int at = q * apart + (q == 0 ? late : 0) + row;
        m[k] = __ldcg(pm + at);
        l[k] = q0 + k * share < pieces ? __ldcg(pl + at) : 0.f;
        const float* src = po + (int64_t)at * D + lane * V;
        if constexpr (V == 4) {
          const float4 y = __ldcg(reinterpret_cast<const float4*>(src));
          x[k][0] = y.x;
          x[k][1] = y.y;
          x[k][2] = y.z;
          x[k][3] = y.w;
        } else {
          const float2 y = __ldcg(reinterpret_cast<const float2*>(src));
          x[k][0] = y.x;
          x[k][1] = y.y;
        }
      }
      float top = M;
#pragma unroll
      for (int k = 0; k < kAhead; ++k) top = l[k] == 0.f ? top : fmaxf(top, m[k]);
      const float base = top == -INFINITY ? 0.f : top, old = ex2(M - base);
      M = top;
      L *= old;
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] *= old;
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if (l[k] == 0.f) continue;
        const float w = ex2(m[k] - base);
        L += w * l[k];
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] += w * x[k][v];
      }
    }
  }
  template <typename T>
  __device__ __forceinline__ void write(const CrossParams& p, int64_t row, int lane) const {
    const float inv = inverse_of(L);
    uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<T*>(p.out) + row * D + lane * V);
#pragma unroll
    for (int v = 0; v < V; v += 2) out[v / 2] = Num<T>::pack(acc[v] * inv, acc[v + 1] * inv);
    if (p.lse && lane == 0) p.lse[row] = lse_of(M, L);
  }
};

// ---------------------------------------------------------------------------- few rows
__device__ __forceinline__ void named_barrier() {
  asm volatile("bar.sync 1, %0;\n" ::"n"(kThreads) : "memory");
}

template <int D>
struct Ring {
  static constexpr int kSteps = 3;
  static constexpr size_t kWarpBytes = (size_t)kSteps * few_keys(D) * D * 2 * 2;
  static constexpr size_t kBytes = kWarps * kWarpBytes;
};

// kSmall: a block takes one sequence and kv head, its warps an eighth of the steps each, and joins
// what they have in shared memory (few and short sequences: p.small). Behind these blocks are a few
// that look for rows to be zeroed.
template <typename T, int D, bool kSmall>
__global__ void __launch_bounds__(kThreads, 1) cross_few_kernel(CrossParams p) {
  constexpr int NS = Ring<D>::kSteps, K = few_keys(D);
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int64_t s_pref[kEntries];
  __shared__ int64_t s_scratch[kWarps + 2];
  __shared__ uint32_t s_live[kWarps][NS];
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int flags = 0;
  const int gw = blockIdx.x * kWarps + warp;
  Plan pl{};
  Cursor cc{};   // step computed
  int nst = 0, unit = 0, sub = 0;
  if constexpr (kSmall) {
    const int work = p.B * p.Hkv;
    if ((int)blockIdx.x >= work) {
      zero_rows<T, D>(p, gw - work * kWarps, ((int)gridDim.x - work) * kWarps, lane, -1);
      return;
    }
    bool zero;
    cc.b = blockIdx.x / p.Hkv;
    cc.r = blockIdx.x - cc.b * p.Hkv;
    cc.q = read_seq<false>(p, cc.b, &flags, &zero);
    if (cc.r > 0 || warp > 0) flags = 0;   // every block of the sequence saw them
    const int share = (cc.q.steps + kWarps - 1) / kWarps;
    cc.s = warp * share;
    nst = max(0, min(share, cc.q.steps - cc.s));
  } else {
    pl = make_plan<kThreads>(p, p.few_units / p.few_heads, s_pref, s_scratch, &flags);
    if (blockIdx.x > 0) flags = 0;   // every block saw them
    unit = gw / p.few_heads;
    sub = gw % p.few_heads;
    const int64_t g0 = (int64_t)unit * pl.W;
    nst = g0 < pl.total ? (int)(min(pl.total, g0 + pl.W) - g0) : 0;
    if (nst > 0) cc = locate(p, pl, s_pref, g0);
  }
  if (nst > 0) {
    T* rk = reinterpret_cast<T*>(smem + warp * Ring<D>::kWarpBytes);
    T* rv = rk + NS * K * D;
    Cursor pc = cc;                                  // next step to copy
    uint32_t* live = s_live[warp];                   // keys of a step that take part
    int64_t ahead = key_offset<D>(p, pc.b, pc.r * p.few_heads + sub, pc.s, pc.q.keys, lane, flags);
    const auto issue = [&](int k, int buf) {
      if (k < nst) {
        copy_step<T, D>(p, ahead, rk + buf * K * D, rv + buf * K * D, lane);
        if (k + 1 < nst) {
          if (++pc.s == pc.q.steps) next_range(p, pc);
        }
      }
      const uint32_t w = __ballot_sync(0xffffffffu, ahead >= 0);
      if (lane == 0) live[buf] = w;
      if (k + 1 < nst)
        ahead = key_offset<D>(p, pc.b, pc.r * p.few_heads + sub, pc.s, pc.q.keys, lane, flags);
      cp_async_commit();
    };
    // one copy of the step's code: unrolled over the ring it did not fit the instruction cache
#pragma unroll 1
    for (int k = 0; k < NS - 1; ++k) issue(k, k);
    uint32_t qa[D / 16][4];
    load_queries<T, D>(p, cc, cc.r * p.few_heads + sub, lane, qa);
    // while the first steps are on their way (in front of them it took 1 us of 64 tokens' 178 us)
    if (!kSmall && lane == 0) write_record(p, pl, s_pref, unit, sub, p.few_rec + 2 * gw);
    __syncwarp();
    const int t4 = lane & 3;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, o[D / 8][4];
#pragma unroll
    for (int d = 0; d < D / 8; ++d) o[d][0] = o[d][1] = o[d][2] = o[d][3] = 0.f;
    bool from_start = cc.s == 0, first = true;

    int in = 0, out = NS - 1;   // ring slots: the step computed, the step copied
#pragma unroll 1
    for (int k = 0; k < nst; ++k) {
      cp_async_wait<NS - 2>();
      __syncwarp();
      issue(k + NS - 1, out);
      const T* sk = rk + in * K * D;
      const T* sv = rv + in * K * D;
      float s[K / 8][4];   // scores of rows lane / 4 and lane / 4 + 8
#pragma unroll
      for (int n = 0; n < K / 8; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
      {
        const int key = (lane & 7) + ((lane >> 4) << 3), half = (lane >> 3) & 1;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
          for (int n = 0; n < K / 16; ++n) {
            uint32_t b0, b1, b2, b3;
            ldsm_x4(b0, b1, b2, b3, sk + chunk_at<D>(n * 16 + key, 2 * ks + half));
            Num<T>::mma(s[2 * n], qa[ks], b0, b1);
            Num<T>::mma(s[2 * n + 1], qa[ks], b2, b3);
          }
      }
      const uint32_t w = live[in];
      const bool all = w == (K == 32 ? 0xffffffffu : 0xffffu);
#pragma unroll
      for (int n = 0; n < K / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[n][e] *= p.scale_log2;
          if (!all && !((w >> (n * 8 + 2 * t4 + (e & 1))) & 1u)) s[n][e] = -INFINITY;
        }
      // online softmax; m is raised when a score exceeds the maximum that it stands for by kRaise
      float top[2];
      bool raise = false;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        top[x] = fmaxf(s[0][2 * x], s[0][2 * x + 1]);
#pragma unroll
        for (int n = 1; n < K / 8; ++n) top[x] = fmaxf(top[x], fmaxf(s[n][2 * x], s[n][2 * x + 1]));
        raise =
            raise || (m[x] == -INFINITY ? top[x] != -INFINITY : top[x] > m[x] + (kLift + kRaise));
      }
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], 1));
          top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], 2));
          const float mn = fmaxf(m[x], top[x] - kLift);
          const float alpha = ex2(m[x] - (mn == -INFINITY ? 0.f : mn));
          m[x] = mn;
          l[x] *= alpha;
#pragma unroll
          for (int d = 0; d < D / 8; ++d) {
            o[d][2 * x] *= alpha;
            o[d][2 * x + 1] *= alpha;
          }
        }
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float base = m[x] == -INFINITY ? 0.f : m[x];   // scores of -inf weigh nothing
#pragma unroll
        for (int n = 0; n < K / 8; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            s[n][2 * x + e] = ex2(s[n][2 * x + e] - base);
            l[x] += s[n][2 * x + e];
          }
      }
      // the weights, rounded once to T, times the value rows (l keeps them unrounded)
      {
        const int key = (lane & 7) + (((lane >> 3) & 1) << 3), half = lane >> 4;
#pragma unroll
        for (int n = 0; n < K / 16; ++n) {
          const uint32_t pa[4] = {
              Num<T>::pack(s[2 * n][0], s[2 * n][1]), Num<T>::pack(s[2 * n][2], s[2 * n][3]),
              Num<T>::pack(s[2 * n + 1][0], s[2 * n + 1][1]),
              Num<T>::pack(s[2 * n + 1][2], s[2 * n + 1][3])};
#pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            uint32_t b0, b1, b2, b3;
            ldsm_x4_t(b0, b1, b2, b3, sv + chunk_at<D>(n * 16 + key, 2 * j + half));
            Num<T>::mma(o[2 * j], pa, b0, b1);
            Num<T>::mma(o[2 * j + 1], pa, b2, b3);
          }
        }
      }
      const bool last = cc.s == cc.q.steps - 1;
      if (!kSmall && (last || k == nst - 1)) {
        flush<T, D>(p, cc, cc.r * p.few_heads + sub, gw, from_start && last, first ? 0 : 1, m, l, o,
                    lane);
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;
#pragma unroll
        for (int d = 0; d < D / 8; ++d) o[d][0] = o[d][1] = o[d][2] = o[d][3] = 0.f;
        first = false;
        from_start = true;
      }
      if (k < nst - 1) {
        if (last) {
          next_range(p, cc);
          load_queries<T, D>(p, cc, cc.r * p.few_heads + sub, lane, qa);
        } else {
          ++cc.s;
        }
      }
      in = in + 1 == NS ? 0 : in + 1;
      out = out + 1 == NS ? 0 : out + 1;
    }
    cp_async_wait<0>();
    if constexpr (kSmall) {
      named_barrier();   // the pieces take the rings' place
      CrossParams here = p;
      here.few_o = reinterpret_cast<float*>(smem);
      here.few_m = here.few_o + 2 * kWarps * 16 * D;
      here.few_l = here.few_m + 2 * kWarps * 16;
      here.few_rows = 16;
      flush<T, D>(here, cc, cc.r, warp, false, 0, m, l, o, lane);
    }
  } else if constexpr (kSmall) {
    named_barrier();
    float* const l = reinterpret_cast<float*>(smem) + 2 * kWarps * 16 * (D + 1);
    if (lane < 16) l[2 * warp * 16 + lane] = 0.f;
  } else if (lane == 0) {
    p.few_rec[2 * gw] = make_int4(0, 0, 0, 0);   // nothing to join
  }
  if constexpr (kSmall) {
    __syncthreads();
    const float* const po = reinterpret_cast<const float*>(smem);
    const float *pm = po + 2 * kWarps * 16 * D, *pl_ = pm + 2 * kWarps * 16;
    const int rows = cc.q.ranges > 0 ? cc.q.rows * p.G : 0;
    for (int r = warp; r < rows; r += kWarps) {
      Joined<D> j;
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w)
        top = pl_[2 * w * 16 + r] == 0.f ? top : fmaxf(top, pm[2 * w * 16 + r]);
      const float base = top == -INFINITY ? 0.f : top;
      j.M = top;
#pragma unroll
      for (int v = 0; v < Joined<D>::V; ++v) j.acc[v] = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const int at = 2 * w * 16 + r;
        if (pl_[at] == 0.f) continue;
        const float by = ex2(pm[at] - base);
        j.L += by * pl_[at];
#pragma unroll
        for (int v = 0; v < Joined<D>::V; ++v)
          j.acc[v] += by * po[at * D + lane * Joined<D>::V + v];
      }
      j.template write<T>(p, (int64_t)(cc.q.cu0 + r / p.G) * p.Hq + cc.r * p.G + r % p.G, lane);
    }
  } else if (pl.zero) {
    zero_rows<T, D>(p, gw, p.few_units, lane, pl.ordered ? 1 : 0);
  }
  if (flags) flag_status(p.status, flags);
  // the join behind this kernel waits for it alone: it must not end before the one in front
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
}

// Blocks 0 .. : kJoinRows rows of a tile's record each (256 / kJoinRows blocks a record). Behind
// them a block for the record of each warp of the kernel for few rows: 8 warps share the rows that
// fall to it, several warps a row when there are fewer.
template <typename T, int D>
__global__ void __launch_bounds__(32 * kJoinWarps) cross_join_kernel(CrossParams p) {
  constexpr int V = D / 32, kBlocks = 256 / kJoinRows;
  __shared__ float s_o[kJoinWarps][D];
  __shared__ float s_m[kJoinWarps], s_l[kJoinWarps];
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tile_blocks = p.tile_units * kBlocks;
  const bool tile = (int)blockIdx.x < tile_blocks;
  const int unit = tile ? blockIdx.x / kBlocks : blockIdx.x - tile_blocks;
  const int4* rec = (tile ? p.tile_rec : p.few_rec) + 2 * unit;
  const int4 a = __ldcg(rec);
  const int2 about = __ldcg(reinterpret_cast<const int2*>(rec + 1));
  const int tokens = about.x;
  if (a.x <= 0) return;
  const unsigned over_g = 65536u / p.G + 1;          // x / G = x * over_g >> 16 for x < 256
  if (tile) {
    const int64_t first = (int64_t)unit * 512;
    const int PT = p.tile_pos / 2, row0 = blockIdx.x % kBlocks * kJoinRows;
    for (int i = warp; i < kJoinRows; i += kJoinWarps) {
      const int row = row0 + i, x = row & 127, by_g = (int)(x * over_g >> 16);
      const int pos = (row >> 7) * PT + by_g;
      if (x >= PT * p.G || pos >= tokens) continue;
      Joined<D> j;
      j.add(p.tile_o + first * D, p.tile_m + first, p.tile_l + first, row, a.y * 256, 512, a.x, 0,
            1, lane);
      j.template write<T>(p, (int64_t)(a.z + pos) * p.Hq + a.w * p.G + x - by_g * p.G, lane);
    }
    return;
  }
  // the rows nth, nth + helpers, ... of the range that begins nth units before: as many helpers as
  // there are loads for (a block has kJoinWarps * kAhead under way)
  const int nth = about.y, all = tokens * p.G;
  const int helpers = min(a.x - 1, (all * a.x - 1) / (kJoinWarps * kAhead) + 1);
  if (nth >= helpers) return;
  const int64_t first = (int64_t)2 * (unit - nth * p.few_heads) * p.few_rows;
  const int rows = (all - nth + helpers - 1) / helpers;   // at most 0: none
  int share = 1;                                     // warps of a row
  while (share * kAhead < a.x && share < kJoinWarps && rows * share * 2 <= kJoinWarps) share *= 2;
  for (int r0 = 0; r0 < rows; r0 += kJoinWarps / share) {
    const int i = r0 + warp / share, part = warp % share, r = nth + i * helpers;
    const bool live = i < rows;
    Joined<D> j;
    j.add(p.few_o + first * D, p.few_m + first, p.few_l + first, live ? r : 0, a.y * p.few_rows,
          2 * p.few_rows * p.few_heads, live ? a.x : 0, part, share, lane);
    if (share > 1) {
#pragma unroll
      for (int v = 0; v < V; ++v) s_o[warp][lane * V + v] = j.acc[v];
      if (lane == 0) {
        s_m[warp] = j.M;
        s_l[warp] = j.L;
      }
      __syncthreads();
      if (part == 0 && live) {
        float top = j.M;
        for (int k = 1; k < share; ++k)
          top = fmaxf(top, s_l[warp + k] == 0.f ? -INFINITY : s_m[warp + k]);
        const float base = top == -INFINITY ? 0.f : top;
        float w = j.L == 0.f ? 0.f : ex2(j.M - base);
        j.L *= w;
#pragma unroll
        for (int v = 0; v < V; ++v) j.acc[v] *= w;
        for (int k = 1; k < share; ++k) {
          if (s_l[warp + k] == 0.f) continue;
          w = ex2(s_m[warp + k] - base);
          j.L += w * s_l[warp + k];
#pragma unroll
          for (int v = 0; v < V; ++v) j.acc[v] += w * s_o[warp + k][lane * V + v];
        }
        j.M = top;
      }
      __syncthreads();
    }
    const int by_g = (int)(r * over_g >> 16);
    if (live && part == 0)
      j.template write<T>(p, (int64_t)(a.z + by_g) * p.Hq + a.w * p.G + r - by_g * p.G, lane);
  }
}

template <typename T, int D>
cudaError_t launch_typed(const CrossParams& p, cudaStream_t s) {
  static std::atomic<uint64_t> configured{0};
  int dev = -1;
  if (needs_configure(configured, &dev)) {
    cudaError_t e = cudaFuncSetAttribute(cross_few_kernel<T, D, false>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)Ring<D>::kBytes);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(cross_few_kernel<T, D, true>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Ring<D>::kBytes);
    if (e != cudaSuccess) return e;
    mark_configured(configured, dev);
  }
  if (p.small) {
    ProfScope ps("cross_decode", s);
    const unsigned zero = (unsigned)((p.T + kThreads - 1) / kThreads);
    cross_few_kernel<T, D, true>
        <<<(unsigned)(p.B * p.Hkv) + zero, kThreads, Ring<D>::kBytes, s>>>(p);
    return cudaGetLastError();
  }
  cudaLaunchConfig_t cfg = {};
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  // The tiles first: the other kernel's blocks then fill the SMs as theirs end (a call without few
  // rows spends 7 us on them otherwise). They read inputs and write rows of their own.
  if (p.tile_units > 0) {
    const cudaError_t e = launch_cross_tiles(p, s);
    if (e != cudaSuccess) return e;
    cfg.numAttrs = 1;
  }
  {
    ProfScope ps("cross_decode", s);
    cfg.gridDim = dim3((unsigned)(p.few_units / kWarps));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Ring<D>::kBytes;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, cross_few_kernel<T, D, false>, p);
    if (e != cudaSuccess) return e;
  }
  ProfScope ps("cross_combine", s);
  cfg.gridDim = dim3((unsigned)(p.few_units + 256 / kJoinRows * p.tile_units));
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cross_join_kernel<T, D>, p);
}

}  // namespace

size_t cross_layout(CrossParams* p, char* base) {
  const int sms = device_sms();
  p->few = 16 / p->G;
  p->tile_pos = 2 * (128 / p->G);
  // no more units than the longest possible work has runs of the least length (in floating point:
  // the products may pass 64 bits)
  const double keys = (double)p->MB * p->BS, seqs = p->T < p->B ? p->T : p->B;
  const double runs = seqs * p->Hkv * (keys / few_keys(p->D) + 1);
  const int ctas = runs >= (double)sms * kWarps ? sms : (int)(runs / kWarps) + 1;
  p->few_units = ctas * kWarps;
  p->few_heads = kWarps;
  while (p->Hkv % p->few_heads != 0) p->few_heads /= 2;
  p->few_rows = (p->max_q < p->few ? p->max_q : p->few) * p->G;
  p->tile_units = 0;
  if (p->max_q > p->few) {
    const double tiles = (double)p->T / p->tile_pos + seqs;
    const double pieces = tiles * p->Hkv * (keys / kTileKeys + 1) / kLeastTile;
    const int most = sms < kMaxTileUnits ? sms : kMaxTileUnits;
    p->tile_units = pieces >= (double)most ? most : (int)pieces + 1;
  }
  p->box_keys = 0;
  if (p->BS % 8 == 0 && p->NB * p->BS <= INT32_MAX) {
    p->box_keys = 8;
    while (p->box_keys < 128 && p->BS % (2 * p->box_keys) == 0) p->box_keys *= 2;
  }
  size_t off = 0;
  const auto take = [&](size_t bytes) {
    char* at = base ? base + off : nullptr;
    off += (bytes + 255) / 256 * 256;
    return at;
  };
  // A block for each sequence and kv head (one launch, no plan) or an even share for every warp and
  // the join, in units of a step of 0.85 us: steps of a warp and 3.5 for every further wave, or 5
  // for plan and join and the even share. 2 tokens over 400 states, 2 heads of 64: 5.2 and 8.9 us;
  // 16 x 500, 8 kv heads of 64: 6.1 and 12.1 us; 19 x 1000, 8 of 128: 16.0 and 23.9 us; 1 x 2000,
  // 2 of 64: 11.8 and 9.9 us; 64 x 250, 8 of 64: 15.3 and 13.9 us.
  const double ranges = (double)p->B * p->Hkv, waves = std::ceil(ranges / sms);
  const double steps = std::ceil(std::ceil(keys / few_keys(p->D)) / kWarps);
  const double even = ranges * steps / sms;
  p->small = p->max_q <= p->few && ranges <= 4.0 * sms &&
             waves * steps + 3.5 * (waves - 1) <= 5 + (even > 1 ? even : 1);
  if (p->small) {
    p->few_heads = 1;
    return 0;
  }
  const size_t fu = (size_t)p->few_units, tu = (size_t)p->tile_units;
  p->few_rec = reinterpret_cast<int4*>(take(fu * 32));
  p->few_o = reinterpret_cast<float*>(take(2 * fu * p->few_rows * p->D * 4));
  p->few_m = reinterpret_cast<float*>(take(2 * fu * p->few_rows * 4));
  p->few_l = reinterpret_cast<float*>(take(2 * fu * p->few_rows * 4));
  p->tile_rec = reinterpret_cast<int4*>(take(tu * 32));
  p->tile_o = reinterpret_cast<float*>(take(2 * tu * 256 * p->D * 4));
  p->tile_m = reinterpret_cast<float*>(take(2 * tu * 256 * 4));
  p->tile_l = reinterpret_cast<float*>(take(2 * tu * 256 * 4));
  return off;
}

cudaError_t launch_cross(const CrossParams& p, cudaStream_t s) {
  if (p.bf16)
    return p.D == 64 ? launch_typed<__nv_bfloat16, 64>(p, s)
                     : launch_typed<__nv_bfloat16, 128>(p, s);
  return p.D == 64 ? launch_typed<__half, 64>(p, s) : launch_typed<__half, 128>(p, s);
}

}  // namespace pkv
