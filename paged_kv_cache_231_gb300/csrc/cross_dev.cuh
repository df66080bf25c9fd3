// What the cross-attention kernels share: element types, the plan of a call, joins.
//
// Plan. A "range" is one (sequence, kv head) with all its query rows (few rows: at most 16)
// or one tile of up to 256 query rows of it (many rows); its length is counted in "steps"
// of 16 or 32 keys (few rows) or 128 keys (many rows). The ranges of a call are laid end to end and
// cut into runs of equally many steps, one for each unit of a persistent grid (a warp, or a
// block): every unit does the same amount whatever the lengths are. A range that lies inside
// one run is finished there; of the others each unit keeps an unnormalised (o, m, l) piece in
// fp32, at most two (where its run begins and where it ends), and the join kernel merges the
// pieces in order. The unit in whose run such a range begins writes the record that the join
// reads. Tiles that are many are dealt out whole first (cross_tiles.cu); the rest is cut.
// Lengths live on the device, so every block makes the plan for itself from cu and klen.
//
// Forms. The kernels are written once and compiled for three kinds of calls:
//   kCross   every row of a sequence sees all of its klen keys;
//   kShared  the same for groups of sequences over the keys that these have in common, all of them
//            as tiles; output and lse go to 32-bit arrays in the workspace;
//   kCausal  row i stands at past + i and sees keys j <= past + i with j > past + i - window or
//            j < sinks, or (behind a shared prefix) with j >= start; then the result of the kShared
//            call is joined in where the row is written.
// Keys that no row of a range sees are not among its steps: those behind the sinks and in front of
// the window are passed over, and the others counted on (see Span).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include "device_common.cuh"
#include "internal.h"
#include "step_ops.h"

// The form that a translation unit compiles (see below) and the name of its launchers.
#ifndef PKV_FORM
#define PKV_FORM kCross
#define PKV_LAUNCH(suffix) launch_cross##suffix
#define PKV_CROSS_FORM
#endif

namespace pkv {
namespace cross {

// keys of a step, few rows: 4 KB of keys
__host__ __device__ constexpr int few_keys(int head_size) { return 2048 / head_size; }
constexpr int kTileKeys = 128;     // keys of a step, many rows
constexpr int kEntries = 1024;     // prefix entries of a plan
// A weight is 2^(score - m), where m is the row's maximum less kLift, raised when the maximum
// passes it by kLift + kRaise: the largest is 2^7 to 2^15. Rounded to fp16 for the product with the
// values, weights of 2^-32 of the largest and less are lost, and others err by as much; without the
// lift it was 2^-25, and 60 000 states of such weights 2e-3 of the whole.
constexpr float kLift = 7.f, kRaise = 8.f;
// pieces of a range (bounds the join): 400000 states of one kv head 76 us, with 128 pieces 228 us,
// without a bound 77 us
constexpr int kMaxPieces = 512;
constexpr int kMaxTileUnits = 256; // blocks of the kernel for many rows

enum Form { kCross, kShared, kCausal };

template <typename T>
struct Num;
template <>
struct Num<__half> {
  static constexpr bool kBf16 = false;
  static __device__ __forceinline__ uint32_t pack(float a, float b) { return pack_half2(a, b); }
  static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                             uint32_t b1) {
    mma_16816(d, a, b0, b1);
  }
};
template <>
struct Num<__nv_bfloat16> {
  static constexpr bool kBf16 = true;
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&x);
  }
  static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                             uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, "
        "{%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};

// One sequence as a kernel of one kind sees it; ranges == 0: nothing to do here.
struct Seq {
  int cu0, rows, keys;   // first query row, query rows, keys
  int steps;             // steps of a range (kCausal, many rows: its tiles differ, see tile_span)
  int ranges;
  int at;                // kCausal: position of the first row; kShared: row of the block table
  int lo;                // kCausal: first key that takes part (in a window or not)
};

// The keys that rows at positions first .. last of a sequence go through, in steps of N: counted
// from 0, the v-th is key v below ns (the sinks) and key v + gap from there on. What is cut out is
// whole boxes of `unit` keys (of a TMA copy), so that a step is whole boxes. A row at position t sees
// v <= t - gap with v > t - gap - window or v < sinks. One key at least, so that every row is written.
// (Cut in whole steps, a tile of 64 positions behind a window of 1024 took 10.5 steps on average
// and not 9.3: 206 and 185 us for 8 prompts of up to 2048 tokens.)
struct Span {
  int ns, gap, steps;
  __device__ __forceinline__ int key_at(int v) const { return v < ns ? v : v + gap; }
};
template <int N>
__device__ __forceinline__ Span span_of(const CrossParams& p, const Seq& q, int first, int last,
                                        int unit) {
  Span x;
  x.ns = p.window > 0 ? (p.sinks + unit - 1) & -unit : 0;
  const int end = min(last + 1, q.keys);
  const int from = p.window > 0 ? max(q.lo, first - p.window + 1) : q.lo;
  // where every row stands behind the last key of the table, the sinks are still among the steps
  x.gap = max(min(from & -unit, (end - 1) & -unit) - x.ns, 0);
  x.steps = (end - x.gap + N - 1) / N;
  return x;
}
// of tile t of a sequence
__device__ __forceinline__ Span tile_span(const CrossParams& p, const Seq& q, int t) {
  const int q0 = t * p.tile_pos;
  return span_of<kTileKeys>(p, q, q.at + q0, q.at + min(q0 + p.tile_pos, q.rows) - 1,
                            max(p.box_keys, 1));
}
// first key in a window that some row of the sequence sees
__device__ __forceinline__ int first_seen(const CrossParams& p, const Seq& q) {
  return p.window > 0 ? max(q.lo, q.at - p.window + 1) : q.lo;
}

// kTiles: the kernel for many rows. *flags gets what is wrong with the sequence, *zero is set
// when some of its rows see no key.
template <bool kTiles, Form F>
__device__ __forceinline__ Seq read_seq(const CrossParams& p, int b, int* flags, bool* zero) {
  // The groups' rows and keys (kShared) are written by the plan, behind which this kernel may already
  // have begun: the read-only path is for memory that nobody writes as long as a kernel lasts.
  const auto at = [](const int32_t* x) { return F == kShared ? __ldcg(x) : __ldg(x); };
  Seq s;
  s.cu0 = at(p.cu + b);
  const int hi = at(p.cu + b + 1);
  s.keys = at((F == kCausal ? p.past : p.klen) + b);
  if (F == kCausal) s.lo = p.start ? __ldcg(p.start + b) : 0;
  if (F == kShared) s.at = __ldcg(p.table_row + b);
  s.steps = s.ranges = 0;
  // Of any two numbers, so it may wrap around, and is looked at behind the other checks only.
  // (Formed behind them: 128 tokens over 1500 states 67.0 us, so 66.2 us.)
  s.rows = (int)((uint32_t)hi - (uint32_t)s.cu0);
  if (s.cu0 < 0 || hi < s.cu0 || hi > p.T || s.rows > p.max_q || s.keys < 0 ||
      (F == kCausal && s.keys > p.MB * p.BS)) {
    *flags |= PKV_DEV_BAD_SEQUENCE;
    *zero = true;
    return s;
  }
  if (F == kCausal) {   // both below 2^30
    s.at = s.keys;
    s.keys += s.rows;
  }
  if (s.rows > 0 && s.keys > p.MB * p.BS) {
    *flags |= PKV_DEV_BAD_BLOCK;
    s.keys = p.MB * p.BS;
  }
  if (s.rows > 0 && s.keys == 0) *zero = true;
  if (s.rows == 0 || s.keys == 0 || (s.rows > p.few) != kTiles) return s;
  if (kTiles) {
    const int tiles = (s.rows + p.tile_pos - 1) / p.tile_pos;
    if (F != kCausal) s.steps = (s.keys + kTileKeys - 1) / kTileKeys;
    s.ranges = p.Hkv * tiles;
  } else {
    const int n = few_keys(p.D);
    if (F == kCausal)
      s.steps = (p.D == 64 ? span_of<few_keys(64)>(p, s, s.at, s.at + s.rows - 1, 1)
                           : span_of<few_keys(128)>(p, s, s.at, s.at + s.rows - 1, 1)).steps;
    else
      s.steps = (s.keys + n - 1) / n;
    s.ranges = p.Hkv / p.few_heads;
  }
  return s;
}

// a / b for a >= 0, b > 0; 64 bits only where they are needed (they cost some 400 cycles)
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
  return a / b;
}

// Inclusive sum over the block's NT threads; *total gets the sum of all.
template <int NT>
__device__ __forceinline__ int64_t block_sum(int64_t v, int64_t* total, int64_t* scratch) {
  constexpr int NW = NT / 32;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  if (lane == 31) scratch[w] = v;
  __syncthreads();
  int64_t before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < NW; ++i) {
    const int64_t x = scratch[i];
    if (i < w) before += x;
    all += x;
  }
  *total = all;
  __syncthreads();
  return before + v;
}

// The plan of the kernel for few rows. A unit is p.few_heads neighbouring warps, one kv head
// each: what lies together in a cache row is read at about the same time.
struct Plan {
  int64_t total;   // steps of all ranges
  int64_t W;       // steps of a run
  int group;       // sequences of a prefix entry
  int entries;
  bool zero;       // some row sees no key (or belongs to no sequence)
  bool ordered;    // the cumulative lengths ascend
};

// Block-wide. pref: [kEntries] steps before entry e (shared memory); scratch: [NT / 32 + 2].
template <int NT, Form F>
__device__ Plan make_plan(const CrossParams& p, int units, int64_t* pref, int64_t* scratch,
                          int* flags) {
  Plan pl;
  pl.group = (p.B + kEntries - 1) / kEntries;
  pl.entries = (p.B + pl.group - 1) / pl.group;
  int longest = 0;
  bool zero = false, descends = false;
  int64_t carry = 0;
  for (int e0 = 0; e0 < pl.entries; e0 += NT) {
    const int e = e0 + threadIdx.x;
    int64_t mine = 0;
    if (e < pl.entries) {
      const int b1 = min(p.B, (e + 1) * pl.group);
      for (int b = e * pl.group; b < b1; ++b) {
        const Seq s = read_seq<false, F>(p, b, flags, &zero);
        descends |= __ldg(p.cu + b + 1) < s.cu0;
        mine += (int64_t)s.steps * s.ranges;
        longest = max(longest, s.steps);
      }
    }
    int64_t total;
    const int64_t upto = block_sum<NT>(mine, &total, scratch);
    if (e < pl.entries) pref[e] = carry + upto - mine;
    carry += total;
  }
  pl.total = carry;
  int* word = reinterpret_cast<int*>(scratch + NT / 32);
  if (threadIdx.x == 0) word[0] = word[1] = 0;
  __syncthreads();
  longest = __reduce_max_sync(0xffffffffu, longest);
  if ((threadIdx.x & 31) == 0) atomicMax(word, longest);
  if (descends) word[1] = 1;
  pl.zero = __syncthreads_or(zero) || __ldg(p.cu) != 0 || __ldg(p.cu + p.B) != p.T;
  pl.ordered = word[1] == 0;
  pl.W = quotient(carry + units - 1, units);
  pl.W = max(pl.W, (int64_t)max(1, (word[0] + kMaxPieces - 2) / (kMaxPieces - 1)));
  return pl;
}

struct Cursor {
  int b, r, s;   // sequence, range of it, step of the range
  Seq q;
};

// cursor at step g < total
template <Form F>
__device__ __forceinline__ Cursor locate(const CrossParams& p, const Plan& pl,
                                         const int64_t* pref, int64_t g) {
  int lo = 0, hi = pl.entries - 1, e = 0;
  while (lo <= hi) {
    const int mid = (lo + hi) >> 1;
    if (pref[mid] <= g) {
      e = mid;
      lo = mid + 1;
    } else {
      hi = mid - 1;
    }
  }
  Cursor c;
  int64_t at = g - pref[e];
  int f = 0;
  bool z = false;
  for (c.b = e * pl.group; c.b < p.B; ++c.b) {
    c.q = read_seq<false, F>(p, c.b, &f, &z);
    const int64_t n = (int64_t)c.q.steps * c.q.ranges;
    if (at < n) break;
    at -= n;
  }
  c.r = c.q.steps > 0 ? (int)quotient(at, c.q.steps) : 0;
  c.s = c.q.steps > 0 ? (int)(at - (int64_t)c.r * c.q.steps) : 0;
  return c;
}

// first step of the next range
template <Form F>
__device__ __forceinline__ void next_range(const CrossParams& p, Cursor& c) {
  c.s = 0;
  if (++c.r < c.q.ranges) return;
  c.r = 0;
  int f = 0;
  bool z = false;
  while (++c.b < p.B) {
    c.q = read_seq<false, F>(p, c.b, &f, &z);
    if (c.q.ranges > 0) return;
  }
}

// Record of warp w, which works on head `sub` of unit u: the range of its last step, if that ends
// behind the unit's run. The unit in whose run the range begins joins its pieces, and so do the
// units that hold nothing else: unit number i of them takes the rows i, i + n, ... of n units.
// rec[2w] = {pieces, first piece's slot, first query row, kv head}, rec[2w + 1] = {query rows, i,
// whether the result of shared keys is joined in}
template <Form F>
__device__ __forceinline__ void write_record(const CrossParams& p, const Plan& pl,
                                             const int64_t* pref, int64_t u, int sub, int4* rec) {
  const int64_t g0 = u * pl.W, g1 = min(pl.total, g0 + pl.W);
  int4 a = make_int4(0, 0, 0, 0), b = make_int4(0, 0, 0, 0);
  if (g0 < pl.total) {
    const Cursor c = locate<F>(p, pl, pref, g1 - 1);
    const int64_t start = g1 - 1 - c.s, end = start + c.q.steps;
    if (end > g1) {
      const int64_t own = quotient(start, pl.W);
      a = make_int4((int)(quotient(end - 1, pl.W) - own) + 1, start == own * pl.W ? 0 : 1, c.q.cu0,
                    c.r * p.few_heads + sub);
      b.x = c.q.rows;
      b.y = (int)(u - own);
      if (F == kCausal) b.z = c.q.lo > 0;
    }
  }
  rec[0] = a;
  rec[1] = b;
}

// natural-log lse of a row with maximum m (log2 units) and sum l; empty: -inf
__device__ __forceinline__ float lse_of(float m, float l) {
  return l == 0.f ? -INFINITY : m * kLn2 + logf(l);
}
__device__ __forceinline__ float inverse_of(float l) { return l == 0.f ? 0.f : 1.f / l; }

// What a row is written with: out = o * own + prior * other, lse. Without a prior result other is 0.
struct Weights {
  float own, other, lse;
};
// m, l: maximum (log2 units) and sum of the row; where `joins` (kCausal, a sequence whose first keys
// its group computes) the result of those, out_1 with lse_1, is joined in:
//   M = max(m, lse_1 log2 e), L = l 2^{m - M} + 2^{lse_1 log2 e - M}
template <Form F>
__device__ __forceinline__ Weights weights_of(const CrossParams& p, int64_t row, float m, float l,
                                              bool joins) {
  if constexpr (F == kCausal) {
    if (joins) {
      asm volatile("griddepcontrol.wait;\n" ::: "memory");   // for whoever writes it
      const float before = __ldcg(p.prior_lse + row) * kLog2e, mine = l == 0.f ? -INFINITY : m;
      const float top = fmaxf(mine, before), base = top == -INFINITY ? 0.f : top;
      const float a = ex2(mine - base), b = ex2(before - base), all = l * a + b;
      const float inv = inverse_of(all);
      return {a * inv, b * inv, lse_of(top, all)};
    }
  }
  return {inverse_of(l), 0.f, lse_of(m, l)};
}

}  // namespace cross
}  // namespace pkv
