// Cross attention, sequences with many query rows: tiles on the 5th-generation tensor core.
//
// A range is a tile of 256 rows = two halves of 128 rows = (128 / G) query positions x G
// heads of one kv head each, against 128 keys a step. Per step the tensor core does
// S = Q K^T and O += P V for both halves (4 * 128 * 128 * D multiply-adds); the halves take
// turns, so one half's softmax runs while the other half's products do:
//   warps 0-3, 4-7  softmax of half 0, 1: a thread owns a row (one TMEM lane). It reads its 128
//                   scores and their maximum (TMEM loads reduce on the way), raises its running
//                   maximum only when they exceed it by 2^8 (then O and l are rescaled), writes
//                   the weights, rounded once to T, over the scores in TMEM, and at the end
//                   writes its output row, or its piece.
//   warps 8, 10     one elected lane each issues the tcgen05.mma of half 0, 1 in the order
//                   S(0) PV(0) S(1) PV(1) ...: products of one issuing thread run in order, so S
//                   may overwrite the weights that the PV before it reads, and a full S tells
//                   that the O of that half is complete.
//                   The whole warp runs the loop and a lane is elected for the instructions: from
//                   a lane that runs alone a tcgen05.mma took 85 to 110 cycles, so 56 to 71.
//   warps 9, 11     load by TMA into 128-byte-swizzled shared memory: Q of the halves, and one
//                   ring of K and V tiles in the order of their use (K0 V0 K1 V1 ...). A box is
//                   up to 128 keys of one cache block; a tile lies in groups of 8 keys, the
//                   64-column halves of a group one after the other, so one copy brings whole
//                   rows. Value rows past the sequence's keys or in
//                   unmapped blocks are zero-filled (a weight of zero times what stands there
//                   must be zero); block sizes that are no multiple of 8 go row by row.
// A tile of at most 128 rows is worked on by both halves: half 0 takes the even steps, half 1 the
// odd ones, and half 0 joins the two (m, l, O) at the end.
// TMEM columns: S_0 0..127 (weights over 0..63), S_1 128..255, O_0 256.., O_1 384...
// Measured: 16 sequences of up to 2048 queries over up to 4096 states, 32 heads of 128 on 8 kv
// heads: 460 us for 0.571 TFLOP, 1240 TFLOP/s (64 % of the measured dense rate; the tensor pipe is
// active 56 % of the time): the two halves' softmaxes, each a chain of TMEM loads, exponentials and
// TMEM stores, and the hand-offs between them and the products set the pace. Few rows and long
// sequences (100 queries, 20000 to 60000 states, 16 heads of 64): 80 us, 4.7 TB/s.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <limits.h>

#include "cross_dev.cuh"
#include "tcgen05.cuh"

namespace pkv {
namespace {

using namespace cross;

constexpr int kSoftmaxWarps = 8;
constexpr int kThreads = 32 * (kSoftmaxWarps + 4);
constexpr int kLeast = 2;              // steps of a run, at least (2 x 100 queries, 200 keys:
                                       // 18.5 us, with 4 20.3 us, with 8 22.3 us)
constexpr int kMasks = 8;              // steps whose masks are held (a ring)
constexpr uint32_t kTries = 1u << 22;  // default bound of a wait (polls)
// registers a thread: launch, softmax warps, the other four; the first take what the last give
constexpr int kLaunchRegs = 168, kSoftmaxRegs = 208, kOtherRegs = 88;
static_assert(32 * (kSoftmaxWarps * kSoftmaxRegs + 4 * kOtherRegs) <= kThreads * kLaunchRegs,
              "register split");

// What a block does: `whole` tiles, the first at `first`, every further one `units` tiles on;
// then `steps` steps from `at`.
struct Run {
  Cursor first, at;
  uint32_t tmem;
  int whole;
  int64_t steps;
};
static_assert(sizeof(Run) <= 96, "run area");

template <int D>
struct Lay {   // byte offsets from a 1024-byte-aligned base
  static constexpr int kStages = D == 128 ? 5 : 12;   // at most 12
  static constexpr bool kScarce = D == 128;             // two steps take nearly all of them
  static constexpr uint32_t kTile = 128u * D * 2;       // 128 rows of Q, K or V
  static constexpr uint32_t kSub = 128u * 128;          // Q: 64 columns
  static constexpr uint32_t kGroup = 8u * D * 2;        // K, V: 8 keys, [D / 64][8][64]
  static constexpr uint32_t kQ = 0;
  static constexpr uint32_t kRing = 2 * kTile;
  static constexpr uint32_t kBars = kRing + kStages * kTile;
  static constexpr uint32_t kSeen = kBars + 384;        // [kMasks] keys of a step that take part
  static constexpr uint32_t kRun = kSeen + 16 * kMasks;  // Run
  static constexpr uint32_t kPairMl = kRun + 96;        // [128] (m, l) of half 1
  static constexpr uint32_t kEnd = kPairMl + 1024;
  static constexpr size_t kBytes = kEnd + 1024;
};
static_assert(Lay<128>::kBytes <= 232448, "shared memory over the limit");
static_assert((3 * kEntries + kThreads + 48) * 8 <= Lay<64>::kStages * Lay<64>::kTile &&
                  (3 * kEntries + kThreads + 48) * 8 <= Lay<128>::kStages * Lay<128>::kTile,
              "plan fits the ring");

// mbarriers
enum {
  kFull = 0,     // + stage: K or V tile landed
  kEmpty = 12,   // + stage: the products that read it completed (2: one for each half)
  kQFull = 24,   // + half
  kQEmpty = 26,  // + half: every S of the range completed
  kSFull = 28,   // + half: S in TMEM (and the O before it complete)
  kPFull = 30,   // + half: the 4 warps wrote their weights of the first 64 keys
  kPRest = 32,   // + half: and of the others
  kOFull = 34,   // + half: the last PV of the range completed
  kTurn = 36,    // + half: the other half issued its products
  kDrain = 38,   // + half: products in flight when a wait gave up
  kPair = 40,    // half 1's (m, l, O) of a shared part are there
  kPairRead = 41,   // half 0 has read them
  kBarriers = 42
};
constexpr uint32_t kAbortWord = kBarriers * 8;      // behind the barriers
constexpr uint32_t kRoomWord = kAbortWord + 4;      // [2] tiles that a loader found room for
static_assert(kRoomWord + 8 <= 384, "barrier area");

struct Maps {
  CUtensorMap q, k, v;
};

struct Wait {   // bounded waits that give up together
  uint64_t* bars;
  volatile int* abort;
  uint32_t tries;
  __device__ __forceinline__ bool operator()(int bar, uint32_t parity) const {
    const uint32_t addr = smem_u32(bars + bar);
    for (uint32_t i = 0; i < tries; ++i) {
      uint32_t done;
      asm volatile(
          "{\n"
          ".reg .pred p;\n"
          "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
          "selp.u32 %0, 1, 0, p;\n"
          "}\n"
          : "=r"(done)
          : "r"(addr), "r"(parity)
          : "memory");
      if (done) return true;
      if ((i & 255u) == 255u && *abort) return false;
    }
    *abort = 1;
    return false;
  }
  // the same for a whole warp (every lane asks: with one lane alone and a vote behind it the
  // kernel took a fifth longer)
  __device__ __forceinline__ bool warp(int bar, uint32_t parity) const {
    return __all_sync(0xffffffffu, (*this)(bar, parity)) != 0;
  }
};

__device__ __forceinline__ void arrive(uint64_t* bar, uint32_t count = 1) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;\n" ::"r"(smem_u32(bar)), "r"(count)
               : "memory");
}

// a place in a ring of N stages and the parity of its round
template <int N>
struct Place {
  int stage = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void step(int n) {
    stage += n;
    if (stage >= N) {   // once for the steps of a loop
      if (n > N) {
        phase ^= (uint32_t)(stage / N) & 1u;
        stage %= N;
      } else {
        phase ^= 1u;
        stage -= N;
      }
    }
  }
};
// D (+)= A B with A in TMEM
__device__ __forceinline__ void mma_tmem_a(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n"
      ".reg .pred p;\n"
      "setp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n"
      "}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// true in one lane of a converged warp, always the same one
__device__ __forceinline__ bool elect() {
  uint32_t yes;
  asm volatile(
      "{\n"
      ".reg .pred p;\n"
      "elect.sync _|p, 0xffffffff;\n"
      "selp.u32 %0, 1, 0, p;\n"
      "}\n"
      : "=r"(yes));
  return yes != 0;
}

// 16 consecutive fp32 columns of this thread's TMEM lane
__device__ __forceinline__ void tmem_ld16(uint32_t at, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(at));
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st16(uint32_t at, const float (&v)[16]) {
  uint32_t r[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(v[i]);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// 32 consecutive fp32 columns of this thread's TMEM lane and the largest of them (NaN passed over)
__device__ __forceinline__ void tmem_ld32_max(uint32_t at, float (&v)[32], float& top) {
  uint32_t r[32], m;
  asm volatile(
      "tcgen05.ld.red.sync.aligned.32x32b.x32.max.f32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, %32, [%33];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(m)
      : "r"(at));
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
  top = __uint_as_float(m);
}

// two floats in a register pair, and arithmetic on both at once (each rounded as alone)
__device__ __forceinline__ uint64_t pair_of(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float low_of(uint64_t x) { return __uint_as_float((uint32_t)x); }
__device__ __forceinline__ float high_of(uint64_t x) {
  return __uint_as_float((uint32_t)(x >> 32));
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add_pair(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// This unit's part of a range: the tile under the cursor, steps [c.s, c.s + n).
struct Part {
  int b, h, row0, pos, n, halves;   // first query row of the tile, its positions, steps, halves
  bool whole, shared;               // shared: one half of rows, both halves at work on it
  // half h works on steps first(h) + stride() * i, i < count(h)
  __device__ __forceinline__ bool active(int half) const { return shared || half < halves; }
  __device__ __forceinline__ int first(int half) const { return shared ? half : 0; }
  __device__ __forceinline__ int stride() const { return shared ? 2 : 1; }
  __device__ __forceinline__ int count(int half) const { return shared ? (n + 1 - half) / 2 : n; }
};
__device__ __forceinline__ Part part_of(const CrossParams& p, const Cursor& c, int64_t left) {
  Part t;
  const int tiles = c.q.ranges / p.Hkv, q0 = (c.r % tiles) * p.tile_pos;
  t.b = c.b;
  t.h = c.r / tiles;
  t.row0 = c.q.cu0 + q0;
  t.pos = min(p.tile_pos, c.q.rows - q0);
  t.n = (int)min((int64_t)(c.q.steps - c.s), left);
  t.halves = t.pos > p.tile_pos / 2 ? 2 : 1;
  t.whole = c.s == 0 && t.n == c.q.steps;
  t.shared = t.halves == 1 && t.n > 1;
  return t;
}

// n ranges on from the start of a range; the whole warp (32 sequences at a time)
__device__ __forceinline__ void skip_ranges(const CrossParams& p, Cursor& c, int n) {
  const int lane = threadIdx.x & 31;
  c.s = 0;
  c.r += n;
  while (c.r >= c.q.ranges) {
    int left = c.r - c.q.ranges, f = 0;
    bool z = false;
    const int b0 = c.b + 1;
    Seq q{};
    if (b0 + lane < p.B) q = read_seq<true>(p, b0 + lane, &f, &z);
    int upto = q.ranges;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, upto > left);
    const int at = past ? __ffs(past) - 1 : 31;
    c.r = left - (__shfl_sync(0xffffffffu, upto, at) - __shfl_sync(0xffffffffu, q.ranges, at));
    c.q.cu0 = __shfl_sync(0xffffffffu, q.cu0, at);
    c.q.rows = __shfl_sync(0xffffffffu, q.rows, at);
    c.q.keys = __shfl_sync(0xffffffffu, q.keys, at);
    c.q.steps = __shfl_sync(0xffffffffu, q.steps, at);
    c.q.ranges = __shfl_sync(0xffffffffu, q.ranges, at);
    c.b = b0 + at;
    if (c.b >= p.B) return;   // never: the tiles asked for exist
  }
}

// Walks the parts of a run; every role walks for itself. f gets the part, its cursor and its
// number among the cut parts (-1: a whole tile).
template <typename F>
__device__ __forceinline__ void each_part(const CrossParams& p, const Run& run, F f) {
  Cursor c = run.first;
  for (int i = run.whole; i > 0; --i) {
    if (!f(part_of(p, c, c.q.steps), c, -1)) return;
    if (i > 1) skip_ranges(p, c, p.tile_units);
  }
  c = run.at;
  int64_t steps = run.steps;
  for (int i = 0; steps > 0; ++i) {
    const Part t = part_of(p, c, steps);
    if (!f(t, c, i)) return;
    steps -= t.n;
    if (steps > 0) skip_ranges(p, c, 1);
  }
}

// The plan, block-wide: tiles 0 .. whole * units - 1 go to the blocks by turns (tile i to block
// i % units), so that the blocks read the same keys at about the same time and the cache holds
// them; of the others (between one and two for each block, if there are as many) each block
// gets a run of steps that evens out what it had before.
// mem: [kEntries + 1] steps and tiles before an entry each, [kThreads + 1] cuts, scratch,
// [kEntries] steps of an entry's tiles (the mean, where an entry holds several sequences).
__device__ void plan_tiles(const CrossParams& p, int64_t* mem, Run* run) {
  int64_t *steps_at = mem, *tiles_at = steps_at + kEntries + 1, *cut = tiles_at + kEntries + 1,
          *scratch = cut + kThreads + 1;
  int* per_tile = reinterpret_cast<int*>(scratch + 32);
  const int tid = threadIdx.x, units = p.tile_units;
  const int group = (p.B + kEntries - 1) / kEntries, entries = (p.B + group - 1) / group;
  int f = 0;
  bool z = false;
  int64_t total = 0, tiles = 0;
  for (int e0 = 0; e0 < entries; e0 += kThreads) {
    const int e = e0 + tid;
    int64_t s = 0, n = 0;
    if (e < entries) {
      const int b1 = min(p.B, (e + 1) * group);
      for (int b = e * group; b < b1; ++b) {
        const Seq q = read_seq<true>(p, b, &f, &z);
        s += (int64_t)q.steps * q.ranges;
        n += q.ranges;
      }
    }
    int64_t all_s, all_n;
    const int64_t upto_s = block_sum<kThreads>(s, &all_s, scratch);
    const int64_t upto_n = block_sum<kThreads>(n, &all_n, scratch);
    if (e < entries) {
      steps_at[e] = total + upto_s - s;
      tiles_at[e] = tiles + upto_n - n;
      per_tile[e] = n > 0 ? (int)quotient(s, n) : 0;
    }
    total += all_s;
    tiles += all_n;
  }
  if (tid == 0) {
    steps_at[entries] = total;
    tiles_at[entries] = tiles;
  }
  __syncthreads();
  const auto entry = [&](const int64_t* at, int64_t k) {   // the last with at[e] <= k
    int lo = 0, hi = entries - 1, e = 0;
    while (lo <= hi) {
      const int mid = (lo + hi) >> 1;
      if (at[mid] <= k) {
        e = mid;
        lo = mid + 1;
      } else {
        hi = mid - 1;
      }
    }
    return e;
  };
  // cursor at tile k, or (by_step) at step k; *before: steps before it
  const auto find = [&](int64_t k, bool by_step, int64_t* before) {
    const int64_t* at = by_step ? steps_at : tiles_at;
    const int e = entry(at, k);
    int64_t left = k - at[e], s = steps_at[e];
    Cursor c{};
    for (c.b = e * group; c.b < p.B; ++c.b) {
      c.q = read_seq<true>(p, c.b, &f, &z);
      const int64_t n = by_step ? (int64_t)c.q.steps * c.q.ranges : c.q.ranges;
      if (left < n) break;
      left -= n;
      s += (int64_t)c.q.steps * c.q.ranges;
    }
    c.r = by_step ? (int)quotient(left, max(c.q.steps, 1)) : (int)left;
    c.s = by_step ? (int)(left - (int64_t)c.r * c.q.steps) : 0;
    *before = s + (int64_t)c.r * c.q.steps + c.s;
    return c;
  };
  const int64_t whole = max(quotient(tiles, units) - 1, (int64_t)0);
  int64_t x, from = 0;
  if (whole > 0) {
    const int64_t k = whole * units;
    if (group == 1) {
      const int e = entry(tiles_at, k);
      from = steps_at[e] + (k - tiles_at[e]) * per_tile[e];
    } else {
      find(k, false, &from);
    }
  }
  const int64_t rest = total - from, share = quotient(total + units - 1, units);
  // what the whole tiles left of a block's share; of very many tiles the last 64 tell
  int64_t weight = 0;
  if (tid < units) {
    const int64_t i0 = max(whole - 64, (int64_t)0);
    int64_t had = i0 > 0 ? quotient(i0 * total, tiles) : 0, k = tid + i0 * units;
    for (int e = whole > 0 ? entry(tiles_at, k) : 0; k < whole * units; k += units) {
      while (tiles_at[e + 1] <= k) ++e;
      had += per_tile[e];
    }
    weight = whole > 0 ? max(share - had, (int64_t)1)
                       : tid < max(quotient(rest + kLeast - 1, kLeast), (int64_t)1);
  }
  // below 2^20 each, so that the product below stays below 2^63
  const int down = max(0, 44 - __clzll(share));
  if (weight > 0) weight = max(weight >> down, (int64_t)1);
  int64_t all;
  const int64_t upto = block_sum<kThreads>(weight, &all, scratch);
  if (tid == 0) cut[0] = from;
  if (tid < units) cut[tid + 1] = from + quotient(rest * upto, max(all, (int64_t)1));
  __syncthreads();
  // Few tiles: if every range can be cut into pieces of its own, at most `units` in all and not
  // much longer than an even share, the kv heads of a sequence are read in step: neighbouring
  // heads lie together in a cache row. (2 sequences of 100 queries, 16 heads of 64, 20000 to
  // 60000 keys: 80 us, cut at even shares 113 us.)
  if (tiles <= units && entries <= 64 && p.Hkv > 1) {
    // thread t tries pieces of at most lo + (hi - lo) * t / (kThreads - 1) steps
    const int lo = (int)max(share, (int64_t)kLeast), span = lo * 2 / 5;
    int need = 0;
    const int W = lo + span * tid / (kThreads - 1);
    for (int e = 0; e < entries; ++e)
      need += (int)(tiles_at[e + 1] - tiles_at[e]) * ((per_tile[e] + W - 1) / W);
    int* least = reinterpret_cast<int*>(scratch);
    if (tid == 0) *least = INT_MAX;
    __syncthreads();
    const uint32_t fit = __ballot_sync(0xffffffffu, need <= units);
    if (fit && (tid & 31) == __ffs(fit) - 1) atomicMin(least, W);
    __syncthreads();
    const int hi = *least;
    const bool found = hi != INT_MAX;
    __syncthreads();
    if (found) {   // hi: the longest piece
      for (int v = tid; v <= units; v += kThreads) cut[v] = total;
      __syncthreads();
      // units before an entry, entry by entry (at most `units` of them hold tiles)
      int first = 0;
      for (int e = 0; e < entries; ++e) {
        const int n = (int)(tiles_at[e + 1] - tiles_at[e]);
        if (n == 0) continue;
        const int s = per_tile[e], k = (s + hi - 1) / hi;
        const int len = (s + k - 1) / k;
        for (int v = tid; v < n * k; v += kThreads)
          cut[first + v] = steps_at[e] + (int64_t)(v / k) * s + min(v % k * len, s);
        first += n * k;
      }
      __syncthreads();
    }
  }
  const int u = blockIdx.x;
  const int64_t c0 = cut[u], c1 = cut[u + 1];
  if (tid == 0) {
    run->whole = (int)whole;
    run->steps = c1 - c0;
  }
  if (tid == 32 && whole > 0) run->first = find(u, false, &x);
  if (tid == 64 && c1 > c0) run->at = find(c0, true, &x);
  if (tid == 96) {   // the record: the range that begins in the run and ends behind it
    int4 a = make_int4(0, 0, 0, 0), b = make_int4(0, 0, 0, 0);
    if (c1 > c0) {
      const Cursor c = find(c1 - 1, true, &x);
      const int64_t start = c1 - 1 - c.s, end = start + c.q.steps;
      if (start >= c0 && end > c1) {
        int v = u;
        while (v + 1 < units && cut[v + 1] < end) ++v;
        const Part t = part_of(p, c, 1);
        a = make_int4(v - u + 1, start == c0 ? 0 : 1, t.row0, t.h);
        b.x = t.pos;
      }
    }
    p.tile_rec[2 * u] = a;
    p.tile_rec[2 * u + 1] = b;
  }
}

// ---------------------------------------------------------------------------- loader
// Two warps, one for the key tiles (and Q, and the masks), one for the value tiles: a box costs
// its issuing warp some 210 cycles.
// R keys from group of 8 `group` of the pool on, kv head h
__device__ __forceinline__ void load_box(void* dst, const void* map, int group, int h,
                                         uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %2, %2, %3, %4}], [%5];\n" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(group), "r"(h), "r"(smem_u32(bar))
      : "memory");
}

template <typename T, int D>
__device__ void load_role(const CrossParams& p, const Maps& maps, unsigned char* sm,
                          int kv, const Run& run, const Wait& wait) {
  using L = Lay<D>;
  uint64_t* bars = wait.bars;
  const int lane = threadIdx.x & 31, R = p.box_keys;
  int flags = 0;
  uint32_t use = (uint32_t)kv, issued = 0;   // ring tile, tiles issued
  Place<L::kStages> to;
  to.step(kv);
  uint32_t* seen_words = reinterpret_cast<uint32_t*>(sm + L::kSeen);
  uint32_t q_use[2] = {0, 0};
  const uint32_t every = R > 0 ? 0xffffffffu >> (32 - kTileKeys / R) : 0u;   // boxes of a tile
  const bool withhold = p.withhold_copy != 0;   // testing hook: the first K tile never comes
  // Room for the tile `use`: the one kStages before it was given back. A wait for a parity tells
  // two rounds of a stage apart, not three, so the round before must be known to be over. That is
  // the loader's own doing where its tiles come back to the same stages; with an odd number of
  // stages they alternate with the other loader's, which has to have found room for that tile.
  //
  // Room for the masks of step J = use / 2, which take the place of step J - kMasks's: those were
  // read by every warp of the halves at work on that step once its value tile was given back (each
  // half gives it back behind its product, and that waits for the weights of all four warps; the
  // key tile is given back in front of that, by one warp). With an odd number of stages the room
  // for the key tile of step J - kMasks + (kStages + 1) / 2 has told so. With an even one the
  // other loader tells: it found room for the tile kStages behind that value tile, 2 (J - kMasks) +
  // 1 + kStages. (That value tile came back before the key tile two steps behind it, whose stage
  // this one takes.)
  volatile uint32_t* found = reinterpret_cast<volatile uint32_t*>(sm + L::kBars + kRoomWord);
  constexpr bool kAlternate = L::kStages % 2 != 0;
  static_assert(kAlternate ? (L::kStages + 1) / 2 <= kMasks : L::kStages < 2 * kMasks, "mask ring");
  const auto other_found = [&](uint32_t tiles) {   // waits for the other loader's `found`
    bool there = false;
    for (uint32_t i = 0; i < wait.tries && !there; ++i) {
      there = found[1 - kv] >= tiles;
      if ((i & 255u) == 255u && *wait.abort) break;
    }
    if (!there) *wait.abort = 1;
    return __all_sync(0xffffffffu, there) != 0;
  };
  const auto room = [&]() {
    if (use >= (uint32_t)L::kStages) {
      if (kAlternate && !other_found(use + 1 - L::kStages)) return false;
      if (!wait.warp(kEmpty + to.stage, to.phase ^ 1u)) return false;
    }
    if (!kAlternate && kv == 0 && use >= 2u * kMasks &&
        !other_found(use + 2 + L::kStages - 2 * kMasks))
      return false;
    if ((kAlternate || kv == 1) && lane == 0) found[kv] = use + 1;
    return true;
  };
  // announces `bytes` and copies the boxes whose bits are set, box i from group `group` of lane i;
  // the whole warp (see the products)
  const auto issue = [&](unsigned char* dst, uint64_t* full, int group, uint32_t boxes,
                         uint32_t bytes, int h) {
    const void* map = kv == 0 ? &maps.k : &maps.v;
    int at[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) at[i] = __shfl_sync(0xffffffffu, group, i);
    if (withhold && use == 0) boxes = 0;
    __syncwarp();   // the masks are written before the tile is announced
    if (elect()) {
      tc::mbar_arrive_expect_tx(full, bytes);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if ((boxes >> i) & 1u) load_box(dst + i * (R / 8) * L::kGroup, map, at[i], h, full);
    }
    __syncwarp();
    for (int i0 = 4; i0 < 16 && (boxes >> i0) != 0; i0 += 4) {   // boxes of 8 or 16 keys
#pragma unroll
      for (int i = 0; i < 4; ++i) at[i] = __shfl_sync(0xffffffffu, group, i0 + i);
      if (elect()) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if ((boxes >> (i0 + i)) & 1u)
            load_box(dst + (i0 + i) * (R / 8) * L::kGroup, map, at[i], h, full);
      }
      __syncwarp();
    }
  };
  each_part(p, run, [&](const Part& t, const Cursor& c, int) {
    const int PT = p.tile_pos / 2;
    for (int h = 0; kv == 0 && h < (t.shared ? 2 : t.halves); ++h) {
      if (q_use[h] > 0 &&
          !wait.warp(kQEmpty + h, (q_use[h] - 1) & 1u))
        return false;
      ++q_use[h];
      if (lane == 0) {
        tc::mbar_arrive_expect_tx(bars + kQFull + h, (uint32_t)(PT * p.G) * (D * 2));
#pragma unroll
        for (int x = 0; x < D / 64; ++x)
          tc::tma_load_3d(sm + L::kQ + h * L::kTile + x * L::kSub, &maps.q, x * 64, t.h * p.G,
                          t.row0 + (t.shared ? 0 : h * PT), bars + kQFull + h);
      }
    }
    // R consecutive keys of a block to a lane (none when rows are copied one by one); the block
    // of the step ahead is on its way while a step is loaded
    const auto column = [&](int key) { return p.bs_shift >= 0 ? key >> p.bs_shift : key / p.BS; };
    const auto lookup = [&](int key) {
      int blk;
      asm volatile("ld.global.nc.b32 %0, [%1];\n"
                   : "=r"(blk)
                   : "l"(p.table + (int64_t)t.b * p.MB + column(min(key, c.q.keys - 1))));
      return blk;
    };
    int ahead = lookup(c.s * kTileKeys + lane * R);
    for (int j = c.s; j < c.s + t.n; ++j, use += 2, ++issued) {
      const int key0 = j * kTileKeys + lane * R;
      const bool there = R > 0 && lane * R < kTileKeys && key0 < c.q.keys;
      const bool mapped = there && ahead >= 0 && ahead < p.NB;
      const int row = ahead * p.BS + (key0 - column(key0) * p.BS);   // where mapped
      const uint32_t boxes = __ballot_sync(0xffffffffu, mapped);
      const bool clear = R > 0 && (j + 1) * kTileKeys <= c.q.keys && boxes == every;
      ahead = lookup(key0 + kTileKeys);
      if (!room()) return false;
      unsigned char* dst = sm + L::kRing + to.stage * L::kTile;
      uint64_t* full = bars + kFull + to.stage;
      to.step(2);
      // Which keys take part: key 4 i + x of the step is bit i of word x.
      uint32_t* seen = seen_words + (use / 2 % kMasks) * 4 + lane;
      if (clear) {   // every key is there: whole boxes, nothing masked
        if (kv == 0 && lane < 4) *seen = 0xffffffffu;
        issue(dst, full, row / 8, boxes, L::kTile, t.h);
        continue;
      }
      if (there && !mapped) flags |= PKV_DEV_BAD_BLOCK;
      if (kv == 0) {
        const int k0 = j * kTileKeys + 4 * lane;   // 4 keys of one block, if boxes are used
        uint32_t words[4];
        if (R > 0) {
          const bool in = __shfl_sync(0xffffffffu, mapped ? 1 : 0, 4 * lane / R) != 0;
#pragma unroll
          for (int x = 0; x < 4; ++x)
            words[x] = __ballot_sync(0xffffffffu, in && k0 + x < c.q.keys);
        } else {
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int blk = lookup(k0 + x);
            words[x] = __ballot_sync(0xffffffffu, blk >= 0 && blk < p.NB && k0 + x < c.q.keys);
          }
        }
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (lane == x) *seen = words[x];
      }
      {
        // key rows behind the last key may stay what they are: their scores are masked
        const bool whole = mapped && key0 + R <= c.q.keys;
        const uint32_t copy = __ballot_sync(0xffffffffu, kv == 0 ? mapped : whole);
        const T* src = static_cast<const T*>(kv == 0 ? p.kc : p.vc);
        bool rows = false;   // rows copied one by one
        if (R == 0) {
          rows = true;
          for (int r = 0; r < kTileKeys; ++r) {
            const int key = j * kTileKeys + r;
            int64_t at = -1;
            if (key < c.q.keys) {
              const int col = p.bs_shift >= 0 ? key >> p.bs_shift : key / p.BS;
              const int blk = __ldg(p.table + (int64_t)t.b * p.MB + col);
              if (blk >= 0 && blk < p.NB)
                at = (((int64_t)blk * p.BS + (key - col * p.BS)) * p.Hkv + t.h) * D;
              else
                flags |= PKV_DEV_BAD_BLOCK;
            }
            if (lane < D / 8)
              cp_async_16(dst + (r >> 3) * L::kGroup + (lane >> 3) * 1024 +
                              tc::sw128(r & 7, lane & 7),
                          at >= 0 ? src + at + lane * 8 : src, at >= 0 ? 16 : 0);
          }
        } else if (kv == 1) {
          uint32_t rest = __ballot_sync(0xffffffffu, lane * R < kTileKeys && !whole);
          rows = rest != 0;
          for (; rest; rest &= rest - 1) {
            const int i = __ffs(rest) - 1;
            const int row_i = __shfl_sync(0xffffffffu, row, i);
            const int mapped_i = __shfl_sync(0xffffffffu, mapped ? 1 : 0, i);
            for (int x = lane; x < R * (D / 8); x += 32) {
              const int r = x / (D / 8), ch = x % (D / 8);
              const bool live = mapped_i && j * kTileKeys + i * R + r < c.q.keys;
              const int64_t at = live ? ((int64_t)(row_i + r) * p.Hkv + t.h) * D + ch * 8 : 0;
              const int k = i * R + r;
              cp_async_16(dst + (k >> 3) * L::kGroup + (ch >> 3) * 1024 + tc::sw128(k & 7, ch & 7),
                          src + at, live ? 16 : 0);
            }
          }
        }
        if (rows) {   // these were written by threads: hand them to the tensor core's proxy
          cp_async_commit();
          cp_async_wait<0>();
          tc::fence_async_shared();
          __syncwarp();
        }
        issue(dst, full, row / 8, copy, (uint32_t)__popc(copy) * R * (D * 2), t.h);
      }
    }
    return true;
  });
  if (flags) flag_status(p.status, flags);
  if (*wait.abort) {   // let what was issued land before the block ends
    for (uint32_t k = 1; k <= min(issued, (uint32_t)(L::kStages + 1) / 2); ++k) {
      const uint32_t u = use - 2 * k;
      tc::mbar_wait(bars + kFull + u % L::kStages, (u / L::kStages) & 1u, wait.tries);
    }
    for (int h = 0; h < 2; ++h)
      if (q_use[h] > 0) tc::mbar_wait(bars + kQFull + h, (q_use[h] - 1) & 1u, wait.tries);
  }
}

// ---------------------------------------------------------------------------- products
template <typename T, int D>
__device__ void mma_role(const CrossParams& p, unsigned char* sm, int half, const Run& run,
                         const Wait& wait) {
  using L = Lay<D>;
  uint64_t* bars = wait.bars;
  constexpr uint32_t fmt = Num<T>::kBf16 ? (1u << 7) | (1u << 10) : 0u;   // types of A and B
  constexpr uint32_t id_s = tc::idesc_f16(128, 128, false, false) | fmt;
  constexpr uint32_t id_o = tc::idesc_f16(128, D, false, true) | fmt;
  const uint32_t q_at = smem_u32(sm + L::kQ) + half * L::kTile, ring = smem_u32(sm + L::kRing);
  const uint32_t s_at = run.tmem + half * 128, o_at = run.tmem + 256 + half * 128;
  uint32_t q_use = 0, p_use = 0, turn = 0;
  Place<L::kStages> next;   // of the part's first K tile
  const auto ready = [&](int bar, uint32_t parity) {
    return wait.warp(bar, parity);
  };
  // The halves issue by turns, half 0 first: without it the tensor core shares itself out
  // between both, they end together, and then both softmaxes run while it idles.
  const auto my_turn = [&](bool both) {
    if (!both) return true;
    const uint32_t n = turn++;
    if (half == 0) return n == 0 || ready(kTurn, (n - 1) & 1u);
    return ready(kTurn + 1, n & 1u);
  };
  each_part(p, run, [&](const Part& t, const Cursor&, int) {
    Place<L::kStages> k = next, v = next;   // K of step j is 2 j tiles on, V 2 j + 1
    next.step(2 * t.n);
    if (!t.active(half)) return true;
    const bool both = t.shared || t.halves == 2;
    const int n = t.count(half), apart = 2 * t.stride();
    k.step(2 * t.first(half));
    v.step(2 * t.first(half) + 1);
    // round i: PV of this half's step i - 1, S of step i
    for (int i = 0; i <= n; ++i) {
      const bool pv = i > 0, s = i < n;
      if (i == 0 && !ready(kQFull + half, q_use++ & 1u)) return false;
      if (pv && !ready(kFull + v.stage, v.phase)) return false;
      // A parity waited for too early is that of two rounds before. What the stage of this K tile
      // held before may be the other half's: an earlier part's, or (an odd number of stages) a
      // value tile of this shared part; then its turn tells that it landed. Else there is no need
      // to wait with the question (head size 64: 80 us, asked behind the turn 84 us).
      const bool early = i > 0 && (L::kStages % 2 == 0 || !t.shared);
      if (s && early && !ready(kFull + k.stage, k.phase)) return false;
      if (!my_turn(both)) return false;
      if (pv && !ready(kPFull + half, p_use & 1u)) return false;
      tc::fence_after_sync();
      const uint32_t va = ring + v.stage * L::kTile, ka = ring + k.stage * L::kTile;
      if (pv) {
        const auto products = [&](int ks) {
          mma_tmem_a(o_at, s_at + (uint32_t)ks * 8u,
                     tc::smem_desc(va + (uint32_t)ks * 2 * L::kGroup, 1024, L::kGroup), id_o,
                     i == 1 && ks == 0 ? 0u : 1u);
        };
        if (elect()) {
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) products(ks);
        }
        __syncwarp();
        if (!ready(kPRest + half, p_use++ & 1u)) return false;
        tc::fence_after_sync();
        if (elect()) {
#pragma unroll
          for (int ks = 4; ks < 8; ++ks) products(ks);
          if (L::kScarce && t.shared) {   // both arrivals; the S behind may wait for its keys
            tc::commit(bars + kEmpty + v.stage);
            tc::commit(bars + kEmpty + v.stage);
          }
        }
        __syncwarp();
        v.step(apart);
      }
      if (s && !early) {   // behind the PV: that gives a stage back while this tile is on its way
        if (!ready(kFull + k.stage, k.phase)) return false;
        tc::fence_after_sync();
      }
      if (elect()) {
        // the other half's turn; it takes about as long to notice as the S below to be issued
        if (both) arrive(bars + kTurn + 1 - half);
        if (s) {
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint32_t x = (uint32_t)(ks & 3) * 32u, sub = (uint32_t)(ks >> 2);
            tc::mma_f16(s_at, tc::smem_desc(q_at + sub * L::kSub + x, 16, 1024),
                        tc::smem_desc(ka + sub * 1024u + x, 16, L::kGroup), id_s, ks > 0 ? 1u : 0u);
          }
          tc::commit(bars + kSFull + half);
          if (i + 1 == n) tc::commit(bars + kQEmpty + half);
        } else {
          tc::commit(bars + kOFull + half);
        }
      }
      __syncwarp();
      k.step(apart);
    }
    if (both && n < t.count(0)) {   // as many turns as the other half
      if (!my_turn(true)) return false;
      if (elect()) arrive(bars + kTurn + 1 - half);
      __syncwarp();
    }
    return true;
  });
  if (*wait.abort) {
    if (elect()) tc::commit(bars + kDrain + half);
    __syncwarp();
    tc::mbar_wait(bars + kDrain + half, 0, wait.tries);
  }
}

// ---------------------------------------------------------------------------- softmax
template <typename T, int D>
__device__ void softmax_role(const CrossParams& p, unsigned char* sm, const Run& run,
                             const Wait& wait) {
  using L = Lay<D>;
  uint64_t* bars = wait.bars;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int half = warp >> 2, r = threadIdx.x & 127;
  const uint32_t lane_at = run.tmem + ((uint32_t)(r & ~31) << 16);
  const uint32_t s_at = lane_at + half * 128, o_at = lane_at + 256 + half * 128;
  const float sl2 = fabsf(p.scale_log2);   // a negative scale turns the scores around
  const uint64_t scale2 = pair_of(sl2, sl2);
  uint32_t s_use = 0, o_use = 0, use = 0, pair_use = 0;
  Place<L::kStages> next;   // of the part's first K tile
  float2* pair_ml = reinterpret_cast<float2*>(sm + L::kPairMl) + r;
  const auto hand_over = [&](int bar) {   // the warp's weights so far, to the products
    tc::tmem_wait_st();
    tc::fence_before_sync();
    __syncwarp();
    if (lane == 0) arrive(bars + bar + half);
  };
  each_part(p, run, [&](const Part& t, const Cursor&, int index) {
    uint32_t k = use + 2 * t.first(half);   // ring tile of this half's K; V is k + 1
    Place<L::kStages> tile = next;          // the next tile to be given back: K, V, K, V ...
    use += 2 * t.n;
    next.step(2 * t.n);
    if (!t.active(half)) return true;
    const uint32_t apart = 2 * t.stride();
    tile.step(2 * t.first(half));
    // Two arrivals free a tile: the halves', or both from the one half that reads it. A full S
    // tells that the products in front of it are done. (Committed by the issuing lane instead, an
    // arrival takes it some 90 cycles; so it is done where stages are scarce alone: the value tiles
    // of shared parts of head size 128. 64 x 4000 states, 20 rows of 8 kv heads: 217 us, 260 us
    // without.)
    const auto give_back = [&](int further, bool given) {
      if (!given) arrive(bars + kEmpty + tile.stage, t.halves == 2 ? 1 : 2);
      tile.step(further);
    };
    float m = -INFINITY, l = 0.f;
    const int n = t.count(half);
    for (int j = 0; j < n; ++j, k += apart) {
      // the loads and stores of TMEM below are the whole warp's
      if (!wait.warp(kSFull + half, s_use & 1u)) return false;
      ++s_use;
      tc::fence_after_sync();
      if (r == 0) {
        if (j > 0) give_back((int)apart - 1, L::kScarce && t.shared);   // V of the step before
        give_back(1, false);                              // K of this one
      }
      float v[128], e[4];
      {
        float (*v32)[32] = reinterpret_cast<float (*)[32]>(v);
#pragma unroll
        for (int x = 0; x < 4; ++x) tmem_ld32_max(s_at + x * 32, v32[x], e[x]);
      }
      const uint4 seen = *reinterpret_cast<const uint4*>(sm + L::kSeen + (k / 2 % kMasks) * 16);
      tc::tmem_wait_ld();
      const bool masked = (seen.x & seen.y & seen.z & seen.w) != 0xffffffffu;
      if (masked || p.scale_log2 < 0.f) {   // the maximum is another one
        const float sign = p.scale_log2 < 0.f ? -1.f : 1.f;
#pragma unroll
        for (int x = 0; x < 32; ++x) {
          v[4 * x] = (seen.x >> x) & 1u ? sign * v[4 * x] : -INFINITY;
          v[4 * x + 1] = (seen.y >> x) & 1u ? sign * v[4 * x + 1] : -INFINITY;
          v[4 * x + 2] = (seen.z >> x) & 1u ? sign * v[4 * x + 2] : -INFINITY;
          v[4 * x + 3] = (seen.w >> x) & 1u ? sign * v[4 * x + 3] : -INFINITY;
        }
#pragma unroll
        for (int y = 0; y < 4; ++y) e[y] = fmaxf(v[2 * y], v[2 * y + 1]);
#pragma unroll
        for (int x = 8; x < 128; x += 8)
#pragma unroll
          for (int y = 0; y < 4; ++y) e[y] = max3(e[y], v[x + 2 * y], v[x + 2 * y + 1]);
      }
      float top = max3(e[0], e[1], fmaxf(e[2], e[3]));
      top *= sl2;   // -inf when nothing of the step is seen
      if (__any_sync(0xffffffffu, m == -INFINITY ? top != -INFINITY : top > m + (kLift + kRaise))) {
        const bool first = m == -INFINITY;
        const bool raise = first ? top != -INFINITY : top > m + (kLift + kRaise);
        const float alpha = raise && !first ? ex2(m - (top - kLift)) : 1.f;
        if (raise) m = top - kLift;
        l *= alpha;
        if (j > 0) {   // O is complete: see the order of the products
#pragma unroll 1
          for (int x = 0; x < D / 16; ++x) {
            float o[16];
            tmem_ld16(o_at + x * 16, o);
            tc::tmem_wait_ld();
#pragma unroll
            for (int y = 0; y < 16; ++y) o[y] *= alpha;
            tmem_st16(o_at + x * 16, o);
          }
        }
      }
      const float base = m == -INFINITY ? 0.f : -m;
      const uint64_t base2 = pair_of(base, base);
      uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float w[16];   // 32 weights as pairs
#pragma unroll
        for (int x = 0; x < 32; x += 2) {
          const uint64_t e2 = fma_pair(pair_of(v[q * 32 + x], v[q * 32 + x + 1]), scale2, base2);
          const float e0 = ex2(low_of(e2)), e1 = ex2(high_of(e2));
          sum[(x >> 1) & 3] = add_pair(sum[(x >> 1) & 3], pair_of(e0, e1));
          w[x / 2] = __uint_as_float(Num<T>::pack(e0, e1));
        }
        tmem_st16(s_at + q * 16, w);
        if (q == 1) hand_over(kPFull);
      }
      sum[0] = add_pair(add_pair(sum[0], sum[1]), add_pair(sum[2], sum[3]));
      l += low_of(sum[0]) + high_of(sum[0]);
      hand_over(kPRest);
    }
    if (!wait.warp(kOFull + half, o_use & 1u)) return false;
    ++o_use;
    tc::fence_after_sync();
    if (r == 0) give_back(1, L::kScarce && t.shared);
    float mine_by = 1.f, other_by = 0.f;   // what this half's O counts for, and the other's
    if (t.shared) {
      if (half == 1) {
        *pair_ml = make_float2(m, l);
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) arrive(bars + kPair);
        if (!wait.warp(kPairRead, pair_use++ & 1u)) return false;
        tc::fence_after_sync();
        return true;
      }
      if (!wait.warp(kPair, pair_use++ & 1u)) return false;
      tc::fence_after_sync();
      const float2 other = *pair_ml;
      const float top = fmaxf(l == 0.f ? -INFINITY : m, other.y == 0.f ? -INFINITY : other.x);
      const float base = top == -INFINITY ? 0.f : top;
      mine_by = l == 0.f ? 0.f : ex2(m - base);
      other_by = other.y == 0.f ? 0.f : ex2(other.x - base);
      m = top;
      l = l * mine_by + other.y * other_by;
    }
    const auto result = [&](int x, float (&o)[32]) {   // 32 columns of O
      tc::tmem_ld32(o_at + x * 32, o);
      tc::tmem_wait_ld();
      if (t.shared) {
        float y[32];
        tc::tmem_ld32(o_at + 128 + x * 32, y);
        tc::tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          o[i] = mine_by == 0.f ? 0.f : o[i] * mine_by;   // no weight: anything may stand there
          o[i] += other_by == 0.f ? 0.f : y[i] * other_by;
        }
      }
    };
    const int pos = half * (p.tile_pos / 2) + r / p.G;
    const bool mine = r < (p.tile_pos / 2) * p.G && pos < t.pos;
    if (t.whole) {
      const float inv = inverse_of(l);
      const int64_t row = (int64_t)(t.row0 + pos) * p.Hq + t.h * p.G + r % p.G;
      uint4* out = reinterpret_cast<uint4*>(static_cast<T*>(p.out) + row * D);
#pragma unroll
      for (int x = 0; x < D / 32; ++x) {
        float o[32];
        result(x, o);
        if (mine) {
#pragma unroll
          for (int y = 0; y < 4; ++y)
            out[x * 4 + y] = make_uint4(Num<T>::pack(o[y * 8] * inv, o[y * 8 + 1] * inv),
                                        Num<T>::pack(o[y * 8 + 2] * inv, o[y * 8 + 3] * inv),
                                        Num<T>::pack(o[y * 8 + 4] * inv, o[y * 8 + 5] * inv),
                                        Num<T>::pack(o[y * 8 + 6] * inv, o[y * 8 + 7] * inv));
        }
      }
      if (mine && p.lse) p.lse[row] = lse_of(m, l);
    } else {
      const int64_t row = (2 * (int64_t)blockIdx.x + (index == 0 ? 0 : 1)) * 256 + half * 128 + r;
      float4* out = reinterpret_cast<float4*>(p.tile_o + row * D);
#pragma unroll
      for (int x = 0; x < D / 32; ++x) {
        float o[32];
        result(x, o);
        if (mine) {
#pragma unroll
          for (int y = 0; y < 8; ++y)
            out[x * 8 + y] = make_float4(o[y * 4], o[y * 4 + 1], o[y * 4 + 2], o[y * 4 + 3]);
        }
      }
      if (mine) {
        p.tile_m[row] = m;
        p.tile_l[row] = l;
      }
    }
    tc::fence_before_sync();
    if (t.shared) {
      __syncwarp();
      if (lane == 0) arrive(bars + kPairRead);
    }
    return true;
  });
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1)
    cross_tiles_kernel(CrossParams p, const __grid_constant__ Maps maps) {
  using L = Lay<D>;
  extern __shared__ __align__(1024) unsigned char raw[];
  unsigned char* sm = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(raw) + 1023) & ~static_cast<uintptr_t>(1023));
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  Wait wait;
  wait.bars = reinterpret_cast<uint64_t*>(sm + L::kBars);
  wait.abort = reinterpret_cast<volatile int*>(sm + L::kBars + kAbortWord);
  wait.tries = p.wait_tries ? p.wait_tries : kTries;
  Run* run = reinterpret_cast<Run*>(sm + L::kRun);
  if (tid == 0) {
    for (int i = 0; i < L::kStages; ++i) {
      tc::mbar_init(wait.bars + kFull + i, 1);
      tc::mbar_init(wait.bars + kEmpty + i, 2);
    }
    for (int h = 0; h < 2; ++h) {
      tc::mbar_init(wait.bars + kQFull + h, 1);
      tc::mbar_init(wait.bars + kQEmpty + h, 1);
      tc::mbar_init(wait.bars + kSFull + h, 1);
      tc::mbar_init(wait.bars + kPFull + h, 4);
      tc::mbar_init(wait.bars + kPRest + h, 4);
      tc::mbar_init(wait.bars + kOFull + h, 1);
      tc::mbar_init(wait.bars + kDrain + h, 1);
      tc::mbar_init(wait.bars + kTurn + h, 1);
    }
    tc::mbar_init(wait.bars + kPair, 4);
    tc::mbar_init(wait.bars + kPairRead, 4);
    tc::mbar_init_fence();
    *wait.abort = 0;
    uint32_t* found = reinterpret_cast<uint32_t*>(sm + L::kBars + kRoomWord);
    found[0] = found[1] = 0;
  }
  if (warp == kSoftmaxWarps + 1 && lane == 0 && p.box_keys > 0) {
    tc::tma_prefetch_desc(&maps.q);
    tc::tma_prefetch_desc(&maps.k);
    tc::tma_prefetch_desc(&maps.v);
  }
  if (warp == 0) {
    tc::tmem_alloc(&run->tmem, 512);
    tc::tmem_relinquish();
  }
  // in the ring's memory before the ring is used; the other kernel reports bad sequences
  plan_tiles(p, reinterpret_cast<int64_t*>(sm + L::kRing), run);
  tc::fence_async_shared();
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (run->steps == 0 && tid < 256)   // a piece of nothing, if a join counts this block in
    p.tile_l[(int64_t)blockIdx.x * 512 + tid] = 0.f;
  if (run->whole > 0 || run->steps > 0) {
    if (warp < kSoftmaxWarps) {
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kSoftmaxRegs));
      softmax_role<T, D>(p, sm, *run, wait);
    } else {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kOtherRegs));
      if (warp == kSoftmaxWarps || warp == kSoftmaxWarps + 2)
        mma_role<T, D>(p, sm, (warp - kSoftmaxWarps) / 2, *run, wait);
      else
        load_role<T, D>(p, maps, sm, warp == kSoftmaxWarps + 1 ? 0 : 1, *run, wait);
    }
  }
  cp_async_wait<0>();
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (tid == 0 && *wait.abort) flag_status(p.status, PKV_DEV_TIMEOUT);
  if (warp == 0) tc::tmem_dealloc(run->tmem, 512);
}

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  return fn;
}

bool encode(CUtensorMap* m, bool bf16, const void* base, int rank, const cuuint64_t* dims,
            const cuuint64_t* strides, const cuuint32_t* box) {
  const PFN_cuTensorMapEncodeTiled_v12000 fn = encoder();
  if (!fn) return false;
  const cuuint32_t unit[5] = {1, 1, 1, 1, 1};
  return fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
            (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, unit,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Q [tokens][Hq][D]: boxes of 64 elements x G heads x 128 / G positions
bool encode_queries(CUtensorMap* m, const CrossParams& p) {
  const cuuint64_t D = p.D, dims[3] = {D, (cuuint64_t)p.Hq, (cuuint64_t)p.T};
  const cuuint64_t strides[2] = {D * 2, p.Hq * D * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)p.G, (cuuint32_t)(p.tile_pos / 2)};
  return encode(m, p.bf16, p.q, 3, dims, strides, box);
}

// a pool [rows][Hkv][D] as [Hkv][rows / 8][D / 64][8][64]: boxes of box_keys rows of one head
bool encode_pool(CUtensorMap* m, const CrossParams& p, const void* base) {
  const cuuint64_t D = p.D, row = p.Hkv * D * 2;
  const cuuint64_t dims[5] = {64, 8, D / 64, (cuuint64_t)p.NB * p.BS / 8, (cuuint64_t)p.Hkv};
  const cuuint64_t strides[4] = {row, 128, 8 * row, D * 2};
  const cuuint32_t box[5] = {64, 8, (cuuint32_t)p.D / 64, (cuuint32_t)p.box_keys / 8, 1};
  return encode(m, p.bf16, base, 5, dims, strides, box);
}

template <typename T, int D>
cudaError_t launch_typed(const CrossParams& p, cudaStream_t s) {
  static std::atomic<uint64_t> configured{0};
  int dev = -1;
  if (needs_configure(configured, &dev)) {
    cudaFuncAttributes at;
    cudaError_t e = cudaFuncGetAttributes(&at, cross_tiles_kernel<T, D>);
    if (e != cudaSuccess) return e;
    if (at.numRegs < kLaunchRegs) return cudaErrorInvalidConfiguration;   // the split would not fit
    e = cudaFuncSetAttribute(cross_tiles_kernel<T, D>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Lay<D>::kBytes);
    if (e != cudaSuccess) return e;
    mark_configured(configured, dev);
  }
  Maps maps;
  if (!encode_queries(&maps.q, p)) return cudaErrorInvalidValue;
  maps.k = maps.v = maps.q;   // not used without boxes
  if (p.box_keys > 0 && (!encode_pool(&maps.k, p, p.kc) || !encode_pool(&maps.v, p, p.vc)))
    return cudaErrorInvalidValue;
  ProfScope ps("cross_tiles", s);
  cross_tiles_kernel<T, D><<<p.tile_units, kThreads, Lay<D>::kBytes, s>>>(p, maps);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cross_tiles(const CrossParams& p, cudaStream_t s) {
  if (p.bf16)
    return p.D == 64 ? launch_typed<__nv_bfloat16, 64>(p, s)
                     : launch_typed<__nv_bfloat16, 128>(p, s);
  return p.D == 64 ? launch_typed<__half, 64>(p, s) : launch_typed<__half, 128>(p, s);
}

}  // namespace pkv
