// Cross attention, sequences with many query rows: tiles on the 5th-generation tensor core.
//
// A range is a tile of 256 rows = two halves of 128 rows = (128 / G) query positions x G
// heads of one kv head each, against 128 keys a step. Per step the tensor core does
// S = Q K^T and O += P V for both halves (4 * 128 * 128 * D multiply-adds); the halves take
// turns, so one half's softmax runs while the other half's products do:
//   warps 0-3, 4-7  softmax of half 0, 1: a thread owns a row (one TMEM lane). It reads its 128
//                   scores, raises its running maximum only when they exceed it by 2^8 (then O
//                   and l are rescaled), writes the weights, rounded once to T, over the scores
//                   in TMEM, and at the end writes its output row, or its piece.
//   warp 8          one thread issues every tcgen05.mma, in the order
//                   PV_0(j) S_0(j+1) PV_1(j) S_1(j+1): products of one issuing thread run in
//                   order, so S may overwrite the weights that the PV before it reads, and a
//                   full S tells that the O of that half is complete.
//   warp 9          loads by TMA into 128-byte-swizzled shared memory: Q of the halves, and one
//                   ring of K and V tiles in the order of their use (K0 V0 K1 V1 ...). A box is
//                   up to 128 keys of one cache block. Value rows past the sequence's keys or in
//                   unmapped blocks are zero-filled (a weight of zero times what stands there
//                   must be zero); block sizes that are no multiple of 8 go row by row.
// TMEM columns: S_0 0..127 (weights over 0..63), S_1 128..255, O_0 256.., O_1 384...
#include <cuda.h>
#include <cudaTypedefs.h>

#include "cross_dev.cuh"
#include "tcgen05.cuh"

namespace pkv {
namespace {

using namespace cross;

constexpr int kThreads = 384;
constexpr int kLeast = 4;              // steps of a run, at least
constexpr uint32_t kTries = 1u << 22;  // default bound of a wait (polls)
constexpr float kRaise = 8.f;          // log2 of the largest weight under an old maximum
// registers a thread: launch, softmax warpgroups, the third warpgroup. 256 * 208 + 128 * 88 =
// 384 * 168: the two that grow take what the third gives back
constexpr int kLaunchRegs = 168, kSoftmaxRegs = 208, kOtherRegs = 88;
static_assert(256 * kSoftmaxRegs + 128 * kOtherRegs <= kThreads * kLaunchRegs, "register split");

template <int D>
struct Lay {   // byte offsets from a 1024-byte-aligned base
  static constexpr int kStages = D == 128 ? 5 : 8;
  static constexpr uint32_t kTile = 128u * D * 2;       // 128 rows of Q, K or V
  static constexpr uint32_t kSub = 128u * 128;          // 64 columns of them
  static constexpr uint32_t kQ = 0;
  static constexpr uint32_t kRing = 2 * kTile;
  static constexpr uint32_t kBars = kRing + kStages * kTile;
  static constexpr uint32_t kEnd = kBars + 256;
  static constexpr size_t kBytes = kEnd + 1024;
};
static_assert(Lay<128>::kBytes <= 232448, "shared memory over the limit");
static_assert((kEntries + 16) * 8 <= Lay<64>::kStages * Lay<64>::kTile, "plan fits the ring");

// mbarriers
enum {
  kFull = 0,     // + stage: K or V tile landed (32 lanes' copies + 1 with the TMA bytes)
  kEmpty = 8,    // + stage: the products that read it completed
  kQFull = 16,   // + half
  kQEmpty = 18,  // + half: every S of the range completed
  kSFull = 20,   // + half: S in TMEM (and the O before it complete)
  kPFull = 22,   // + half: the 4 warps wrote their weights
  kOFull = 24,   // + half: the last PV of the range completed
  kDrain = 26,   // products in flight when a wait gave up
  kBarriers = 27
};
constexpr uint32_t kTmemWord = 27 * 8, kAbortWord = 27 * 8 + 4;   // behind the barriers
static_assert(kAbortWord + 4 <= 256, "barrier area");

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
};

__device__ __forceinline__ void arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(smem_u32(bar)) : "memory");
}
// arrive when every cp.async that this thread issued has landed
__device__ __forceinline__ void arrive_copies(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];\n" ::"r"(smem_u32(bar))
               : "memory");
}

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

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// This unit's part of a range: the tile under the cursor, steps [c.s, c.s + n).
struct Part {
  int b, h, row0, pos, n, halves;   // first query row of the tile, its positions, steps, halves
  bool whole;
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
  return t;
}

// Walks the parts of a run; every role walks for itself.
template <typename F>
__device__ __forceinline__ void each_part(const CrossParams& p, Cursor c, int64_t steps, F f) {
  for (int i = 0; steps > 0; ++i) {
    const Part t = part_of(p, c, steps);
    if (!f(t, c, i)) return;
    steps -= t.n;
    if (steps > 0) next_range<true>(p, c);
  }
}

// ---------------------------------------------------------------------------- loader
template <typename T, int D>
__device__ void load_role(const CrossParams& p, const Maps& maps, unsigned char* sm,
                          const Cursor& c0, int64_t steps, const Wait& wait, int& flags) {
  using L = Lay<D>;
  uint64_t* bars = wait.bars;
  const int lane = threadIdx.x & 31, R = p.box_keys;
  uint32_t use = 0;   // ring tiles issued
  uint32_t q_use[2] = {0, 0};
  const bool withhold = p.withhold_copy != 0;   // testing hook: the first K tile never comes
  each_part(p, c0, steps, [&](const Part& t, const Cursor& c, int) {
    const int PT = p.tile_pos / 2;
    for (int h = 0; h < t.halves; ++h) {
      if (q_use[h] > 0 &&
          !__all_sync(0xffffffffu, wait(kQEmpty + h, (q_use[h] - 1) & 1u)))
        return false;
      ++q_use[h];
      if (lane == 0) {
        tc::mbar_arrive_expect_tx(bars + kQFull + h, (uint32_t)(PT * p.G) * (D * 2));
#pragma unroll
        for (int x = 0; x < D / 64; ++x)
          tc::tma_load_3d(sm + L::kQ + h * L::kTile + x * L::kSub, &maps.q, x * 64, t.h * p.G,
                          t.row0 + h * PT, bars + kQFull + h);
      }
    }
    for (int j = c.s; j < c.s + t.n; ++j) {
      // R consecutive keys of a block to a lane (none when rows are copied one by one)
      const int key0 = j * kTileKeys + lane * max(R, 1);
      int row = 0;
      bool mapped = false;
      if (R > 0 && lane * R < kTileKeys && key0 < c.q.keys) {
        const int col = p.bs_shift >= 0 ? key0 >> p.bs_shift : key0 / p.BS;
        const int blk = __ldg(p.table + (int64_t)t.b * p.MB + col);
        mapped = blk >= 0 && blk < p.NB;
        if (mapped)
          row = blk * p.BS + (key0 - col * p.BS);
        else
          flags |= PKV_DEV_BAD_BLOCK;
      }
      const bool whole = mapped && key0 + R <= c.q.keys;
#pragma unroll 1
      for (int kv = 0; kv < 2; ++kv, ++use) {
        const uint32_t st = use % L::kStages, round = use / L::kStages;
        const bool ok = round == 0 || wait(kEmpty + (int)st, (round - 1) & 1u);
        if (!__all_sync(0xffffffffu, ok)) return false;
        unsigned char* dst = sm + L::kRing + st * L::kTile;
        uint64_t* full = bars + kFull + st;
        // keys behind the last one may stay what they are: their scores are masked
        const bool box = kv == 0 ? mapped : whole;
        const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, box));
        if (lane == 0) tc::mbar_arrive_expect_tx(full, boxes * R * (D * 2));
        __syncwarp();
        if (box && !(withhold && use == 0)) {
#pragma unroll
          for (int x = 0; x < D / 64; ++x)
            tc::tma_load_3d(dst + x * L::kSub + lane * R * 128, kv == 0 ? &maps.k : &maps.v, x * 64,
                            t.h, row, full);
        }
        const T* src = static_cast<const T*>(kv == 0 ? p.kc : p.vc);
        if (R == 0) {
          for (int r = 0; r < kTileKeys; ++r) {   // 2 or 4 rows would fit an instruction: rare path
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
              cp_async_16(dst + (lane >> 3) * L::kSub + tc::sw128(r, lane & 7),
                          at >= 0 ? src + at + lane * 8 : src, at >= 0 ? 16 : 0);
          }
        } else if (kv == 1) {
          uint32_t rest = __ballot_sync(0xffffffffu, lane * R < kTileKeys && !whole);
          for (; rest; rest &= rest - 1) {
            const int i = __ffs(rest) - 1;
            const int row_i = __shfl_sync(0xffffffffu, row, i);
            const int mapped_i = __shfl_sync(0xffffffffu, mapped ? 1 : 0, i);
            for (int x = lane; x < R * (D / 8); x += 32) {
              const int r = x / (D / 8), ch = x % (D / 8);
              const bool live = mapped_i && j * kTileKeys + i * R + r < c.q.keys;
              const int64_t at = live ? ((int64_t)(row_i + r) * p.Hkv + t.h) * D + ch * 8 : 0;
              cp_async_16(dst + (ch >> 3) * L::kSub + tc::sw128(i * R + r, ch & 7), src + at,
                          live ? 16 : 0);
            }
          }
        }
        arrive_copies(full);
      }
    }
    return true;
  });
  if (*wait.abort) {   // let what was issued land before the block ends
    const uint32_t n = use < (uint32_t)L::kStages ? use : (uint32_t)L::kStages;
    for (uint32_t k = 0; k < n; ++k) {
      const uint32_t u = use - 1 - k;
      tc::mbar_wait(bars + kFull + u % L::kStages, (u / L::kStages) & 1u, wait.tries);
    }
    for (int h = 0; h < 2; ++h)
      if (q_use[h] > 0) tc::mbar_wait(bars + kQFull + h, (q_use[h] - 1) & 1u, wait.tries);
  }
}

// ---------------------------------------------------------------------------- products
template <typename T, int D>
__device__ void mma_role(const CrossParams& p, unsigned char* sm, uint32_t tmem,
                         const Cursor& c0, int64_t steps, const Wait& wait) {
  using L = Lay<D>;
  uint64_t* bars = wait.bars;
  constexpr uint32_t fmt = Num<T>::kBf16 ? (1u << 7) | (1u << 10) : 0u;   // types of A and B
  constexpr uint32_t id_s = tc::idesc_f16(128, 128, false, false) | fmt;
  constexpr uint32_t id_o = tc::idesc_f16(128, D, false, true) | fmt;
  const uint32_t q_at = smem_u32(sm + L::kQ), ring = smem_u32(sm + L::kRing);
  uint32_t use = 0, q_use[2] = {0, 0}, p_use[2] = {0, 0};
  const auto scores = [&](int h, uint32_t st) {
    const uint32_t qa = q_at + h * L::kTile, ka = ring + st * L::kTile;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      const uint32_t off = (uint32_t)(ks >> 2) * L::kSub + (uint32_t)(ks & 3) * 32u;
      tc::mma_f16(tmem + h * 128, tc::smem_desc(qa + off, 16, 1024),
                  tc::smem_desc(ka + off, 16, 1024), id_s, ks > 0 ? 1u : 0u);
    }
    tc::commit(bars + kSFull + h);
  };
  const auto products = [&](int h, uint32_t st, bool first) {
    const uint32_t va = ring + st * L::kTile;
#pragma unroll
    for (int ks = 0; ks < 8; ++ks)
      mma_tmem_a(tmem + 256 + h * 128, tmem + h * 128 + (uint32_t)ks * 8u,
                 tc::smem_desc(va + (uint32_t)ks * 2048u, L::kSub, 1024), id_o,
                 first && ks == 0 ? 0u : 1u);
  };
  const auto full = [&](uint32_t u) {
    if (!wait(kFull + (int)(u % L::kStages), (u / L::kStages) & 1u)) return false;
    tc::fence_async_shared();   // rows written by cp.async
    return true;
  };
  each_part(p, c0, steps, [&](const Part& t, const Cursor&, int) {
    if (!full(use)) return false;                        // K of the first step
    for (int h = 0; h < t.halves; ++h) {
      if (!wait(kQFull + h, q_use[h]++ & 1u)) return false;
      tc::fence_after_sync();
      scores(h, use % L::kStages);
      if (t.n == 1) tc::commit(bars + kQEmpty + h);
    }
    tc::commit(bars + kEmpty + use % L::kStages);
    for (int j = 0; j < t.n; ++j) {
      const uint32_t v = use + 1, k = use + 2;           // V of step j, K of step j + 1
      const bool more = j + 1 < t.n;
      for (int h = 0; h < t.halves; ++h) {
        if (!wait(kPFull + h, p_use[h]++ & 1u)) return false;
        if (h == 0 && !full(v)) return false;
        tc::fence_after_sync();
        products(h, v % L::kStages, j == 0);
        if (h == t.halves - 1) tc::commit(bars + kEmpty + v % L::kStages);
        if (!more) {
          tc::commit(bars + kOFull + h);
          continue;
        }
        if (h == 0 && !full(k)) return false;
        scores(h, k % L::kStages);
        if (j + 2 == t.n) tc::commit(bars + kQEmpty + h);
        if (h == t.halves - 1) tc::commit(bars + kEmpty + k % L::kStages);
      }
      use += 2;
    }
    return true;
  });
  if (*wait.abort) {
    tc::commit(bars + kDrain);
    tc::mbar_wait(bars + kDrain, 0, wait.tries);
  }
}

// ---------------------------------------------------------------------------- softmax
template <typename T, int D>
__device__ void softmax_role(const CrossParams& p, uint32_t tmem, int half, int64_t unit,
                             const Cursor& c0, int64_t steps, const Wait& wait) {
  uint64_t* bars = wait.bars;
  const int r = threadIdx.x & 127, lane = r & 31;
  const uint32_t lane_at = tmem + ((uint32_t)(r & ~31) << 16);
  const uint32_t s_at = lane_at + half * 128, o_at = lane_at + 256 + half * 128;
  const float sl2 = p.scale_log2;
  const bool up = sl2 >= 0.f;   // a negative scale turns the maximum into a minimum
  const float hide = up ? -INFINITY : INFINITY;
  uint32_t s_use = 0, o_use = 0;
  each_part(p, c0, steps, [&](const Part& t, const Cursor& c, int index) {
    if (half >= t.halves) return true;
    const int pos = half * (p.tile_pos / 2) + r / p.G;
    const bool mine = r < (p.tile_pos / 2) * p.G && pos < t.pos;
    // lane covers keys [128 j + 4 lane, + 4): one block when its size is a multiple of 4
    const auto lookup = [&](int key) -> bool {
      if (key >= c.q.keys) return false;
      const int col = p.bs_shift >= 0 ? key >> p.bs_shift : key / p.BS;
      const int blk = __ldg(p.table + (int64_t)t.b * p.MB + col);
      return blk >= 0 && blk < p.NB;
    };
    bool page = lookup(c.s * kTileKeys + 4 * lane);
    float m = -INFINITY, l = 0.f;
    for (int j = c.s; j < c.s + t.n; ++j) {
      const int key0 = j * kTileKeys + 4 * lane;
      uint32_t words[4];   // key 4 i + x of the step is bit i of words[x]
      if (p.box_keys > 0) {
#pragma unroll
        for (int x = 0; x < 4; ++x)
          words[x] = __ballot_sync(0xffffffffu, page && key0 + x < c.q.keys);
        if (j + 1 < c.s + t.n) page = lookup(key0 + kTileKeys);
      } else {
#pragma unroll
        for (int x = 0; x < 4; ++x) words[x] = __ballot_sync(0xffffffffu, lookup(key0 + x));
      }
      // the loads and stores of TMEM below are the whole warp's
      if (!__all_sync(0xffffffffu, wait(kSFull + half, s_use & 1u))) return false;
      ++s_use;
      tc::fence_after_sync();
      float v[128];
      {
        float (*v32)[32] = reinterpret_cast<float (*)[32]>(v);
#pragma unroll
        for (int x = 0; x < 4; ++x) tc::tmem_ld32(s_at + x * 32, v32[x]);
        tc::tmem_wait_ld();
      }
      if ((words[0] & words[1] & words[2] & words[3]) != 0xffffffffu) {
#pragma unroll
        for (int x = 0; x < 128; ++x)
          v[x] = (words[x & 3] >> (x >> 2)) & 1u ? v[x] : hide;
      }
      float top;
      if (up) {
        float e[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) e[x] = fmaxf(v[2 * x], v[2 * x + 1]);
#pragma unroll
        for (int x = 8; x < 128; x += 8)
#pragma unroll
          for (int y = 0; y < 4; ++y) e[y] = max3(e[y], v[x + 2 * y], v[x + 2 * y + 1]);
        top = max3(e[0], e[1], fmaxf(e[2], e[3]));
      } else {
        top = v[0];
#pragma unroll
        for (int x = 1; x < 128; ++x) top = fminf(top, v[x]);
      }
      top *= sl2;   // -inf when nothing of the step is seen
      const bool first = m == -INFINITY;
      const bool raise = first ? top != -INFINITY : top > m + kRaise;
      const float alpha = raise && !first ? ex2(m - top) : 1.f;
      if (raise) m = top;
      const float base = m == -INFINITY ? 0.f : -m;
      if (__any_sync(0xffffffffu, alpha != 1.f) && j > c.s) {   // O is complete: see the order
#pragma unroll
        for (int x = 0; x < D / 32; ++x) {
          float o[32];
          tc::tmem_ld32(o_at + x * 32, o);
          tc::tmem_wait_ld();
#pragma unroll
          for (int y = 0; y < 32; ++y) o[y] *= alpha;
          tc::tmem_st32(o_at + x * 32, o);
        }
      }
      float la[4] = {0.f, 0.f, 0.f, 0.f}, lb[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        float w[32];   // 64 weights as pairs
#pragma unroll
        for (int x = 0; x < 64; x += 2) {
          float e0, e1;
          fma2(e0, e1, v[q * 64 + x], v[q * 64 + x + 1], sl2, base);
          e0 = ex2(e0);
          e1 = ex2(e1);
          add2(la[(x >> 1) & 3], lb[(x >> 1) & 3], e0, e1);
          w[x / 2] = __uint_as_float(Num<T>::pack(e0, e1));
        }
        tc::tmem_st32(s_at + q * 32, w);
      }
      l = l * alpha + (((la[0] + lb[0]) + (la[1] + lb[1])) + ((la[2] + lb[2]) + (la[3] + lb[3])));
      tc::tmem_wait_st();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) arrive(bars + kPFull + half);
    }
    if (!__all_sync(0xffffffffu, wait(kOFull + half, o_use & 1u))) return false;
    ++o_use;
    tc::fence_after_sync();
    if (t.whole) {
      const float inv = inverse_of(l);
      const int64_t row = (int64_t)(t.row0 + pos) * p.Hq + t.h * p.G + r % p.G;
      uint4* out = reinterpret_cast<uint4*>(static_cast<T*>(p.out) + row * D);
#pragma unroll
      for (int x = 0; x < D / 32; ++x) {
        float o[32];
        tc::tmem_ld32(o_at + x * 32, o);
        tc::tmem_wait_ld();
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
      const int64_t row = (2 * unit + (index == 0 ? 0 : 1)) * 256 + half * 128 + r;
      float4* out = reinterpret_cast<float4*>(p.tile_o + row * D);
#pragma unroll
      for (int x = 0; x < D / 32; ++x) {
        float o[32];
        tc::tmem_ld32(o_at + x * 32, o);
        tc::tmem_wait_ld();
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
  uint32_t* tmem_word = reinterpret_cast<uint32_t*>(sm + L::kBars + kTmemWord);
  if (tid == 0) {
    for (int i = 0; i < L::kStages; ++i) {
      tc::mbar_init(wait.bars + kFull + i, 33);
      tc::mbar_init(wait.bars + kEmpty + i, 1);
    }
    for (int h = 0; h < 2; ++h) {
      tc::mbar_init(wait.bars + kQFull + h, 1);
      tc::mbar_init(wait.bars + kQEmpty + h, 1);
      tc::mbar_init(wait.bars + kSFull + h, 1);
      tc::mbar_init(wait.bars + kPFull + h, 4);
      tc::mbar_init(wait.bars + kOFull + h, 1);
    }
    tc::mbar_init(wait.bars + kDrain, 1);
    tc::mbar_init_fence();
    *wait.abort = 0;
  }
  if (warp == 9 && lane == 0 && p.box_keys > 0) {
    tc::tma_prefetch_desc(&maps.q);
    tc::tma_prefetch_desc(&maps.k);
    tc::tma_prefetch_desc(&maps.v);
  }
  if (warp == 0) {
    tc::tmem_alloc(tmem_word, 512);
    tc::tmem_relinquish();
  }
  // the plan, in the ring's memory before the ring is used
  int64_t* pref = reinterpret_cast<int64_t*>(sm + L::kRing);
  int flags = 0;
  const Plan pl = make_plan<true, kThreads>(p, p.tile_units, kLeast, pref, pref + kEntries, &flags);
  flags = 0;   // the other kernel reports the sequences
  const int64_t unit = blockIdx.x, g0 = unit * pl.W;
  const int64_t steps = g0 < pl.total ? min(pl.total, g0 + pl.W) - g0 : 0;
  if (tid == 0) write_record<true>(p, pl, pref, unit, p.tile_rec);
  Cursor c{};
  if (steps > 0) c = locate<true>(p, pl, pref, g0);
  tc::fence_async_shared();
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_word;
  if (steps > 0) {
    if (warp < 8) {
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kSoftmaxRegs));
      softmax_role<T, D>(p, tmem, warp >> 2, unit, c, steps, wait);
    } else {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kOtherRegs));
      if (tid == 256)
        mma_role<T, D>(p, sm, tmem, c, steps, wait);
      else if (warp == 9)
        load_role<T, D>(p, maps, sm, c, steps, wait, flags);
    }
  }
  if (tid == 0 && *wait.abort) flags |= PKV_DEV_TIMEOUT;
  if (flags) flag_status(p.status, flags);
  cp_async_wait<0>();
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (tid == 0 && *wait.abort) flag_status(p.status, PKV_DEV_TIMEOUT);
  if (warp == 0) tc::tmem_dealloc(tmem, 512);
  // the join behind this kernel waits for it alone: it must not end before the one in front
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
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

// rows of heads of D elements, boxes of 64 elements x b1 x b2 in the 128-byte swizzle
bool encode(CUtensorMap* m, bool bf16, const void* base, int D, int64_t heads, int64_t rows,
            int b1, int b2) {
  const PFN_cuTensorMapEncodeTiled_v12000 fn = encoder();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)heads * D * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)b1, (cuuint32_t)b2};
  const cuuint32_t unit[3] = {1, 1, 1};
  return fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
            const_cast<void*>(base), dims, strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
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
  const int64_t rows = p.NB * p.BS;
  if (!encode(&maps.q, p.bf16, p.q, D, p.Hq, p.T, p.G, p.tile_pos / 2)) return cudaErrorInvalidValue;
  maps.k = maps.v = maps.q;   // not used without boxes
  if (p.box_keys > 0 && (!encode(&maps.k, p.bf16, p.kc, D, p.Hkv, rows, 1, p.box_keys) ||
                         !encode(&maps.v, p.bf16, p.vc, D, p.Hkv, rows, 1, p.box_keys)))
    return cudaErrorInvalidValue;
  // may start as blocks of the kernel in front end: it reads inputs and writes other rows
  ProfScope ps("cross_tiles", s);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.tile_units);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Lay<D>::kBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cross_tiles_kernel<T, D>, p, maps);
}

}  // namespace

cudaError_t launch_cross_tiles(const CrossParams& p, cudaStream_t s) {
  if (p.bf16)
    return p.D == 64 ? launch_typed<__nv_bfloat16, 64>(p, s) : launch_typed<__nv_bfloat16, 128>(p, s);
  return p.D == 64 ? launch_typed<__half, 64>(p, s) : launch_typed<__half, 128>(p, s);
}

}  // namespace pkv
