// Causal attention of sequences that begin alike (pkv_paged_prefix_attention).
//
// Keys [0, S) of a group lie in the same blocks for all its sequences, and every row of them sees
// all of these. With s = scale <q, k> and e^x taken over either part,
//   out = (e^{lse_1} out_1 + e^{lse_2} out_2) / (e^{lse_1} + e^{lse_2}),
// where (out_1, lse_1) comes from the shared keys, computed once for the rows of the whole group
// (kShared: a group is a sequence of as many rows, no causal mask), and (out_2, lse_2) from a
// row's own keys j >= S (kCausal). The first goes to 32-bit arrays in the workspace, the second
// takes it in where it writes a row. Single tokens with few keys of their own go beside the first:
// both parts go to the workspace, and the join behind them writes the rows. So a group's S keys are read once and multiplied as matrices
// with all its rows, where every sequence for itself would read them again: 64 single tokens
// behind 8192 keys read 1/64 of that.
// Where that saves less than it costs (few sequences or short prefixes, which the cache holds
// for those that read them again; prompts that fill tiles by themselves) nothing is shared.
//
// This file: the plan, which finds how many keys each group can share, and the launches; the
// kShared form of cross.cu is at the end.
#define PKV_FORM kShared
#define PKV_LAUNCH(suffix) launch_shared##suffix
#include "cross.cu"

namespace pkv {
namespace {

constexpr int kPlanThreads = 1024, kPlanWarps = kPlanThreads / 32;

// What sharing saves, in nanoseconds. A sequence of few rows reads all of its keys, from the cache
// where others read the same (64 single tokens over the same 8192 keys: 7.3 TB/s); one of many rows
// takes half a tile's step for each 128 rows and keys. Shared, a group's rows fill tiles together,
// and their result makes a way through memory. The kernels of the shared keys cost a call some 30 us,
// 24 us where the kernel for few and short sequences runs beside them (saved by this count, shared,
// alone: 32 tokens behind 1024 keys 17.7, 30.5, 28.2 us, behind 2048 35.6, 32.0, 44.2 us; 64 behind 512 17.4,
// 34.3, 36.2 us; with 16 heads of 64 32 behind 1024 17.8, 31.6, 31.6 us, 8 behind 8192 32.7, 35.8, 46.1 us).
// A call that looks and finds nothing has paid for kLookCost of that (8 to 12 us), so what is saved weighs
// against the rest of what the path that would run costs. Saved, shared, not shared though looked at: 64
// behind 512 keys 17.4, 34.3, 48.8 us; 32 behind 768 with 3000 keys of their own one of them (an even share
// for every warp) 13.2, 46.1, 41.3 us; 16 drafts of 8 tokens behind 4096 19.8, 65.4, 72.9 us; 16 prompts of up
// to 100 behind 8192 25.6, 151.5, 173.3 us.
constexpr int64_t kCallCost = 30000, kBesideCost = 24000, kLookCost = 11000;
// Of the tiles: plan, first steps, pieces. Of a block of the kernel for few and short sequences beside
// them, and what each step of a sequence (few_keys) adds.
constexpr int64_t kTilesFirst = 15000, kBlockFirst = 4200, kBlockStep = 200;
__device__ __forceinline__ int64_t few_cost(const CrossParams& p, int64_t keys) {
  return keys * p.Hkv * p.D * 4 / 7300;
}
__device__ __forceinline__ int64_t tile_cost(const CrossParams& p, int sms, int rows, int keys) {
  const int half = p.tile_pos / 2;
  const int64_t steps = (int64_t)((rows + half - 1) / half) * ((keys + kTileKeys - 1) / kTileKeys);
  return steps * p.Hkv * (p.D == 64 ? 600 : 1030) / sms;
}

// One block. A warp looks at a group: how many keys it can share, and what that saves. If all of
// them together save more than the call costs, group_cu, group_keys, table_row of each group and
// `start` of its sequences say what is shared; else nothing is.
__global__ void __launch_bounds__(kPlanThreads) prefix_plan_kernel(CrossParams p, PrefixParams x) {
  __shared__ unsigned long long s_saved, s_steps, s_tiles, s_best;
  __shared__ int s_longest;
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // the least that sharing costs: whether single tokens' own keys go beside it is known further down
  const int64_t cost = (x.choice ? kBesideCost : kCallCost) - kLookCost;
  bool wrong = false;   // group offsets that descend or leave 0 .. B
  for (int g = tid; g < x.groups; g += kPlanThreads) {
    const int lo = __ldg(x.offsets + g), hi = __ldg(x.offsets + g + 1);
    wrong = wrong || lo < 0 || hi < lo || hi > p.B;
  }
  if (tid == 0) {
    s_saved = s_steps = s_tiles = 0;
    s_best = ~0ull;
    s_longest = 0;
  }
  wrong = __syncthreads_or(wrong) != 0;
  int flags = wrong ? PKV_DEV_BAD_SEQUENCE : 0;
  for (int g = warp; g < x.groups; g += kPlanWarps) {
    const int lo = wrong ? 0 : __ldg(x.offsets + g), hi = wrong ? 0 : __ldg(x.offsets + g + 1);
    const int asked = __ldg(x.shared + g);
    if (asked < 0) flags |= PKV_DEV_BAD_SEQUENCE;
    int least = INT32_MAX, first = p.B, live = 0, rows = 0;
    bool bad = false;
    for (int b = lo + lane; b < hi; b += 32) {
      const int c0 = __ldg(p.cu + b), c1 = __ldg(p.cu + b + 1), past = __ldg(p.past + b);
      if (c0 < 0 || c1 < c0 || c1 > p.T || c1 - c0 > p.max_q || past < 0 || past > p.MB * p.BS) {
        bad = true;
      } else if (c1 > c0) {
        least = min(least, past);
        first = min(first, b);
        rows += c1 - c0;
        ++live;
      }
    }
    least = __reduce_min_sync(0xffffffffu, least);
    first = __reduce_min_sync(0xffffffffu, first);
    live = __reduce_add_sync(0xffffffffu, live);
    rows = __reduce_add_sync(0xffffffffu, rows);
    bad = __any_sync(0xffffffffu, bad);
    int keys = bad || live < 2 ? 0 : min(max(asked, 0), least);
    int64_t saved = 0;
    if (keys > 0) {
      for (int b = lo + lane; b < hi; b += 32) {
        const int n = __ldg(p.cu + b + 1) - __ldg(p.cu + b);
        if (n > 0) saved += n > p.few ? tile_cost(p, x.sms, n, keys) : few_cost(p, keys);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) saved += __shfl_xor_sync(0xffffffffu, saved, o);
      const int64_t tiles = tile_cost(p, x.sms, rows, keys);
      saved -= tiles + (int64_t)rows * p.Hq * p.D * 8 / 4000;
      if (saved <= 0 && !x.always) keys = 0;
      if (lane == 0 && keys > 0) atomicAdd(&s_tiles, (unsigned long long)tiles);
    }
    if (lane == 0) {
      if (keys > 0) atomicAdd(&s_saved, (unsigned long long)(x.always ? cost + 1 : saved));
      x.group_keys[g] = keys;
      x.group_cu[g] = wrong ? 0 : __ldg(p.cu + lo);
      if (g == x.groups - 1) x.group_cu[g + 1] = wrong ? 0 : __ldg(p.cu + hi);
      x.table_row[g] = keys > 0 ? first : 0;
    }
  }
  if (flags) flag_status(p.status, flags);
  const int from = wrong || x.groups == 0 ? p.B : __ldg(x.offsets);
  const int to = wrong || x.groups == 0 ? p.B : __ldg(x.offsets + x.groups);
  for (int b = tid; b < p.B; b += kPlanThreads)   // sequences that lie in no group
    if (b < from || b >= to) x.start[b] = 0;
  __syncthreads();
  bool share = (int64_t)s_saved > cost, small = false;
  const int step = few_keys(p.D), shift = 31 - __clz(step);   // a power of two
#pragma unroll 1   // once, or once more where that turns out to save less than it costs
  for (;;) {
    // what is shared of each sequence, and of its own keys the steps of the kernel for few rows
    int64_t steps = 0;
    int longest = 0;
    const auto own = [&](int b, int start) {
      const int64_t n = (int64_t)__ldg(p.past + b) + __ldg(p.cu + b + 1) - __ldg(p.cu + b) - start;
      const int k = (int)min(max((n + step - 1) >> shift, (int64_t)0), (int64_t)p.MB * p.BS);
      steps += k;
      longest = max(longest, k);
    };
    for (int g = warp; g < x.groups; g += kPlanWarps) {
      const int lo = wrong ? 0 : __ldg(x.offsets + g), hi = wrong ? 0 : __ldg(x.offsets + g + 1);
      const int keys = share ? __ldcg(x.group_keys + g) : 0;
      for (int b = lo + lane; b < hi; b += 32) {
        x.start[b] = keys;
        own(b, keys);
      }
    }
    for (int b = tid; b < p.B; b += kPlanThreads)
      if (b < from || b >= to) own(b, 0);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) steps += __shfl_xor_sync(0xffffffffu, steps, o);
    longest = __reduce_max_sync(0xffffffffu, longest);
    if (lane == 0) {
      atomicAdd(&s_steps, (unsigned long long)steps);
      atomicMax(&s_longest, longest);
    }
    __syncthreads();
    if (!x.choice) break;
    // The kernel for few and short sequences, or an even share of the steps for every warp and a join:
    // in units of a step of 0.85 us, the longest sequence's share of a warp and 3.5 for every wave of
    // blocks behind the first, or the even share and 15 for its plan and the join (64 tokens behind 8192
    // shared keys and up to 64, 256, 512, 1024 of their own: 42.5, 47.9, 56.4 and 67.6 us, or 64.8, 70.6,
    // 81.8 and 95.8 us; behind the tiles instead of beside them the first took 52.8, 60.5, 70.0 and 79.6 us).
    // (n <= 2 * floor(s / m), without the division of 64 bits)
    const int waves = (p.B * p.Hkv + x.sms - 1) / x.sms;   // at most 4
    const int64_t n = (int64_t)(s_longest + 7) / 8 * 2 + 7 * (waves - 1) - 30;
    small = n <= 0 || (n + 1) / 2 * (8 * x.sms) <= (int64_t)s_steps * p.Hkv;
    if (!share || small || x.always || (int64_t)s_saved > kCallCost - kLookCost) break;
    share = false;   // these kernels would follow one another, and cost more
    __syncthreads();
    if (tid == 0) s_steps = s_longest = 0;
    __syncthreads();
  }
  if (tid == 0) *x.active = share ? 1 : 0;
  if (!x.choice) return;
  if (tid == 0) *x.choice = small;
  // The kernel for few and short sequences runs beside the tiles: on the SMs that these leave free
  // and, as they end, on theirs. The tiles take `at` ns on n SMs, the other kernel's blocks `all` on
  // one; the n for which both are done first (64 tokens behind 8192 shared keys and up to 256,
  // 512 of their own: on 16, 48, 76, 104 and 152 SMs 77.5, 49.0, 49.0, 55.2 and 61.1 us, or 86.7, 53.7,
  // 63.2, 64.8 and 70.4 us).
  const int64_t all = ((int64_t)p.B * kBlockFirst + (int64_t)s_steps * kBlockStep) * p.Hkv;
  for (int n = tid + 1; n <= x.units_most; n += kPlanThreads) {
    const int64_t at = kTilesFirst + (int64_t)s_tiles * x.sms / n;
    const int64_t end = max(at, (all + n * at) / x.sms);
    atomicMin(&s_best, (unsigned long long)end << 16 | (unsigned)n);
  }
  __syncthreads();
  if (tid == 0) *x.units = small ? (int)(s_best & 0xffff) : x.units_most;
}

}  // namespace

// What the rows may cost at most, one by one (see prefix_plan_kernel).
static double most_alone(const CrossParams& p, int sms) {
  const double keys = (double)p.MB * p.BS, seqs = p.T < p.B ? p.T : p.B;
  double ns = seqs * keys * p.Hkv * p.D * 4 / 7300;
  if (p.max_q > p.few)
    ns += ((double)p.T / (p.tile_pos / 2) + seqs) * (keys / kTileKeys + 1) * p.Hkv *
          (p.D == 64 ? 600 : 1030) / sms;
  return ns;
}

size_t prefix_layout(CrossParams* shared, CrossParams* own, PrefixParams* x, char* base) {
  size_t off = 0;
  const auto take = [&](size_t bytes) {
    char* at = base ? base + off : nullptr;
    off += (bytes + 255) / 256 * 256;
    return at;
  };
  x->sms = device_sms();
  own->few = 16 / own->G;
  own->tile_pos = 2 * (128 / own->G);
  const int hook = testing_prefix_sharing();
  x->always = hook == 1;
  if (x->groups == 0 || hook == 2 || (hook == 0 && most_alone(*own, x->sms) <=
                                               (own->max_q <= own->few ? kBesideCost : kCallCost))) {
    own->check_offsets = x->offsets;
    own->check_shared = x->shared;
    own->check_groups = x->groups;
    x->start = nullptr;
    return cross_layout(own, base);
  }
  static const int32_t some = 0;   // sizes alone are asked for: any address
  const size_t G = (size_t)x->groups, rows = (size_t)own->T * own->Hq;
  x->start = reinterpret_cast<int32_t*>(take((size_t)own->B * 4));
  x->group_cu = reinterpret_cast<int32_t*>(take((G + 1) * 4));
  x->group_keys = reinterpret_cast<int32_t*>(take(G * 4));
  x->table_row = reinterpret_cast<int32_t*>(take(G * 4));
  x->active = reinterpret_cast<int32_t*>(take(4));
  x->choice = reinterpret_cast<int32_t*>(take(4));
  x->units = reinterpret_cast<int32_t*>(take(4));
  float* lse = reinterpret_cast<float*>(take(rows * 4));
  float* out = reinterpret_cast<float*>(take(rows * own->D * 4));
  if (own->max_q <= own->few) {   // single tokens
    own->apart_o = reinterpret_cast<float*>(take(rows * own->D * 4));
    own->apart_ml = reinterpret_cast<float2*>(take(rows * 8));
  }
  *shared = *own;
  shared->B = x->groups;
  shared->cu = x->group_cu;
  shared->klen = x->group_keys;
  shared->table_row = x->table_row;
  shared->active = x->active;
  shared->out = out;
  shared->lse = lse;
  shared->max_q = own->T;
  own->start = x->start;
  own->prior_o = out;
  own->prior_lse = lse;
  if (own->max_q <= own->few) own->choice = base ? x->choice : &some;
  // apart: the second call's kernels begin while the first one's pieces are still joined
  const size_t a = cross_layout(shared, base ? base + off : nullptr, true);
  const size_t b = cross_layout(own, base ? base + off + a : nullptr);
  if (!own->small) own->choice = nullptr;   // too many sequences for the one kernel
  if (!own->choice) {
    x->choice = nullptr;
    own->apart_o = nullptr;
  } else {
    shared->units = x->units;
  }
  x->units_most = shared->tile_units;
  return off + a + b;
}

cudaError_t launch_prefix(const CrossParams& shared, const CrossParams& own, const PrefixParams& x,
                          cudaStream_t s) {
  if (!x.start) return launch_causal(own, s);
  {
    ProfScope ps("prefix_plan", s);
    prefix_plan_kernel<<<1, kPlanThreads, 0, s>>>(own, x);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (!own.choice) {
    const cudaError_t e = launch_shared(shared, s);
    return e == cudaSuccess ? launch_causal(own, s) : e;
  }
  cudaError_t e = launch_shared(shared, s, kTilesPart);
  if (e == cudaSuccess) e = launch_causal(own, s, kSmallPart);
  if (e == cudaSuccess) e = launch_shared(shared, s, kRestPart);
  return e == cudaSuccess ? launch_causal(own, s, kRestPart) : e;
}

}  // namespace pkv
