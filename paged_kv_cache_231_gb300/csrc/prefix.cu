// Causal attention of sequences that begin alike (pkv_paged_prefix_attention).
//
// Keys [0, S) of a group lie in the same blocks for all its sequences, and every row of them sees
// all of these. With s = scale <q, k> and e^x taken over either part,
//   out = (e^{lse_1} out_1 + e^{lse_2} out_2) / (e^{lse_1} + e^{lse_2}),
// where (out_1, lse_1) comes from the shared keys, computed once for the rows of the whole group
// (kShared: a group is a sequence of as many rows, no causal mask), and (out_2, lse_2) from a
// row's own keys j >= S (kCausal). The first goes to 32-bit arrays in the workspace, the second
// takes it in where it writes a row. So a group's S keys are read once and multiplied as matrices
// with all its rows, where every sequence for itself would read them again: 64 single tokens
// behind 8192 keys read 1/64 of that.
//
// This file: the plan, which finds how many keys each group can share, and the launches; the
// kShared form of cross.cu is at the end.
#define PKV_FORM kShared
#define PKV_LAUNCH(suffix) launch_shared##suffix
#include "cross.cu"

namespace pkv {
namespace {

constexpr int kPlanThreads = 256;

// A block takes the groups blockIdx.x, + gridDim.x, ... and writes group_cu, shared, table_row of
// each and `start` of its sequences (0: nothing shared).
__global__ void __launch_bounds__(kPlanThreads) prefix_plan_kernel(CrossParams p, PrefixParams x) {
  __shared__ int s_past, s_live, s_first, s_bad;
  const int tid = threadIdx.x;
  bool wrong = false;   // group offsets that descend or leave 0 .. B
  for (int g = tid; g < x.groups; g += kPlanThreads) {
    const int lo = __ldg(x.offsets + g), hi = __ldg(x.offsets + g + 1);
    wrong = wrong || lo < 0 || hi < lo || hi > p.B;
  }
  wrong = __syncthreads_or(wrong) != 0;
  if (wrong && blockIdx.x == 0 && tid == 0) flag_status(p.status, PKV_DEV_BAD_SEQUENCE);
  // sequences that lie in no group
  const int from = wrong || x.groups == 0 ? p.B : __ldg(x.offsets);
  const int to = wrong || x.groups == 0 ? p.B : __ldg(x.offsets + x.groups);
  for (int b = blockIdx.x * kPlanThreads + tid; b < p.B; b += gridDim.x * kPlanThreads)
    if (b < from || b >= to) x.start[b] = 0;
  for (int g = blockIdx.x; g < x.groups; g += gridDim.x) {
    const int lo = wrong ? 0 : __ldg(x.offsets + g), hi = wrong ? 0 : __ldg(x.offsets + g + 1);
    const int asked = __ldg(x.shared + g);
    if (tid == 0) {
      s_past = INT32_MAX;
      s_first = p.B;
      s_live = s_bad = 0;
      if (asked < 0) flag_status(p.status, PKV_DEV_BAD_SEQUENCE);
    }
    __syncthreads();
    int least = INT32_MAX, first = p.B, live = 0, bad = 0;
    for (int b = lo + tid; b < hi; b += kPlanThreads) {
      const int c0 = __ldg(p.cu + b), c1 = __ldg(p.cu + b + 1), past = __ldg(p.past + b);
      if (c0 < 0 || c1 < c0 || c1 > p.T || c1 - c0 > p.max_q || past < 0 || past > p.MB * p.BS) {
        bad = 1;
      } else if (c1 > c0) {
        least = min(least, past);
        first = min(first, b);
        ++live;
      }
    }
    least = __reduce_min_sync(0xffffffffu, least);
    first = __reduce_min_sync(0xffffffffu, first);
    live = __reduce_add_sync(0xffffffffu, live);
    bad = __reduce_or_sync(0xffffffffu, bad);
    if ((tid & 31) == 0) {
      atomicMin(&s_past, least);
      atomicMin(&s_first, first);
      atomicAdd(&s_live, live);
      atomicOr(&s_bad, bad);
    }
    __syncthreads();
    const int keys = s_bad || s_live < 2 ? 0 : min(max(asked, 0), s_past);
    for (int b = lo + tid; b < hi; b += kPlanThreads) x.start[b] = keys;
    if (tid == 0) {
      x.group_keys[g] = keys;
      x.group_cu[g] = wrong ? 0 : __ldg(p.cu + lo);
      if (g == x.groups - 1) x.group_cu[g + 1] = wrong ? 0 : __ldg(p.cu + hi);
      x.table_row[g] = keys > 0 ? s_first : 0;
    }
    __syncthreads();
  }
}

}  // namespace

size_t prefix_layout(CrossParams* shared, CrossParams* own, PrefixParams* x, char* base) {
  size_t off = 0;
  const auto take = [&](size_t bytes) {
    char* at = base ? base + off : nullptr;
    off += (bytes + 255) / 256 * 256;
    return at;
  };
  const size_t G = (size_t)x->groups, rows = (size_t)own->T * own->Hq;
  x->start = reinterpret_cast<int32_t*>(take((size_t)own->B * 4));
  x->group_cu = reinterpret_cast<int32_t*>(take((G + 1) * 4));
  x->group_keys = reinterpret_cast<int32_t*>(take(G * 4));
  x->table_row = reinterpret_cast<int32_t*>(take(G * 4));
  float* lse = reinterpret_cast<float*>(take(rows * 4));
  float* out = reinterpret_cast<float*>(take(rows * own->D * 4));
  *shared = *own;
  shared->B = x->groups;
  shared->cu = x->group_cu;
  shared->klen = x->group_keys;
  shared->table_row = x->table_row;
  shared->out = out;
  shared->lse = lse;
  shared->max_q = own->T;
  own->start = x->start;
  own->prior_o = out;
  own->prior_lse = lse;
  // one after the other, so both calls' pieces lie in the same place
  char* const at = base ? base + off : nullptr;
  const size_t a = G > 0 ? cross_layout(shared, at) : 0, b = cross_layout(own, at);
  return off + (a > b ? a : b);
}

cudaError_t launch_prefix(const CrossParams& shared, const CrossParams& own, const PrefixParams& x,
                          cudaStream_t s) {
  {
    ProfScope ps("prefix_plan", s);
    const int fit = 4 * device_sms(), most = x.groups > 1 ? x.groups : 1;
    prefix_plan_kernel<<<most < fit ? most : fit, kPlanThreads, 0, s>>>(own, x);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (x.groups > 0) {
    const cudaError_t e = launch_shared(shared, s);
    if (e != cudaSuccess) return e;
    return launch_causal(own, s);
  }
  CrossParams alone = own;   // nothing is shared: no prior results
  alone.prior_o = alone.prior_lse = nullptr;
  return launch_causal(alone, s);
}

}  // namespace pkv
