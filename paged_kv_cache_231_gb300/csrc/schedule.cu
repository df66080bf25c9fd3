// Block tables, slot maps and cumulative lengths from request lengths (pkv_paged_schedule).
//
// With past p_b and new n_b, row b holds h_b = ceil(p_b / BS) blocks and asks for
//   a_b = ceil((p_b + n_b) / BS) - h_b,   A_b = a_0 + ... + a_b;
// free blocks are the ids that no row holds, and the r-th block asked for (r from 0) is the
// r-th free id, so row b takes ranks [A_b - a_b, A_b). Row b is granted when a_b = 0 or
// A_b <= F (F free blocks), and the granted tokens up to it fit the token buffers; both
// conditions are prefix sums. Token i of row b (cu_b <= i < cu_{b+1}) has position
// p_b + i - cu_b and slot table[b][pos / BS] * BS + pos % BS.
//
// One cluster of C blocks, no workspace. Every block marks the held entries that
// it reads in a bitmap of the whole pool in its own shared memory (local atomics); group g of
// 1024 ids belongs to block g % C, which joins the C bitmaps of the group through distributed
// shared memory and hands its count of free ids to all. Each block then scans the rows for
// itself (cheaper than passing the sums around), writes the new table entries of its groups
// and, after a cluster barrier, the slots of its share of the tokens.
// Very many tokens' slots are left to a second kernel on all SMs.
// What bounds it is latency, phase behind phase: 2 rows take 6.0 us (9700 cycles of scans and
// barriers), 64 rows of up to 8192 tokens 10.7 us (19 100: marking 4000, new entries and the barrier
// behind them 6000), 16 rows of which half take in up to 2048 tokens 13.9 us (24 900: new entries
// 13 800, as a lane writes those of its 32 ids one after the other); with 2048 rows, 433 000 held
// entries and 325 000 new tokens (27.2 us) the marking takes 18 400 of 42 900 cycles.
#include <cooperative_groups.h>

#include "device_common.cuh"
#include "internal.h"
#include "step_ops.h"

namespace pkv {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kChunk = 128;   // table columns of a row that a warp marks as one piece
constexpr unsigned kMaxCluster = 16;
constexpr int kUnits = 4;     // such pieces whose loads are under way at once
constexpr int kTokens = 8;    // tokens of a thread
// Tokens from which their slots are a kernel of their own, on all SMs: 487 000 tokens of 2048 rows
// 23.6 us, with the cluster's blocks 32.9 us; 61 000 tokens 16.1 and 16.4 us, 31 000 16.4 and 15.5.
constexpr int kApartFrom = 65536;
static_assert(kScheduleMaxBlocks / 1024 <= kThreads, "a thread a group");

struct Row {
  int past, held, tokens, asked, flags;
};

__device__ __forceinline__ int blocks_for(const ScheduleParams& p, int tokens) {
  if (tokens <= 0) return 0;
  return (p.bs_shift >= 0 ? (tokens - 1) >> p.bs_shift : (tokens - 1) / p.BS) + 1;
}

__device__ __forceinline__ int column(const ScheduleParams& p, int pos) {
  return p.bs_shift >= 0 ? pos >> p.bs_shift : pos / p.BS;
}

__device__ __forceinline__ Row read_row(const ScheduleParams& p, int b) {
  Row r;
  r.past = __ldg(p.past + b);
  r.tokens = __ldg(p.fresh + b);
  r.flags = 0;
  const int limit = p.MB * p.BS;   // below 2^31, checked on the host
  if (r.past < 0 || r.tokens < 0) {
    r.flags = PKV_DEV_BAD_SEQUENCE;
    r.tokens = 0;
  }
  if (r.past > limit || r.tokens > limit - max(r.past, 0)) {
    r.flags |= PKV_DEV_BAD_BLOCK;
    r.tokens = 0;
  }
  r.held = min(blocks_for(p, r.past), p.MB);
  r.asked = r.tokens > 0 ? blocks_for(p, r.past + r.tokens) - r.held : 0;
  return r;
}

// Inclusive sum over the block's threads; *total gets the sum of all. scratch: kWarps words that
// neither the call before nor the one behind uses.
template <typename T>
__device__ __forceinline__ T block_sum(T v, T* total, T* scratch) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  if (lane == 31) scratch[w] = v;
  __syncthreads();
  T upto = scratch[lane];   // every warp sums the warps' sums for itself
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  *total = __shfl_sync(0xffffffffu, upto, kWarps - 1);
  const T before = __shfl_sync(0xffffffffu, upto, w > 0 ? w - 1 : 0);
  return w > 0 ? v + before : v;
}

// first index i of the ascending a[0, n) with a[i] > x (n when there is none)
__device__ __forceinline__ int first_above(const int* a, int n, int x) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] > x)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

// Slots and positions of many tokens, kTokens to a thread from `from` on and every further
// `stride`: the first one's row by a search in cu (shared memory), its block and the next one ahead
// of the rest. Returns what is wrong.
__device__ __forceinline__ int many_slots(const ScheduleParams& p, const int* cu, int granted,
                                          int64_t from, int64_t stride) {
  int flags = 0;
  const bool wide = ((reinterpret_cast<uintptr_t>(p.slots) |
                      reinterpret_cast<uintptr_t>(p.positions)) & 15u) == 0;
  for (int64_t i0 = from; i0 < p.T; i0 += stride) {
    int slot[kTokens], pos[kTokens];
#pragma unroll
    for (int k = 0; k < kTokens; ++k) slot[k] = pos[k] = -1;
    if (i0 < granted) {
      int b = first_above(cu + 1, p.B, (int)i0);
      const int pos0 = __ldg(p.past + b) + (int)i0 - cu[b], col0 = column(p, pos0);
      const int32_t* entry = p.table + (int64_t)b * p.MB + col0;
      const int id0 = __ldcg(entry), id1 = col0 + 1 < p.MB ? __ldcg(entry + 1) : -1;
      const int last = column(p, pos0 + kTokens - 1);
      if (i0 + kTokens <= cu[b + 1] && last <= col0 + 1 && id0 >= 0 && id0 < p.NB &&
          (last == col0 || (id1 >= 0 && id1 < p.NB))) {   // one row, at most two blocks
        const int turn = (col0 + 1) * p.BS - pos0;          // tokens of the first block
        const int base0 = id0 * p.BS + (pos0 - col0 * p.BS), base1 = id1 * p.BS - turn;
#pragma unroll
        for (int k = 0; k < kTokens; ++k) {
          pos[k] = pos0 + k;
          slot[k] = (k < turn ? base0 : base1) + k;
        }
      } else {
        int id[kTokens];   // all the blocks at once: the loads are what takes time
#pragma unroll
        for (int k = 0; k < kTokens; ++k) {
          id[k] = 0;
          if (i0 + k >= granted) continue;
          while (cu[b + 1] <= i0 + k) ++b;
          pos[k] = __ldg(p.past + b) + (int)(i0 + k) - cu[b];
          id[k] = __ldcg(p.table + (int64_t)b * p.MB + column(p, pos[k]));
        }
#pragma unroll
        for (int k = 0; k < kTokens; ++k) {
          if (i0 + k >= granted) continue;
          if (id[k] >= 0 && id[k] < p.NB)
            slot[k] = id[k] * p.BS + (pos[k] - column(p, pos[k]) * p.BS);
          else
            flags |= PKV_DEV_BAD_BLOCK;
        }
      }
    }
    if (wide && i0 + kTokens <= p.T) {
#pragma unroll
      for (int k = 0; k < kTokens; k += 4) {
        if (p.slots)
          *reinterpret_cast<int4*>(p.slots + i0 + k) =
              make_int4(slot[k], slot[k + 1], slot[k + 2], slot[k + 3]);
        if (p.positions)
          *reinterpret_cast<int4*>(p.positions + i0 + k) =
              make_int4(pos[k], pos[k + 1], pos[k + 2], pos[k + 3]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < kTokens; ++k) {
        if (i0 + k >= p.T) break;
        if (p.slots) p.slots[i0 + k] = slot[k];
        if (p.positions) p.positions[i0 + k] = pos[k];
      }
    }
  }
  return flags;
}

__global__ void __launch_bounds__(kThreads) schedule_kernel(ScheduleParams p) {
  extern __shared__ __align__(16) int smem[];
  __shared__ int s_asked[2][kWarps], s_groups[kWarps];   // one of two: see block_sum
  __shared__ int64_t s_tokens[2][kWarps];
  __shared__ int s_used, s_last;
  int* upto = smem;                  // [B] A_b
  int* cu = upto + p.B;              // [B + 1]
  int* gfree = cu + p.B + 1;         // [groups] free ids of a group, then those before it
  uint32_t* bits = reinterpret_cast<uint32_t*>(gfree + p.groups);   // [groups * 32]

  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int flags = 0;

  for (int i = tid; i < p.groups * 32; i += kThreads) bits[i] = 0u;
  if (tid == 0) s_used = s_last = cu[0] = 0;
  int asked_all = 0;
#pragma unroll 1
  for (int c0 = 0; c0 < p.B; c0 += kThreads) {
    const int b = c0 + tid;
    int asked = 0;
    if (b < p.B) {
      const Row r = read_row(p, b);
      asked = r.asked;
      cu[b + 1] = r.held;            // for the marking pass below
      flags |= r.flags;
    }
    int total;
    const int a = block_sum<int>(asked, &total, s_asked[(c0 / kThreads) & 1]);
    if (b < p.B) upto[b] = asked_all + a;
    asked_all += total;
  }
  __syncthreads();

  // mark the held entries, a warp kUnits pieces of a row at a time
  const int chunks = (p.MB + kChunk - 1) / kChunk, units = p.B * chunks;
  const int apart = C * kWarps;
  for (int u0 = rank + C * warp; u0 < units; u0 += apart * kUnits) {
    int id[kUnits][kChunk / 32];
#pragma unroll
    for (int x = 0; x < kUnits; ++x) {
      const int u = u0 + x * apart, b = u / chunks, c0 = (u - b * chunks) * kChunk;
      const int held = u < units ? cu[b + 1] : 0;
      const int32_t* row = p.table + (int64_t)b * p.MB;
#pragma unroll
      for (int k = 0; k < kChunk / 32; ++k) {
        const int c = c0 + k * 32 + lane;
        id[x][k] = c < held ? __ldcg(row + c) : -1;
      }
    }
#pragma unroll
    for (int x = 0; x < kUnits; ++x)
#pragma unroll
      for (int k = 0; k < kChunk / 32; ++k) {
        const int v = id[x][k];
        if (v >= 0 && v < p.NB)
          atomicOr(bits + (v >> 5), 1u << (v & 31));
        else if (v != -1)
          flags |= PKV_DEV_BAD_BLOCK;
      }
  }
  cluster.sync();

  // join the bitmaps of the groups that this block owns; free ids become set bits
  for (int g = rank + C * warp; g < p.groups; g += C * kWarps) {
    uint32_t used = 0u;
    for (int r0 = 0; r0 < C; r0 += 8)   // loads of 8 blocks' memory under way at once
#pragma unroll
      for (int r = r0; r < r0 + 8; ++r)
        if (r < C) used |= cluster.map_shared_rank(bits, r)[g * 32 + lane];
    const int first = g * 1024 + lane * 32;
    uint32_t open = ~used;
    if (first + 32 > p.NB) open &= first < p.NB ? (1u << (p.NB - first)) - 1u : 0u;
    const int n = __reduce_add_sync(0xffffffffu, __popc(open));
    bits[g * 32 + lane] = open;   // only the owner reads its copy of the group
    if (lane < C) cluster.map_shared_rank(gfree, lane)[g] = n;
  }
  cluster.sync();

  int free_ids;
  {   // at most 1024 groups
    const int n = tid < p.groups ? gfree[tid] : 0;
    const int upto_g = block_sum<int>(n, &free_ids, s_groups);
    if (tid < p.groups) gfree[tid] = upto_g - n;
  }
  // which rows are granted
  int64_t tokens = 0;
#pragma unroll 1
  for (int c0 = 0; c0 < p.B; c0 += kThreads) {
    const int b = c0 + tid;
    int want = 0, asked = 0, given = 0;
    if (b < p.B) {
      const Row r = read_row(p, b);
      want = r.tokens;
      asked = r.asked;
      given = asked == 0 || upto[b] <= free_ids ? want : 0;
    }
    int64_t total;
    const int64_t upto_t =
        tokens + block_sum<int64_t>(given, &total, s_tokens[(c0 / kThreads) & 1]);
    tokens += total;
    const bool fits = upto_t <= p.T;
    if (b < p.B) cu[b + 1] = fits ? (int)upto_t : -1;
    if (want > 0 && given == 0) flags |= PKV_DEV_NO_BLOCKS;
    if (given > 0 && !fits) flags |= PKV_DEV_BAD_SEQUENCE;
    const int last = __reduce_max_sync(0xffffffffu, fits ? (int)upto_t : 0);
    const int used = __reduce_add_sync(0xffffffffu, given > 0 && fits ? asked : 0);
    if (lane == 0) {
      atomicMax(&s_last, last);
      atomicAdd(&s_used, used);
    }
  }
  __syncthreads();
  for (int b = tid; b < p.B; b += kThreads)
    if (cu[b + 1] < 0) cu[b + 1] = s_last;   // behind the last row that fits
  __syncthreads();

  // new table entries: the free ids of this block's groups, by rank
  asked_all = min(asked_all, free_ids);
  for (int g = rank + C * warp; g < p.groups; g += C * kWarps) {
    if (gfree[g] >= asked_all) break;   // ranks only grow
    uint32_t open = bits[g * 32 + lane];
    const int n = __popc(open);
    int x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    int r = gfree[g] + x - n;
    int b = open && r < asked_all ? first_above(upto, p.B, r) : 0;
    for (; open && r < asked_all; open &= open - 1, ++r) {
      while (upto[b] <= r) ++b;
      if (cu[b + 1] > cu[b]) {
        const int nth = r - (b > 0 ? upto[b - 1] : 0);
        const int held = blocks_for(p, __ldg(p.past + b));
        p.table[(int64_t)b * p.MB + held + nth] = g * 1024 + lane * 32 + __ffs(open) - 1;
      }
    }
  }
  cluster.sync();   // every block sees the entries written above

  if (rank == C - 1) {
    for (int b = tid; b <= p.B; b += kThreads) p.cu[b] = cu[b];
    if (p.total)
      for (int b = tid; b < p.B; b += kThreads) p.total[b] = p.past[b] + cu[b + 1] - cu[b];
    if (p.free_out && tid == 0) *p.free_out = free_ids - s_used;
  }

  const int granted = cu[p.B];
  if (p.T <= C * kThreads) {   // few tokens: one to a thread
    const int i = tid * C + rank;   // spread over the blocks
    if (i < p.T && (p.slots || p.positions)) {
      int slot = -1, pos = -1;
      if (i < granted) {
        const int b = first_above(cu + 1, p.B, i);
        pos = __ldg(p.past + b) + i - cu[b];
        const int col = column(p, pos), id = __ldcg(p.table + (int64_t)b * p.MB + col);
        if (id >= 0 && id < p.NB)
          slot = id * p.BS + (pos - col * p.BS);
        else
          flags |= PKV_DEV_BAD_BLOCK;
      }
      if (p.slots) p.slots[i] = slot;
      if (p.positions) p.positions[i] = pos;
    }
    if (flags) flag_status(p.status, flags);
    return;
  }
  const int64_t stride = (int64_t)C * kThreads * kTokens;
  const int at = p.T <= stride ? tid * C + rank : rank * kThreads + tid;   // one round: spread
  if (!p.apart && (p.slots || p.positions))
    flags |= many_slots(p, cu, granted, (int64_t)at * kTokens, stride);
  if (flags) flag_status(p.status, flags);
}

// The slots of very many tokens, on all SMs, behind the kernel above.
constexpr int kSlotThreads = 512;
__global__ void __launch_bounds__(kSlotThreads) schedule_slots_kernel(ScheduleParams p) {
  extern __shared__ __align__(16) int smem[];
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  for (int b = threadIdx.x; b <= p.B; b += kSlotThreads) smem[b] = __ldcg(p.cu + b);
  __syncthreads();
  const int64_t at = (int64_t)blockIdx.x * kSlotThreads + threadIdx.x;
  const int flags =
      many_slots(p, smem, smem[p.B], at * kTokens, (int64_t)gridDim.x * kSlotThreads * kTokens);
  if (flags) flag_status(p.status, flags);
}

size_t schedule_smem(const ScheduleParams& p) {
  return sizeof(int) * ((size_t)2 * p.B + 1 + (size_t)p.groups * 33);
}
constexpr size_t kMaxSmem =
    sizeof(int) * ((size_t)2 * kScheduleMaxBatch + 1 + (size_t)(kScheduleMaxBlocks / 1024) * 33);
static_assert(kMaxSmem <= 230000, "schedule shared memory over the limit");

}  // namespace

cudaError_t launch_schedule(const ScheduleParams& p, cudaStream_t s) {
  static std::atomic<uint64_t> configured{0}, wide{0};   // wide: the device takes clusters of 16
  int dev = -1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kMaxCluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (needs_configure(configured, &dev)) {
    cudaError_t e = cudaFuncSetAttribute(
        schedule_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxSmem);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(schedule_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(kMaxCluster);
    cfg.dynamicSmemBytes = kMaxSmem;
    int clusters = 0;
    if (cudaOccupancyMaxActiveClusters(&clusters, schedule_kernel, &cfg) == cudaSuccess &&
        clusters > 0)
      mark_configured(wide, dev);
    else
      (void)cudaGetLastError();
    mark_configured(configured, dev);
  }
  // Blocks of the cluster: 16 where many entries or tokens are to be gone through (2048 rows of
  // 600 entries and 325 000 tokens, their slots included: 52 us with 8, 33 us with 16), else 8 (64
  // rows of 520 entries: 10.6 us with 8, 13.9 us with 1; 2 rows: 6.1 us with either).
  const int64_t work = (int64_t)p.B * ((p.MB + kChunk - 1) / kChunk) / kWarps +
                       (int64_t)p.T / (kThreads * kTokens) + p.groups / kWarps;
  const bool can = dev >= 0 && dev < 64 && (wide.load() & (1ull << dev));
  const unsigned C = work < 64 || !can ? 8 : kMaxCluster;
  ScheduleParams q = p;
  q.apart = (p.slots || p.positions) && p.T >= kApartFrom ? 1 : 0;
  {
    ProfScope ps("schedule", s);
    cfg.gridDim = dim3(C);
    cfg.dynamicSmemBytes = schedule_smem(p);
    attr[0].val.clusterDim.x = C;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, schedule_kernel, q);
    if (e != cudaSuccess || !q.apart) return e;
  }
  ProfScope ps("schedule", s);
  const int64_t blocks = ((int64_t)p.T + kSlotThreads * kTokens - 1) / (kSlotThreads * kTokens);
  const int fit = 2 * device_sms();
  cfg.gridDim = dim3((unsigned)(blocks < fit ? blocks : fit));
  cfg.blockDim = dim3(kSlotThreads);
  cfg.dynamicSmemBytes = sizeof(int) * ((size_t)p.B + 1);
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  return cudaLaunchKernelEx(&cfg, schedule_slots_kernel, q);
}

}  // namespace pkv
