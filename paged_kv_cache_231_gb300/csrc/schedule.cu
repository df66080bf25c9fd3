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
// One launch, one cluster of C blocks, no workspace. Every block marks the held entries that
// it reads in a bitmap of the whole pool in its own shared memory (local atomics); group g of
// 1024 ids belongs to block g % C, which joins the C bitmaps of the group through distributed
// shared memory and hands its count of free ids to all. Each block then scans the rows for
// itself (cheaper than passing the sums around), writes the new table entries of its groups
// and, after a cluster barrier, the slots of its share of the tokens.
#include <cooperative_groups.h>

#include "device_common.cuh"
#include "internal.h"
#include "step_ops.h"

namespace pkv {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kChunk = 128;   // table columns that a warp marks at a time

struct Row {
  int past, held, tokens, asked, flags;
};

__device__ __forceinline__ int blocks_for(const ScheduleParams& p, int tokens) {
  if (tokens <= 0) return 0;
  return (p.bs_shift >= 0 ? (tokens - 1) >> p.bs_shift : (tokens - 1) / p.BS) + 1;
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

// Inclusive sum over the block's threads; *total gets the sum of all.
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
  if (w == 0) {
    T t = scratch[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T y = __shfl_up_sync(0xffffffffu, t, o);
      if (lane >= o) t += y;
    }
    scratch[lane] = t;
  }
  __syncthreads();
  if (w > 0) v += scratch[w - 1];
  *total = scratch[kWarps - 1];
  __syncthreads();
  return v;
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

__global__ void __launch_bounds__(kThreads) schedule_kernel(ScheduleParams p) {
  extern __shared__ __align__(16) int smem[];
  __shared__ int64_t s_scan[kWarps];
  __shared__ int s_used, s_last;
  int* upto = smem;                  // [B] A_b
  int* cu = upto + p.B;              // [B + 1]
  int* gfree = cu + p.B + 1;         // [groups] free ids of a group, then those before it
  uint32_t* bits = reinterpret_cast<uint32_t*>(gfree + p.groups);   // [groups * 32]

  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int flags = 0;

  for (int i = tid; i < p.groups * 32; i += kThreads) bits[i] = 0u;
  if (tid == 0) s_used = s_last = cu[0] = 0;

  int carry = 0;
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
    const int a = block_sum<int>(asked, &total, reinterpret_cast<int*>(s_scan));
    if (b < p.B) upto[b] = carry + a;
    carry += total;
  }
  __syncthreads();

  // mark the held entries
  const int chunks = (p.MB + kChunk - 1) / kChunk;
  const int64_t units = (int64_t)p.B * chunks;
  for (int64_t u = (int64_t)rank * kWarps + warp; u < units; u += (int64_t)C * kWarps) {
    const int b = (int)(u / chunks), c0 = (int)(u % chunks) * kChunk;
    const int held = cu[b + 1];
    if (c0 >= held) continue;
    const int32_t* row = p.table + (int64_t)b * p.MB;
    int id[kChunk / 32];
#pragma unroll
    for (int k = 0; k < kChunk / 32; ++k) {
      const int c = c0 + k * 32 + lane;
      id[k] = c < held ? __ldcg(row + c) : -1;
    }
#pragma unroll
    for (int k = 0; k < kChunk / 32; ++k) {
      if (id[k] >= 0 && id[k] < p.NB)
        atomicOr(bits + (id[k] >> 5), 1u << (id[k] & 31));
      else if (id[k] != -1)
        flags |= PKV_DEV_BAD_BLOCK;
    }
  }
  cluster.sync();

  // join the bitmaps of the groups that this block owns; free ids become set bits
  for (int g = rank + C * warp; g < p.groups; g += C * kWarps) {
    uint32_t used = 0u;
    for (int r = 0; r < C; ++r) used |= cluster.map_shared_rank(bits, r)[g * 32 + lane];
    const int first = g * 1024 + lane * 32;
    uint32_t open = ~used;
    if (first + 32 > p.NB) open &= first < p.NB ? (1u << (p.NB - first)) - 1u : 0u;
    int n = __popc(open);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    __syncwarp();
    bits[g * 32 + lane] = open;   // only the owner reads its copy of the group
    if (lane < C) cluster.map_shared_rank(gfree, lane)[g] = n;
  }
  cluster.sync();

  int free_ids = 0;
  for (int c0 = 0; c0 < p.groups; c0 += kThreads) {
    const int g = c0 + tid;
    const int n = g < p.groups ? gfree[g] : 0;
    int total;
    const int upto_g = block_sum<int>(n, &total, reinterpret_cast<int*>(s_scan));
    if (g < p.groups) gfree[g] = free_ids + upto_g - n;
    free_ids += total;
  }

  // which rows are granted
  int64_t tokens = 0;
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
    const int64_t upto_t = tokens + block_sum<int64_t>(given, &total, s_scan);
    tokens += total;
    if (b < p.B) {
      const bool fits = upto_t <= p.T;
      cu[b + 1] = fits ? (int)upto_t : -1;
      if (fits) atomicMax(&s_last, (int)upto_t);
      if (given > 0 && fits) atomicAdd(&s_used, asked);
      if (want > 0 && given == 0) flags |= PKV_DEV_NO_BLOCKS;
      if (given > 0 && !fits) flags |= PKV_DEV_BAD_SEQUENCE;
    }
  }
  __syncthreads();
  for (int b = tid; b < p.B; b += kThreads)
    if (cu[b + 1] < 0) cu[b + 1] = s_last;   // behind the last row that fits
  __syncthreads();

  if (rank == 0) {
    for (int b = tid; b <= p.B; b += kThreads) p.cu[b] = cu[b];
    if (p.total)
      for (int b = tid; b < p.B; b += kThreads) p.total[b] = p.past[b] + cu[b + 1] - cu[b];
    if (p.free_out && tid == 0) *p.free_out = free_ids - s_used;
  }

  // new table entries: the free ids of this block's groups, by rank
  const int asked_all = min(upto[p.B - 1], free_ids);
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

  // slots and positions, four tokens to a thread
  const int granted = cu[p.B];
  const bool wide = ((reinterpret_cast<uintptr_t>(p.slots) | reinterpret_cast<uintptr_t>(p.positions)) & 15u) == 0;
  if (p.slots || p.positions) {
    for (int64_t i0 = ((int64_t)rank * kThreads + tid) * 4; i0 < p.T;
         i0 += (int64_t)C * kThreads * 4) {
      int slot[4], pos[4];
      int b = i0 < granted ? first_above(cu + 1, p.B, (int)i0) : 0;
      int col_at = -1, row_at = -1, id = -1;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int64_t i = i0 + k;
        slot[k] = pos[k] = -1;
        if (i >= granted) continue;
        while (cu[b + 1] <= i) ++b;
        pos[k] = __ldg(p.past + b) + (int)(i - cu[b]);
        const int col = p.bs_shift >= 0 ? pos[k] >> p.bs_shift : pos[k] / p.BS;
        if (col != col_at || b != row_at) {
          id = __ldcg(p.table + (int64_t)b * p.MB + col);
          if (id < 0 || id >= p.NB) {
            id = -1;
            flags |= PKV_DEV_BAD_BLOCK;
          }
          col_at = col;
          row_at = b;
        }
        if (id >= 0) slot[k] = id * p.BS + (pos[k] - col * p.BS);
      }
      if (wide && i0 + 4 <= p.T) {
        if (p.slots) *reinterpret_cast<int4*>(p.slots + i0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
        if (p.positions) *reinterpret_cast<int4*>(p.positions + i0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (i0 + k >= p.T) break;
          if (p.slots) p.slots[i0 + k] = slot[k];
          if (p.positions) p.positions[i0 + k] = pos[k];
        }
      }
    }
  }
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
  static std::atomic<uint64_t> configured{0};
  int dev = -1;
  if (needs_configure(configured, &dev)) {
    const cudaError_t e = cudaFuncSetAttribute(
        schedule_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxSmem);
    if (e != cudaSuccess) return e;
    mark_configured(configured, dev);
  }
  ProfScope ps("schedule", s);
  cudaLaunchConfig_t cfg = {};
  const unsigned C = 1;
  cfg.gridDim = dim3(C);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = schedule_smem(p);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, schedule_kernel, p);
}

}  // namespace pkv
