// Rows of the block table copied, reordered and freed (pkv_paged_fork).
//
// New row b takes over n = past[p] tokens of old row p = parents[b]. With BS tokens to a block its
// whole blocks n / BS are shared; the partly filled one behind them (n % BS > 0) is kept by one
// row of those with the same parent (the parent itself, else the first), the others ask for a
// block each. Blocks are free when no new row holds them: it is enough to mark what every parent
// that goes on holds, once. The r-th row that asks gets the r-th free id.
//
// Two kernels. The first is one cluster of blocks, as the schedule's: the parents' entries are
// marked in bitmaps of the whole pool in each block's shared memory, joined through distributed
// shared memory; ranks are prefix sums. It writes the new lengths, the entries of partly filled
// blocks and a list of (source, destination, rows), and is bound by latency. The second, on all SMs,
// writes the table and copies the list's rows in every cache: bound by HBM, 2 * (n % BS) * row
// bytes for each copy and cache. A source is held by the row that keeps it and a destination by
// nobody, so no copy reads what another one writes.
#include <cooperative_groups.h>
#include <limits.h>

#include "device_common.cuh"
#include "internal.h"
#include "pool_dev.cuh"
#include "step_ops.h"

namespace pkv {
namespace {

namespace cg = cooperative_groups;
using pool::block_sum;
using pool::kThreads;
using pool::kWarps;

constexpr int kChunk = 128;   // table columns of a row that a warp marks as one piece
constexpr int kUnits = 4;     // such pieces whose loads are under way at once
constexpr unsigned kMaxCluster = 16;
static_assert(kScheduleMaxBlocks / 1024 <= kThreads, "a thread a group");

__device__ __forceinline__ int column(const ForkParams& p, int pos) {
  return p.bs_shift >= 0 ? pos >> p.bs_shift : pos / p.BS;
}
__device__ __forceinline__ bool in_pool(const ForkParams& p, int id) {
  return id >= 0 && id < p.NB;
}
// tokens that a row of this parent takes over
__device__ __forceinline__ int tokens_of(const ForkParams& p, int parent, int* flags) {
  if (parent < 0) return 0;
  if (parent >= p.B) {
    *flags |= PKV_DEV_BAD_SEQUENCE;
    return 0;
  }
  const int n = __ldg(p.past + parent);
  if (n < 0) *flags |= PKV_DEV_BAD_SEQUENCE;
  if (n > p.MB * p.BS) *flags |= PKV_DEV_BAD_BLOCK;   // the product is below 2^31
  return n < 0 || n > p.MB * p.BS ? 0 : n;
}

__global__ void __launch_bounds__(kThreads)
    fork_plan_kernel(const __grid_constant__ ForkParams p) {
  extern __shared__ __align__(16) int smem[];
  __shared__ int s_asked[2][kWarps], s_groups[kWarps];   // one of two: see block_sum
  int* keep = smem;                  // [B] row that keeps a parent's last block; then held entries
  int* upto = keep + p.B;            // [B] blocks asked for by the rows up to this one
  int* gfree = upto + p.B;           // [groups] free ids of a group, then those before it
  uint32_t* bits = reinterpret_cast<uint32_t*>(gfree + p.groups);   // [groups * 32]

  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int flags = 0;

  for (int i = tid; i < p.groups * 32; i += kThreads) bits[i] = 0u;
  for (int b = tid; b < p.B; b += kThreads) keep[b] = INT_MAX;
  __syncthreads();
  for (int b = tid; b < p.B; b += kThreads) {
    const int from = __ldg(p.parents + b);
    if (from >= 0 && from < p.B) atomicMin(keep + from, from == b ? -1 : b);
  }
  __syncthreads();
  int asked_all = 0;
#pragma unroll 1
  for (int c0 = 0; c0 < p.B; c0 += kThreads) {
    const int b = c0 + tid;
    int asked = 0;
    if (b < p.B) {
      const int from = __ldg(p.parents + b), n = tokens_of(p, from, &flags);
      const int full = column(p, n);
      if (n > full * p.BS && from != b && keep[from] != b)
        asked = in_pool(p, __ldg(p.table + (int64_t)from * p.MB + full)) ? 1 : 0;
    }
    int total;
    const int a = block_sum<int>(asked, &total, s_asked[(c0 / kThreads) & 1]);
    if (b < p.B) upto[b] = asked_all + a;
    asked_all += total;
  }
  __syncthreads();
  for (int b = tid; b < p.B; b += kThreads) {   // entries of old row b that go on being held
    int f = 0;
    const int n = keep[b] != INT_MAX ? tokens_of(p, b, &f) : 0;
    keep[b] = n > 0 ? column(p, n - 1) + 1 : 0;
  }
  if (rank > 0) flags = 0;   // every block saw them
  __syncthreads();

  // mark them, a warp kUnits pieces of a row at a time
  const int chunks = (p.MB - 1) / kChunk + 1, units = p.B * chunks;
  const int apart = C * kWarps;
  for (int u0 = rank + C * warp; u0 < units; u0 += apart * kUnits) {
    int id[kUnits][kChunk / 32];
#pragma unroll
    for (int x = 0; x < kUnits; ++x) {
      const int u = u0 + x * apart, b = u / chunks, c0 = (u - b * chunks) * kChunk;
      const int held = u < units ? keep[b] : 0;
      const int32_t* row = p.table + (int64_t)b * p.MB;
#pragma unroll
      for (int k = 0; k < kChunk / 32; ++k) {
        const int c = c0 + k * 32 + lane;
        id[x][k] = c < held ? __ldg(row + c) : -1;
      }
    }
#pragma unroll
    for (int x = 0; x < kUnits; ++x)
#pragma unroll
      for (int k = 0; k < kChunk / 32; ++k) {
        const int v = id[x][k];
        if (in_pool(p, v))
          atomicOr(bits + (v >> 5), 1u << (v & 31));
        else if (v != -1)
          flags |= PKV_DEV_BAD_BLOCK;
      }
  }
  cluster.sync();

  // join the bitmaps of the groups of 1024 ids that this block owns; free ids become set bits
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
  __syncthreads();
  const int given = min(asked_all, free_ids);
  // the blocks asked for: the free ids of this block's groups, by rank
  for (int g = rank + C * warp; g < p.groups; g += C * kWarps) {
    if (gfree[g] >= given) break;   // ranks only grow
    uint32_t open = bits[g * 32 + lane];
    const int n = __popc(open);
    int x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    for (int r = gfree[g] + x - n; open && r < given; open &= open - 1, ++r)
      p.list[r].y = g * 1024 + lane * 32 + __ffs(open) - 1;
  }
  cluster.sync();   // every block sees the ids written above
  // lengths, the entries of partly filled blocks, and the list
  for (int b = rank * kThreads + tid; b < p.B; b += C * kThreads) {
    int f = 0;
    const int from = __ldg(p.parents + b), upto_b = upto[b];
    int n = tokens_of(p, from, &f);
    const bool asked = upto_b > (b > 0 ? upto[b - 1] : 0);
    if (asked && upto_b > given) {
      flags |= PKV_DEV_NO_BLOCKS;
      n = 0;
    }
    p.new_past[b] = n;
    const int full = column(p, n);
    if (n == full * p.BS) continue;
    int id = __ldg(p.table + (int64_t)from * p.MB + full);
    if (asked) {
      const int src = id;
      id = __ldcg(&p.list[upto_b - 1].y);
      p.list[upto_b - 1] = make_int4(src, id, n - full * p.BS, 0);
    }
    p.new_table[(int64_t)b * p.MB + full] = id;
  }
  if (rank == 0 && tid == 0) {
    p.count[0] = given;
    if (p.free_out) *p.free_out = free_ids - given;
  }
  if (flags) flag_status(p.status, flags);
}

// Behind it: the whole table, but for the entries written above, and the copies.
constexpr int kCopyThreads = 256;
constexpr int kDeep = 8;   // 16-byte words of a thread under way
constexpr int kPiece = kForkPiece;
static_assert(kPiece == kCopyThreads * kDeep, "words of a unit");
__global__ void __launch_bounds__(kCopyThreads)
    fork_copy_kernel(const __grid_constant__ ForkParams p) {
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const int tid = threadIdx.x;
  const int each = p.caches * p.pieces;                 // units of a copy
  const int64_t total = (int64_t)__ldcg(p.count) * each;
  for (int64_t u = blockIdx.x; u < total; u += gridDim.x) {
    const int nth = (int)(u / each), rest = (int)(u - (int64_t)nth * each);
    const int cache = rest / p.pieces, piece = rest - cache * p.pieces;
    const int4 c = __ldcg(p.list + nth);
    const int words = p.row_words[cache], n = c.z * words;
    if (piece * kPiece >= n) continue;
    uint4* const base = static_cast<uint4*>(p.cache[cache]);
    const uint4* src = base + (int64_t)c.x * p.BS * words;
    uint4* dst = base + (int64_t)c.y * p.BS * words;
    uint4 x[kDeep];
#pragma unroll
    for (int k = 0; k < kDeep; ++k) {
      const int i = piece * kPiece + k * kCopyThreads + tid;
      if (i < n) x[k] = __ldg(src + i);   // the next copies read the same block
    }
#pragma unroll
    for (int k = 0; k < kDeep; ++k) {
      const int i = piece * kPiece + k * kCopyThreads + tid;
      if (i < n) __stcs(dst + i, x[k]);
    }
  }
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    const int n = __ldcg(p.new_past + b), from = __ldg(p.parents + b);
    const int full = column(p, n), part = n > full * p.BS ? full : -1;
    const int32_t* old = p.table + (int64_t)from * p.MB;   // read where n > 0 alone
    int32_t* row = p.new_table + (int64_t)b * p.MB;
    // unsigned: a row may end less than a block's step in front of 2^31
    for (uint32_t c = tid; c < (uint32_t)p.MB; c += kCopyThreads)
      if ((int)c != part) row[c] = (int)c < full ? __ldg(old + c) : -1;
  }
}

size_t fork_smem(const ForkParams& p) {
  return sizeof(int) * ((size_t)2 * p.B + (size_t)p.groups * 33);
}
constexpr size_t kMaxSmem =
    sizeof(int) * ((size_t)2 * kScheduleMaxBatch + (size_t)(kScheduleMaxBlocks / 1024) * 33);
static_assert(kMaxSmem <= 230000, "fork shared memory over the limit");

}  // namespace

cudaError_t launch_fork(const ForkParams& p, cudaStream_t s) {
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
        fork_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxSmem);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(fork_plan_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(kMaxCluster);
    cfg.dynamicSmemBytes = kMaxSmem;
    int clusters = 0;
    if (cudaOccupancyMaxActiveClusters(&clusters, fork_plan_kernel, &cfg) == cudaSuccess &&
        clusters > 0)
      mark_configured(wide, dev);
    else
      (void)cudaGetLastError();
    mark_configured(configured, dev);
  }
  // as the schedule's cluster: 16 blocks where there are many entries to mark
  const int64_t work =
      (int64_t)p.B * ((p.MB - 1) / kChunk + 1) / kWarps + p.groups / kWarps;
  const bool can = dev >= 0 && dev < 64 && (wide.load() & (1ull << dev));
  {
    ProfScope ps("fork_plan", s);
    attr[0].val.clusterDim.x = work < 64 || !can ? 8 : kMaxCluster;
    cfg.gridDim = dim3(attr[0].val.clusterDim.x);
    cfg.dynamicSmemBytes = fork_smem(p);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, fork_plan_kernel, p);
    if (e != cudaSuccess) return e;
  }
  ProfScope ps("fork_copy", s);
  const int64_t most = (int64_t)p.B * (p.caches > 0 ? (int64_t)p.caches * p.pieces : 1);
  const int64_t fit = (int64_t)8 * device_sms();
  cfg.gridDim = dim3((unsigned)(most < fit ? most : fit));
  cfg.blockDim = dim3(kCopyThreads);
  cfg.dynamicSmemBytes = 0;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  return cudaLaunchKernelEx(&cfg, fork_copy_kernel, p);
}

}  // namespace pkv
