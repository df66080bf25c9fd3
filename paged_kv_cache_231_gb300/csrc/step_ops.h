// Parameter blocks and launchers of the step operators (schedule, append with rotary axes,
// cross attention), shared by step_runtime.cpp and the kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "pagedkv.h"

namespace pkv {

// ---- schedule -------------------------------------------------------------------------
struct ScheduleParams {
  const int32_t* past;
  const int32_t* fresh;      // new tokens of each row
  int32_t* table;
  int32_t* cu;
  int32_t* slots;            // may be NULL, like the four below
  int32_t* positions;
  int32_t* total;
  int32_t* free_out;
  int32_t* status;
  int B, MB, BS, NB, T;
  int bs_shift;              // log2(BS) when BS is a power of two, else -1
  int groups;                // groups of 1024 block ids
  int apart;                 // the tokens' slots are left to a kernel of their own
};
constexpr int kScheduleMaxBatch = 8192;
constexpr int kScheduleMaxBlocks = 1 << 20;
cudaError_t launch_schedule(const ScheduleParams& p, cudaStream_t s);

// ---- append with rotary axes ----------------------------------------------------------
struct AxesParams {
  const void* q;             // first query element of token 0 (NULL: no queries)
  const void* k;
  const void* v;
  int64_t q_stride;          // elements between token rows
  int64_t kv_stride;
  void* q_out;
  void* kc;
  void* vc;
  const int32_t* slots;
  const int32_t* pos;
  const void* cos;
  const void* sin;
  int32_t* status;
  int64_t pool_rows;
  int T, Hq, Hkv, D, R, axes, P;
  int interleaved, bf16, table_f32;
  uint32_t used_axes;        // bit a: some pair turns by axis a
  uint8_t pair_axis[PKV_MAX_ROTARY_PAIRS];
};
cudaError_t launch_append_axes(const AxesParams& p, cudaStream_t s);

// ---- cross attention ------------------------------------------------------------------
struct CrossParams {
  const void* q;
  const void* kc;
  const void* vc;
  const int32_t* cu;
  const int32_t* klen;
  const int32_t* table;
  void* out;
  float* lse;
  int32_t* status;
  int T, B, Hq, Hkv, G, D, BS, MB;
  int64_t NB;
  int bs_shift;
  int max_q;                 // longest sequence the call admits
  int bf16;
  float scale_log2;          // softmax scale * log2(e)
  // plan (cross_dev.cuh)
  int few;                   // query rows of a sequence that the kernel for few rows takes
  int tile_pos;              // query positions of a tile of the kernel for many rows
  int few_heads;             // kv heads that as many neighbouring warps of the first take together
  int few_units;             // warps of the first, blocks of the second (0: not launched)
  int tile_units;
  int small;                 // a block for each sequence and kv head, nothing else (few rows)
  int few_rows;              // rows of a piece of the first: at most 16
  int box_keys;              // keys of a TMA box (0: rows are copied one by one)
  uint32_t wait_tries;       // testing hook (pkv_testing_wait_limit), as in AttnParams
  int withhold_copy;
  // workspace: records, and pieces of warp or block u at slots 2u and 2u + 1
  int4* few_rec;
  float* few_o;              // [2 * few_units][few_rows][D], a piece for each warp and slot
  float* few_m;              // [2 * few_units][few_rows], log2 units
  float* few_l;
  int4* tile_rec;
  float* tile_o;             // [2 * tile_units][256][D]
  float* tile_m;
  float* tile_l;
};
// fills the plan fields and the workspace pointers (from base, which may be NULL); returns
// the workspace bytes
size_t cross_layout(CrossParams* p, char* base);
cudaError_t launch_cross(const CrossParams& p, cudaStream_t s);
// kernel for many rows (cross_tiles.cu)
cudaError_t launch_cross_tiles(const CrossParams& p, cudaStream_t s);

}  // namespace pkv
