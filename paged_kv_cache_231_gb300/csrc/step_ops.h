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

// ---- append with norms ----------------------------------------------------------------
struct NormParams {
  AxesParams axes;
  const void* qw;            // NULL: not normed
  const void* kw;
  float epsilon;
  int weight_f32;
};
cudaError_t launch_append_norm(const NormParams& p, cudaStream_t s);

// ---- fork -----------------------------------------------------------------------------
struct ForkParams {
  const int32_t* parents;
  const int32_t* past;
  const int32_t* table;
  int32_t* new_past;
  int32_t* new_table;
  int32_t* free_out;         // may be NULL
  int32_t* status;
  int32_t* count;            // workspace: copies, and their [B] (source, destination, rows, -)
  int4* list;
  int B, MB, BS, NB, bs_shift;
  int groups;                // groups of 1024 block ids
  int caches;
  int pieces;                // units of 32 KB that a block of the widest cache has
  int row_words[PKV_MAX_FORK_CACHES];   // 16-byte words of a token's row
  void* cache[PKV_MAX_FORK_CACHES];
};
constexpr int kForkPiece = 2048;   // words of a unit
cudaError_t launch_fork(const ForkParams& p, cudaStream_t s);

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
  // causal forms: query row i of a sequence stands at past + i
  const int32_t* past;
  int window;                // keys that a row sees, 0: all
  int sinks;                 // first keys that stay visible
  // behind a shared prefix (NULL without): keys of a sequence that its group computes
  const int32_t* start;      // [B]
  const float* prior_o;      // [T][Hq][D] what the shared keys gave, and its lse [T][Hq]
  const float* prior_lse;
  const int32_t* choice;     // 1: single tokens take the kernel for few and short sequences
  // Where that kernel runs beside the tiles of the shared keys, what a sequence's own keys gave:
  // [T][Hq][D] sums and [T][Hq] (maximum in log2 units, sum of weights); the join takes both in
  float* apart_o;
  float2* apart_ml;
  const int32_t* check_offsets;   // groups that are looked at for faults alone
  const int32_t* check_shared;
  int check_groups;
  // the shared keys' own call: B groups; row of the block table of each
  const int32_t* table_row;  // [B]
  const int32_t* active;     // 0: nothing is shared
  const int32_t* units;      // blocks of the tiles that work (NULL: all)
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
struct PrefixParams {
  const int32_t* offsets;    // [groups + 1]
  const int32_t* shared;     // [groups] keys that the caller says they share
  int groups;
  // workspace, written by the plan
  int32_t* start;            // [B] keys that are computed for the sequence's group
  int32_t* group_cu;         // [groups + 1] query rows
  int32_t* group_keys;       // [groups]
  int32_t* table_row;        // [groups]
  int32_t* active;           // see CrossParams
  int32_t* choice;
  int32_t* units;
  int units_most;            // blocks of the tiles
  int sms;
  int always;                // testing hook: share whatever it saves
};
// the parameters of both calls from those of the second (its query, cache and sizes); the bytes.
// Without a start nothing is shared, whatever the lengths are.
size_t prefix_layout(CrossParams* shared, CrossParams* own, PrefixParams* x, char* base);
cudaError_t launch_prefix(const CrossParams& shared, const CrossParams& own, const PrefixParams& x,
                          cudaStream_t s);
// fills the plan fields and the workspace pointers (from base, which may be NULL); returns
// the workspace bytes
size_t cross_layout(CrossParams* p, char* base, bool tiles_only = false);
// the kernels of the three forms (cross_dev.cuh) and, of each, the one for many rows (*_tiles.cu)
// parts of a call: the tiles, the kernel for few and short sequences, and what follows them
enum { kTilesPart = 1, kSmallPart = 2, kRestPart = 4, kAllParts = 7 };
cudaError_t launch_cross(const CrossParams& p, cudaStream_t s, int parts = kAllParts);
cudaError_t launch_shared(const CrossParams& p, cudaStream_t s, int parts = kAllParts);
cudaError_t launch_causal(const CrossParams& p, cudaStream_t s, int parts = kAllParts);
cudaError_t launch_cross_tiles(const CrossParams& p, cudaStream_t s);
cudaError_t launch_shared_tiles(const CrossParams& p, cudaStream_t s);
cudaError_t launch_causal_tiles(const CrossParams& p, cudaStream_t s);

}  // namespace pkv
