// Host side of the step operators: argument checks and launches of pkv_paged_schedule,
// the appends with rotary axes, the cross, window and prefix attention and pkv_paged_fork.
// Every check is made before anything is enqueued; no function here throws.
#include <cmath>

#include "internal.h"
#include "step_ops.h"

namespace pkv {
namespace {

inline bool aligned(const void* p, uintptr_t n) {
  return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}
inline int log2_or(int64_t x) {   // log2 of a power of two, else -1
  if (x <= 0 || (x & (x - 1)) != 0) return -1;
  int s = 0;
  while ((int64_t(1) << s) < x) ++s;
  return s;
}
inline int status_of(cudaError_t e) { return e == cudaSuccess ? PKV_OK : PKV_ERR_LAUNCH; }
constexpr int64_t kMax32 = INT32_MAX;

// What the cross, the window and the prefix attention check alike; `lengths` is the third of a
// sequence's arrays (its states, or the tokens in front of its rows).
template <typename Args>
int check_attention(const Args* a, const int32_t* lengths, CrossParams* p) {
  if (a->dtype != PKV_F16 && a->dtype != PKV_BF16) return PKV_ERR_DTYPE;
  if (a->num_heads <= 0 || a->kv_num_heads <= 0 || a->num_heads % a->kv_num_heads != 0)
    return PKV_ERR_HEADS;
  if (a->head_size <= 0 || a->block_size <= 0 || a->num_blocks <= 0 || a->batch < 1 ||
      a->max_blocks < 1 || a->num_tokens < 0 || a->max_query_len < 0)
    return PKV_ERR_SHAPE;
  if (std::isnan(a->scale) || std::isinf(a->scale)) return PKV_ERR_SHAPE;
  // products of these are formed as int64 below: bound the factors first
  if (a->num_heads > 65536 || a->block_size > kMax32 || a->max_blocks > kMax32 ||
      a->num_blocks > kMax32 || a->num_tokens > kMax32 / 2 || a->batch > kMax32 / 2)
    return PKV_ERR_UNSUPPORTED;
  if (a->head_size != 64 && a->head_size != 128) return PKV_ERR_UNSUPPORTED;
  const int64_t G = a->num_heads / a->kv_num_heads;
  if (G > 16 || a->max_blocks * a->block_size > kMax32 / 2) return PKV_ERR_UNSUPPORTED;
  p->T = (int)a->num_tokens;
  p->B = (int)a->batch;
  p->Hq = (int)a->num_heads;
  p->Hkv = (int)a->kv_num_heads;
  p->G = (int)G;
  p->D = (int)a->head_size;
  p->BS = (int)a->block_size;
  p->MB = (int)a->max_blocks;
  p->NB = a->num_blocks;
  p->bs_shift = log2_or(a->block_size);
  p->max_q = (int)(a->max_query_len > 0 && a->max_query_len < a->num_tokens ? a->max_query_len
                                                                          : a->num_tokens);
  p->bf16 = a->dtype == PKV_BF16 ? 1 : 0;
  if (a->num_tokens == 0) return PKV_OK;   // nothing is read or written
  if (!a->query || !a->key_cache || !a->value_cache || !a->cumulative_sequence_length ||
      !lengths || !a->block_table || !a->output)
    return PKV_ERR_NULL;
  if (!aligned(a->query, 16) || !aligned(a->key_cache, 16) || !aligned(a->value_cache, 16) ||
      !aligned(a->output, 16) || !aligned(a->lse, 4))
    return PKV_ERR_ALIGN;
  p->q = a->query;
  p->kc = a->key_cache;
  p->vc = a->value_cache;
  p->cu = a->cumulative_sequence_length;
  p->table = a->block_table;
  p->out = a->output;
  p->lse = a->lse;
  p->status = a->device_status;
  const double scale = a->scale != 0.f ? (double)a->scale : 1.0 / std::sqrt((double)p->D);
  p->scale_log2 = (float)(scale * 1.4426950408889634);
  p->wait_tries = testing_wait_tries();
  p->withhold_copy = testing_withhold_copy();
  return PKV_OK;
}

int check_cross(const pkv_cross_attention_args* a, CrossParams* p) {
  if (!a) return PKV_ERR_NULL;
  p->klen = a->key_seqlens;
  return check_attention(a, a->key_seqlens, p);
}

int check_window(const pkv_window_attention_args* a, CrossParams* p) {
  if (!a) return PKV_ERR_NULL;
  if (a->window < 0 || a->sinks < 0) return PKV_ERR_SHAPE;
  p->past = a->past_seqlens;
  // positions lie below 2^30: longer windows see everything
  p->window = (int)(a->window < kMax32 / 2 ? a->window : 0);
  p->sinks = p->window > 0 ? (int)(a->sinks < kMax32 / 2 ? a->sinks : kMax32 / 2) : 0;
  return check_attention(a, a->past_seqlens, p);
}

int check_prefix(const pkv_prefix_attention_args* a, CrossParams* p, PrefixParams* x) {
  if (!a) return PKV_ERR_NULL;
  if (a->num_groups < 0) return PKV_ERR_SHAPE;
  if (a->num_groups > kMax32 / 2) return PKV_ERR_UNSUPPORTED;
  x->groups = (int)a->num_groups;
  x->offsets = a->group_offsets;
  x->shared = a->shared_seqlens;
  p->past = a->past_seqlens;
  const int st = check_attention(a, a->past_seqlens, p);
  if (st != PKV_OK || a->num_tokens == 0) return st;
  if (a->num_groups > 0 && (!a->group_offsets || !a->shared_seqlens)) return PKV_ERR_NULL;
  return PKV_OK;
}

// *nothing: no tokens, nothing to launch
int check_append(const pkv_append_axes_args* a, AxesParams* out, bool* nothing) {
  *nothing = false;
  if (a->dtype != PKV_F16 && a->dtype != PKV_BF16) return PKV_ERR_DTYPE;
  if (a->num_heads <= 0 || a->kv_num_heads <= 0 || a->num_heads % a->kv_num_heads != 0)
    return PKV_ERR_HEADS;
  if (a->num_tokens < 0 || a->head_size <= 0 || a->block_size <= 0 || a->num_blocks <= 0)
    return PKV_ERR_SHAPE;
  if (a->rotary_dim < 0 || a->rotary_dim % 2 != 0 || a->rotary_dim > a->head_size)
    return PKV_ERR_SHAPE;
  const bool rot = a->rotary_dim > 0;
  if (rot && (a->num_axes < 1 || a->num_axes > PKV_MAX_ROTARY_AXES || a->rotary_positions <= 0))
    return PKV_ERR_SHAPE;
  if (rot && a->table_dtype != a->dtype && a->table_dtype != PKV_F32) return PKV_ERR_DTYPE;
  if (a->head_size % 8 != 0 || a->head_size > 256 || a->num_heads > 65536 ||
      a->block_size > kMax32 || a->num_blocks > kMax32 || a->num_tokens > kMax32 / 2)
    return PKV_ERR_UNSUPPORTED;
  uint32_t used = 0;
  if (rot)
    for (int64_t i = 0; i < a->rotary_dim / 2; ++i) {
      if (a->pair_axis[i] >= a->num_axes) return PKV_ERR_SHAPE;
      used |= 1u << a->pair_axis[i];
    }
  if (a->num_tokens == 0) {
    *nothing = true;
    return PKV_OK;
  }
  const bool hk = a->key != nullptr, hv = a->value != nullptr;
  if (hk != hv) return PKV_ERR_KV_MODE;
  if (!a->key_cache || !a->value_cache || !a->slot_mapping) return PKV_ERR_NULL;
  if ((!hk || a->query_out) && !a->query) return PKV_ERR_NULL;
  if (rot && (!a->positions || !a->cos_cache || !a->sin_cache)) return PKV_ERR_NULL;
  if (!aligned(a->query, 16) || !aligned(a->key, 16) || !aligned(a->value, 16) ||
      !aligned(a->query_out, 16) || !aligned(a->key_cache, 16) || !aligned(a->value_cache, 16) ||
      (rot && (!aligned(a->cos_cache, 4) || !aligned(a->sin_cache, 4))))
    return PKV_ERR_ALIGN;
  if (a->query_out && a->query_out == a->query) return PKV_ERR_SHAPE;
  AxesParams& p = *out;
  const int64_t D = a->head_size, qh = a->num_heads * D, kvh = a->kv_num_heads * D;
  const char* q = static_cast<const char*>(a->query);
  if (hk) {
    p.k = a->key;
    p.v = a->value;
    p.q_stride = qh;
    p.kv_stride = kvh;
  } else {
    p.k = q + qh * 2;
    p.v = q + (qh + kvh) * 2;
    p.q_stride = p.kv_stride = qh + 2 * kvh;
  }
  p.q = a->query_out ? q : nullptr;
  p.q_out = a->query_out;
  p.kc = a->key_cache;
  p.vc = a->value_cache;
  p.slots = a->slot_mapping;
  p.pos = a->positions;
  p.cos = a->cos_cache;
  p.sin = a->sin_cache;
  p.status = a->device_status;
  p.pool_rows = a->num_blocks * a->block_size;
  p.T = (int)a->num_tokens;
  p.Hq = a->query_out ? (int)a->num_heads : 0;
  p.Hkv = (int)a->kv_num_heads;
  p.D = (int)D;
  p.R = (int)a->rotary_dim;
  p.axes = rot ? a->num_axes : 0;
  p.P = (int)(a->rotary_positions < kMax32 ? a->rotary_positions : kMax32);
  p.interleaved = a->rotary_interleaved ? 1 : 0;
  p.bf16 = a->dtype == PKV_BF16 ? 1 : 0;
  p.table_f32 = a->table_dtype == PKV_F32 ? 1 : 0;
  p.used_axes = used;
  for (int i = 0; i < p.R / 2; ++i) p.pair_axis[i] = a->pair_axis[i];
  return PKV_OK;
}

size_t fork_workspace(const ForkParams& p) { return 256 + (size_t)p.B * sizeof(int4); }

int check_fork(const pkv_fork_args* a, ForkParams* p) {
  if (!a) return PKV_ERR_NULL;
  if (a->batch < 1 || a->max_blocks < 1 || a->num_blocks < 1 || a->block_size < 1 ||
      a->num_caches < 0)
    return PKV_ERR_SHAPE;
  if (a->batch > kScheduleMaxBatch || a->num_blocks > kScheduleMaxBlocks ||
      a->block_size > kMax32 || a->max_blocks > kMax32 ||
      a->num_blocks * a->block_size > kMax32 || a->max_blocks * a->block_size > kMax32 - 16 ||
      a->batch * a->max_blocks > kMax32 || a->num_caches > PKV_MAX_FORK_CACHES)
    return PKV_ERR_UNSUPPORTED;
  if (!a->parents || !a->past_seqlens || !a->block_table || !a->new_past_seqlens ||
      !a->new_block_table || (a->num_caches > 0 && (!a->caches || !a->cache_row_bytes)))
    return PKV_ERR_NULL;
  // the inputs are read while the outputs are written
  const int32_t* outs[] = {a->new_past_seqlens, a->new_block_table, a->free_blocks};
  for (const int32_t* o : outs)
    if (o && (o == a->parents || o == a->past_seqlens || o == a->block_table))
      return PKV_ERR_SHAPE;
  int64_t widest = 0;
  for (int64_t i = 0; i < a->num_caches; ++i) {
    const int64_t n = a->cache_row_bytes[i];
    if (n <= 0) return PKV_ERR_SHAPE;
    if (n % 16 != 0 || n > kMax32 / a->block_size) return PKV_ERR_UNSUPPORTED;
    if (!a->caches[i]) return PKV_ERR_NULL;
    if (!aligned(a->caches[i], 16)) return PKV_ERR_ALIGN;
    p->cache[i] = a->caches[i];
    p->row_words[i] = (int)(n / 16);
    if (n > widest) widest = n;
  }
  p->parents = a->parents;
  p->past = a->past_seqlens;
  p->table = a->block_table;
  p->new_past = a->new_past_seqlens;
  p->new_table = a->new_block_table;
  p->free_out = a->free_blocks;
  p->status = a->device_status;
  p->B = (int)a->batch;
  p->MB = (int)a->max_blocks;
  p->BS = (int)a->block_size;
  p->NB = (int)a->num_blocks;
  p->bs_shift = log2_or(a->block_size);
  p->groups = (p->NB + 1023) / 1024;
  p->caches = (int)a->num_caches;
  p->pieces = (int)((widest / 16 * a->block_size + kForkPiece - 1) / kForkPiece);
  return PKV_OK;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" {

int pkv_paged_schedule(const pkv_schedule_args* a, void* stream) {
  if (!a) return PKV_ERR_NULL;
  if (a->batch < 1 || a->max_blocks < 1 || a->num_blocks < 1 || a->block_size < 1 ||
      a->num_tokens < 0)
    return PKV_ERR_SHAPE;
  if (a->batch > kScheduleMaxBatch || a->num_blocks > kScheduleMaxBlocks ||
      a->block_size > kMax32 || a->max_blocks > kMax32 || a->num_tokens >= kMax32 ||
      a->num_blocks * a->block_size > kMax32 || a->max_blocks * a->block_size > kMax32 - 16 ||
      a->batch * a->max_blocks > kMax32)
    return PKV_ERR_UNSUPPORTED;
  if (!a->past_seqlens || !a->new_seqlens || !a->block_table || !a->cumulative_sequence_length)
    return PKV_ERR_NULL;
  // the lengths are read while the outputs are written
  const int32_t* outs[] = {a->block_table, a->cumulative_sequence_length, a->slot_mapping,
                           a->positions, a->total_seqlens, a->free_blocks};
  for (const int32_t* o : outs)
    if (o == a->past_seqlens || o == a->new_seqlens) return PKV_ERR_SHAPE;
  ScheduleParams p{};
  p.past = a->past_seqlens;
  p.fresh = a->new_seqlens;
  p.table = a->block_table;
  p.cu = a->cumulative_sequence_length;
  p.slots = a->slot_mapping;
  p.positions = a->positions;
  p.total = a->total_seqlens;
  p.free_out = a->free_blocks;
  p.status = a->device_status;
  p.B = (int)a->batch;
  p.MB = (int)a->max_blocks;
  p.BS = (int)a->block_size;
  p.NB = (int)a->num_blocks;
  p.T = (int)a->num_tokens;
  p.bs_shift = log2_or(a->block_size);
  p.groups = (p.NB + 1023) / 1024;
  return status_of(launch_schedule(p, static_cast<cudaStream_t>(stream)));
}

int pkv_paged_append_rotary_axes(const pkv_append_axes_args* a, void* stream) {
  if (!a) return PKV_ERR_NULL;
  AxesParams p{};
  bool nothing;
  const int st = check_append(a, &p, &nothing);
  if (st != PKV_OK || nothing) return st;
  return status_of(launch_append_axes(p, static_cast<cudaStream_t>(stream)));
}

int pkv_paged_append_norm_rotary(const pkv_append_norm_args* a, void* stream) {
  if (!a) return PKV_ERR_NULL;
  if (!(a->epsilon > 0.f) || std::isinf(a->epsilon)) return PKV_ERR_SHAPE;
  if (a->weight_dtype != a->append.dtype && a->weight_dtype != PKV_F32) return PKV_ERR_DTYPE;
  NormParams p{};
  bool nothing;
  const int st = check_append(&a->append, &p.axes, &nothing);
  if (st != PKV_OK || nothing) return st;
  if (!a->query_weight && !a->key_weight) return PKV_ERR_NULL;
  if (!aligned(a->query_weight, 4) || !aligned(a->key_weight, 4)) return PKV_ERR_ALIGN;
  p.qw = a->query_weight;
  p.kw = a->key_weight;
  p.epsilon = a->epsilon;
  p.weight_f32 = a->weight_dtype == PKV_F32 ? 1 : 0;
  return status_of(launch_append_norm(p, static_cast<cudaStream_t>(stream)));
}

int pkv_paged_fork_workspace_size(const pkv_fork_args* a, size_t* bytes) {
  if (!bytes) return PKV_ERR_NULL;
  ForkParams p{};
  const int st = check_fork(a, &p);
  if (st != PKV_OK) return st;
  *bytes = fork_workspace(p);
  return PKV_OK;
}

int pkv_paged_fork(const pkv_fork_args* a, void* workspace, size_t workspace_bytes,
                   void* stream) {
  ForkParams p{};
  const int st = check_fork(a, &p);
  if (st != PKV_OK) return st;
  if (!workspace || workspace_bytes < fork_workspace(p) || !aligned(workspace, 256))
    return PKV_ERR_WORKSPACE;
  p.count = static_cast<int32_t*>(workspace);
  p.list = reinterpret_cast<int4*>(static_cast<char*>(workspace) + 256);
  return status_of(launch_fork(p, static_cast<cudaStream_t>(stream)));
}

int pkv_cross_attention_workspace_size(const pkv_cross_attention_args* args, size_t* bytes) {
  if (!bytes) return PKV_ERR_NULL;
  CrossParams p{};
  const int st = check_cross(args, &p);
  if (st != PKV_OK) return st;
  *bytes = cross_layout(&p, nullptr);
  return PKV_OK;
}

int pkv_cross_attention(const pkv_cross_attention_args* args, void* workspace,
                        size_t workspace_bytes, void* stream) {
  CrossParams p{};
  const int st = check_cross(args, &p);
  if (st != PKV_OK) return st;
  if (args->num_tokens == 0) return PKV_OK;
  if (args->output == args->query) return PKV_ERR_SHAPE;
  const size_t need = cross_layout(&p, static_cast<char*>(workspace));
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 256)))
    return PKV_ERR_WORKSPACE;
  return status_of(launch_cross(p, static_cast<cudaStream_t>(stream)));
}

int pkv_paged_window_attention_workspace_size(const pkv_window_attention_args* args,
                                              size_t* bytes) {
  if (!bytes) return PKV_ERR_NULL;
  CrossParams p{};
  const int st = check_window(args, &p);
  if (st != PKV_OK) return st;
  *bytes = cross_layout(&p, nullptr);
  return PKV_OK;
}

int pkv_paged_window_attention(const pkv_window_attention_args* args, void* workspace,
                               size_t workspace_bytes, void* stream) {
  CrossParams p{};
  const int st = check_window(args, &p);
  if (st != PKV_OK) return st;
  if (args->num_tokens == 0) return PKV_OK;
  if (args->output == args->query) return PKV_ERR_SHAPE;
  const size_t need = cross_layout(&p, static_cast<char*>(workspace));
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 256)))
    return PKV_ERR_WORKSPACE;
  return status_of(launch_causal(p, static_cast<cudaStream_t>(stream)));
}

int pkv_paged_prefix_attention_workspace_size(const pkv_prefix_attention_args* args,
                                              size_t* bytes) {
  if (!bytes) return PKV_ERR_NULL;
  CrossParams p{}, shared{};
  PrefixParams x{};
  const int st = check_prefix(args, &p, &x);
  if (st != PKV_OK) return st;
  *bytes = prefix_layout(&shared, &p, &x, nullptr);
  return PKV_OK;
}

int pkv_paged_prefix_attention(const pkv_prefix_attention_args* args, void* workspace,
                               size_t workspace_bytes, void* stream) {
  CrossParams p{}, shared{};
  PrefixParams x{};
  const int st = check_prefix(args, &p, &x);
  if (st != PKV_OK) return st;
  if (args->num_tokens == 0) return PKV_OK;
  if (args->output == args->query) return PKV_ERR_SHAPE;
  const size_t need = prefix_layout(&shared, &p, &x, static_cast<char*>(workspace));
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 256)))
    return PKV_ERR_WORKSPACE;
  return status_of(launch_prefix(shared, p, x, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
