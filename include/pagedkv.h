/*
 * pagedkv.h - C ABI of the GB300 paged / block-sparse grouped-query attention library.
 *
 * Operations (each names the page and passage that defines it):
 *
 *   pkv_paged_attention        "com.microsoft.PagedAttention manifest.json": operator
 *                              inputs/outputs/attributes, the derive table and the
 *                              ScatterKV -> AttendSplitK -> AttendSplitKMerge passes.
 *   pkv_paged_scatter_kv       the ScatterKV pass of the same manifest on its own.
 *   pkv_kv_append_rotary       "com.microsoft.SparseAttention sparse-kv-append.wgsl.jinja":
 *                              sparse_schedule, sparse_rotary and the KV-append main.
 *   pkv_sparse_attention_partials
 *                              "alice-llm src/shaders/sparse_attention_forward.wgsl":
 *                              sparse_forward and its layout comment block.
 *   pkv_combine_partials       log-sum-exp merge of (o, m, l) partials: the manifest's
 *                              AttendSplitKMerge pass and the merge of sparse partials.
 *
 * Step operators of a decoder with image, video or audio inputs (the pages have no
 * counterpart; their formulas stand at each call):
 *
 *   pkv_paged_schedule         block tables, slot maps and cumulative lengths built on the
 *                              GPU from request lengths.
 *   pkv_paged_append_rotary_axes
 *                              K / V of new tokens into the paged cache, K and Q rotated
 *                              with one position per axis (time, height, width, ...).
 *   pkv_cross_attention        attention of ragged queries over an encoder's states in a
 *                              paged cache (no causal mask, another length).
 *   pkv_paged_append_norm_rotary
 *                              the append above with a norm of every query and key head in
 *                              front of the rotation.
 *   pkv_paged_window_attention causal attention over the paged cache, fp16 or bf16, with a
 *                              sliding window and first tokens that stay visible.
 *   pkv_paged_prefix_attention causal attention of requests whose first blocks are the same:
 *                              what they share is computed once for all of them.
 *   pkv_paged_fork             rows of the block table copied, reordered and freed.
 *
 * Conventions for every call:
 *   - Tensor pointers are DEVICE pointers owned by the caller; the library never frees
 *     or retains them. Scratch memory is a caller-provided device workspace whose size
 *     the matching *_workspace_size call returns; the library allocates nothing.
 *   - `stream` is a cudaStream_t (CUstream) handle passed as void*; NULL is the legacy
 *     default stream. Calls enqueue work and return without synchronising.
 *   - Host-side argument errors return a pkv_status before anything is enqueued.
 *     Invalid DATA found on the device (a block id outside the pool, a slot past the
 *     pool, ...) never traps: the offending row is skipped or masked as documented and
 *     a PKV_DEV_* bit is OR-ed into the optional `device_status` int32 word.
 *   - All layouts are row-major and dense; sizes are element counts.
 *   - fp16 tensors and every row stride must be 16-byte aligned (head_size % 8 == 0).
 */
#ifndef PAGEDKV_H
#define PAGEDKV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define PKV_ABI_VERSION 3

typedef enum pkv_status {
  PKV_OK = 0,
  PKV_ERR_NULL = 1,        /* a required pointer is NULL */
  PKV_ERR_SHAPE = 2,       /* a size breaks the contract (cacheShapeOk, ioShapeOk,
                              scheduleShapeOk or slotShapeOk of the manifest) */
  PKV_ERR_HEADS = 3,       /* num_heads or kv_num_heads <= 0, or not divisible */
  PKV_ERR_DTYPE = 4,       /* dtype other than the operation's type constraint */
  PKV_ERR_KV_MODE = 5,     /* exactly one of key / value given (neither separateKv
                              nor packedKv holds) */
  PKV_ERR_CAUSAL = 6,      /* is_causal != 1 (the manifest admits only 1) */
  PKV_ERR_WORKSPACE = 7,   /* workspace NULL, too small or not 256-byte aligned */
  PKV_ERR_ALIGN = 8,       /* a tensor pointer is not 16-byte aligned */
  PKV_ERR_UNSUPPORTED = 9, /* a size outside the compiled kernel variants (see each call) */
  PKV_ERR_LAUNCH = 10      /* a CUDA launch or API call failed */
} pkv_status;

/* Bits OR-ed into *device_status by kernels that meet invalid data. */
#define PKV_DEV_BAD_BLOCK 1u     /* block-table entry outside [0, num_blocks), or a key
                                    position past max_blocks * block_size: key masked,
                                    row not written */
#define PKV_DEV_BAD_SLOT 2u      /* slot_mapping entry >= num_blocks * block_size: the
                                    token's K/V are not written (negative = padding,
                                    skipped without a flag) */
#define PKV_DEV_BAD_POSITION 4u  /* KV-append position >= max_cache_seq: row skipped */
#define PKV_DEV_BAD_SEQUENCE 8u  /* cumulative_sequence_length / past_seqlens
                                    inconsistent for a sequence: its tokens get zero
                                    output and are not scattered */
#define PKV_DEV_BAD_EDGE 16u     /* edge_meta field out of range: block_len clipped to
                                    block_size, or a page slot / page id treated as
                                    unmapped; an edge whose q_idx, head, batch or
                                    block lies outside the tensors gets the empty
                                    partial */
#define PKV_DEV_TIMEOUT 32u      /* a bounded wait of a tensor-core kernel gave up: the
                                    outputs that CTA had not yet written (prefill tiles,
                                    block-sparse partials, tiles of the cross, window and
                                    prefix attention) are
                                    not written or not valid; it waited
                                    (bounded) for what it had issued, freed its tensor
                                    memory and returned */
#define PKV_DEV_NO_BLOCKS 64u    /* pkv_paged_schedule: the pool has too few free blocks:
                                    the row gets no tokens this time; pkv_paged_fork: the
                                    row is freed */

typedef enum pkv_dtype { PKV_F16 = 1, PKV_BF16 = 2, PKV_F32 = 3, PKV_I32 = 4 } pkv_dtype;

/* ---------------------------------------------------------------------------------
 * Paged attention (PagedAttention manifest)
 * ------------------------------------------------------------------------------- */

/* Split policy for the attention pass. */
#define PKV_SPLIT_AUTO 0   /* per-sequence split count chosen on the device: up to
                              max_splits splits of >= split_min_keys keys, sized so the
                              whole batch covers the GPU several times over */
#define PKV_SPLIT_PAGES 1  /* every decoding sequence uses the manifest's numSplits */
#define PKV_SPLIT_FIXED 2  /* every decoding sequence uses fixed_splits (tests) */

typedef struct pkv_paged_attention_args {
  /* query  fp16 [num_tokens, query_hidden]. query_hidden = num_heads*head_size when
            key/value are given (separateKv); (num_heads + 2*kv_num_heads)*head_size for
            packed [Q | K | V] rows when key == value == NULL (packedKv). */
  const void* query;
  /* key, value  fp16 [num_tokens, kv_num_heads*head_size] or both NULL. */
  const void* key;
  const void* value;
  /* key_cache, value_cache  fp16 [num_blocks, block_size, kv_num_heads, head_size];
            updated in place by the scatter pass (the manifest's optional outputs). */
  void* key_cache;
  void* value_cache;
  /* cumulative_sequence_length int32 [batch + 1]: tokens of sequence b are rows
            [cu[b], cu[b+1]) of query. past_seqlens int32 [batch]: tokens already in
            the cache. block_table int32 [batch, max_blocks]: entry c is the physical
            block holding keys [c*block_size, (c+1)*block_size) of the sequence; -1 (or
            any id outside the pool) = unmapped. */
  const int32_t* cumulative_sequence_length;
  const int32_t* past_seqlens;
  const int32_t* block_table;
  /* slot_mapping int32 [num_tokens] or NULL: flat pool row blk*block_size + offset of
            each new token (negative = padding, not written). When NULL the scatter
            destination comes from block_table at the token's absolute position. The
            attention pass always reads keys through block_table. */
  const int32_t* slot_mapping;
  /* output fp16 [num_tokens, num_heads*head_size]. */
  void* output;
  /* optional int32 word that kernels OR PKV_DEV_* bits into (may be NULL). */
  int32_t* device_status;
  /* optional rotary of the new keys before they enter the cache (NULL = none):
            fp16 [rotary_positions, rotary_dim/2] cos / sin tables, rotation rule of the
            SparseAttention append page at the token's absolute position. */
  const void* cos_cache;
  const void* sin_cache;

  int64_t num_tokens;
  int64_t query_hidden;
  int64_t batch;
  int64_t num_heads;
  int64_t kv_num_heads;
  int64_t head_size;
  int64_t block_size;
  int64_t num_blocks;
  int64_t max_blocks;
  int64_t rotary_dim;        /* 0 = no rotary; else even and <= head_size */
  int64_t rotary_positions;  /* rows of cos_cache / sin_cache */
  int32_t rotary_interleaved;/* 0 = NeoX split pairs, 1 = interleaved pairs */
  int32_t is_causal;         /* must be 1 */
  int32_t dtype;             /* must be PKV_F16 (type constraint T = float16) */
  float scale;               /* softmax scale; 0 means 1/sqrt(head_size) */
  int32_t split_policy;      /* PKV_SPLIT_* */
  int32_t fixed_splits;      /* for PKV_SPLIT_FIXED */
  int32_t max_splits;        /* 0 = 16 (manifest MAX_SPLITS) */
  int32_t split_min_keys;    /* 0 = 128 (manifest SPLIT_MIN_KEYS) */
  /* 1 (with rotary_dim > 0): every query head of a new token is rotated at the token's
            absolute position with the key's rule and cos/sin tables before the
            attention (the append page rotates keys only; this is the query half of
            rotary attention). The rotated query is rounded to fp16 into the workspace
            (num_tokens*num_heads*head_size*2 more bytes); the query input is not
            written. A token whose position has no cos/sin row keeps its query
            unrotated (its key is skipped with PKV_DEV_BAD_POSITION). 0: keys only. */
  int32_t rotary_query;
  int32_t reserved;
} pkv_paged_attention_args;

typedef struct pkv_paged_plan {
  int32_t mode;              /* 1 = separate K/V, 2 = packed QKV */
  int32_t group_size;        /* num_heads / kv_num_heads */
  int32_t pages_num_splits;  /* the manifest's derive.numSplits for these shapes */
  int32_t max_splits;        /* per-sequence split bound used by this call */
  int64_t pages_partial_bytes; /* the manifest's pagedSplitScratchBytes at its numSplits */
  int64_t pages_stats_bytes;   /* the manifest's pagedSplitStatsBytes */
  int64_t workspace_bytes;     /* bytes pkv_paged_attention needs */
  int64_t decode_item_bound;   /* grid bound of the split-KV decode pass */
  int64_t prefill_item_bound;  /* grid bound of the tiled prefill pass */
  int64_t partial_slot_bound;  /* tokens that may need split partials */
} pkv_paged_plan;

/* Host only (no CUDA call): validates the arguments against the contract and fills
 * *plan. Returns PKV_OK or the first failing status. Pointers are checked for NULL /
 * alignment only if non-NULL values are required by the chosen mode. */
int pkv_paged_attention_plan(const pkv_paged_attention_args* args, pkv_paged_plan* plan);

/* Host only: workspace bytes pkv_paged_attention needs for these sizes. */
int pkv_paged_attention_workspace_size(const pkv_paged_attention_args* args,
                                       size_t* bytes);

/* ScatterKV + AttendSplitK + AttendSplitKMerge of the manifest, GB300 form:
 *   1. scatter: new K/V rows (rotated first when cos/sin are given) -> caches;
 *   2. plan (device): per-sequence work items; multi-token sequences become query
 *      tiles, short sequences become split-KV items;
 *   3. attention: causal GQA, token at absolute position pos sees keys 0..pos, query
 *      head hq uses kv head hq / (num_heads / kv_num_heads); tiles write the output
 *      directly, split items write fp32 (o, m, l) partials to the workspace;
 *   4. combine: LSE merge of the partials into output.
 * When every sequence has one split (the resolved split bound is 1: short caches under
 * PKV_SPLIT_AUTO, max_splits = 1, fixed_splits = 1, or a manifest numSplits of 1) and
 * the call is small (ceil(num_tokens * group / 16) * max_blocks * block_size <= 2^18),
 * the manifest's non-split form (ScatterKV then Attend) runs as ONE launch: each CTA
 * scatters one (sequence, kv head)'s new rows and attends all of that pair's query rows;
 * no partials, no combine. Larger one-split calls skip only the combine.
 * workspace: device memory of at least pkv_paged_attention_workspace_size bytes,
 * 256-byte aligned, owned by the caller, contents need not be initialised and are
 * scratch after the call. Supported: head_size in {64, 128}; num_heads/kv_num_heads
 * <= 16; any block_size >= 1. Otherwise PKV_ERR_UNSUPPORTED. */
int pkv_paged_attention(const pkv_paged_attention_args* args, void* workspace,
                        size_t workspace_bytes, void* stream);

/* Paged attention without a caller-provided workspace. The pages have no counterpart
 * to this call: it serves callers that may not allocate device memory (for example an
 * engine plugin whose enqueue step must not allocate, or a framework that has given
 * all device memory to its own pool). Scratch comes from a __device__ array of
 * PKV_STATIC_WORKSPACE_BYTES inside this library, which every GPU that loads the
 * library holds until the process exits; the call itself allocates nothing.
 *   - Same arguments, results and status codes as pkv_paged_attention; returns
 *     PKV_ERR_WORKSPACE when pkv_paged_attention_workspace_size exceeds
 *     PKV_STATIC_WORKSPACE_BYTES.
 *   - The first call on a device looks up the array's device address (a runtime
 *     call, once per device, with that device current): make that first call before
 *     any stream capture. With CUDA's default lazy module loading that first call is
 *     also when the library's device code is loaded on the device and the array's
 *     memory is committed: make it before a caller's own pool reserves the device's
 *     memory (or load modules eagerly, CUDA_MODULE_LOADING=EAGER), else it fails with
 *     PKV_ERR_LAUNCH.
 *   - The address is cached per device for the life of the process: a device reset
 *     (cudaDeviceReset) after the first call is not supported, because the reloaded
 *     module may place the array elsewhere.
 *   - All calls on a device share the one array and it keeps the last call's contents;
 *     nothing in it needs to start at zero. Calls whose work overlaps on the GPU (other
 *     streams, other threads) race on it: serialise them. */
#define PKV_STATIC_WORKSPACE_BYTES (32u << 20)
int pkv_paged_attention_static_workspace(const pkv_paged_attention_args* args,
                                         void* stream);

/* The ScatterKV pass alone (same argument block; query is read only in packed mode,
 * output and the attention fields are ignored). Bit-exact copy when rotary_dim == 0. */
int pkv_paged_scatter_kv(const pkv_paged_attention_args* args, void* stream);

/* Shape-level contract check of the manifest (host only). Each tensor is described
 * by presence, rank, dtype (pkv_dtype) and up to 4 dims. On return *failed holds
 * PKV_PRED_* bits of the predicates that are false and *mode is 1 (separate),
 * 2 (packed) or 0 (neither). Returns PKV_OK when pagedContractOk holds, a mode
 * exists and is_causal == 1; else the status of the first failure. */
typedef struct pkv_tensor_desc {
  int32_t present;
  int32_t rank;
  int32_t dtype;
  int32_t reserved;
  int64_t dims[4];
} pkv_tensor_desc;

typedef struct pkv_paged_shapes {
  pkv_tensor_desc query, key, value, key_cache, value_cache;
  pkv_tensor_desc cumulative_sequence_length, past_seqlens, block_table, slot_mapping;
  pkv_tensor_desc output;
  int64_t num_heads;
  int64_t kv_num_heads;
  int32_t is_causal;
  int32_t reserved;
} pkv_paged_shapes;

#define PKV_PRED_CACHE_SHAPE 1u
#define PKV_PRED_HEAD_LAYOUT 2u
#define PKV_PRED_SCHEDULE_SHAPE 4u
#define PKV_PRED_IO_SHAPE 8u
#define PKV_PRED_SEPARATE_KV 16u
#define PKV_PRED_PACKED_KV 32u
#define PKV_PRED_SLOT_SHAPE 64u

int pkv_paged_contract_check(const pkv_paged_shapes* shapes, uint32_t* failed,
                             int32_t* mode);

/* ---------------------------------------------------------------------------------
 * KV append + RoPE into a [batch, kv_heads, max_cache_seq, head] cache
 * (SparseAttention append page)
 * ------------------------------------------------------------------------------- */
typedef struct pkv_kv_append_args {
  /* source fp16: packed [batch*seq_len, (num_heads + 2*kv_num_heads)*head_size] rows
     [Q | K | V] when packed != 0, else key rows [batch*seq_len, kv_num_heads*head_size]. */
  const void* source;
  const void* value;                         /* separate mode: [batch*seq_len, kv*head] */
  const int32_t* total_sequence_length;      /* device scalar: == seq_len -> prompt mode */
  const int32_t* key_total_sequence_lengths; /* [batch]: history = total - seq_len */
  const void* cos_cache;                     /* fp16 [rotary_positions, rotary_dim/2] */
  const void* sin_cache;
  void* present_key;                         /* fp16 [batch, kv, max_cache_seq, head] */
  void* present_value;
  int32_t* device_status;                    /* optional */
  int64_t batch;
  int64_t seq_len;
  int64_t num_heads;
  int64_t kv_num_heads;
  int64_t head_size;
  int64_t max_cache_seq;
  int64_t rotary_dim;                        /* 0 = plain copy; else even, <= head_size */
  int64_t rotary_positions;
  int32_t packed;
  int32_t interleaved;
  int32_t dtype;                             /* PKV_F16 */
  int32_t reserved;
  /* optional query rotation (query_out NULL: none). The num_heads query heads of each
     new row, read from the packed row's leading heads or, in separate mode, from
     `query` [batch*seq_len, num_heads*head_size], are rotated at the row's position
     with K's rule and tables and written to query_out fp16 [batch*seq_len,
     num_heads*head_size]; with rotary_dim == 0, or at a position without a cos/sin
     row, the row is copied unrotated. The page rotates keys only; the query half
     uses nothing it does not define. Independent of max_cache_seq. */
  const void* query;
  void* query_out;
} pkv_kv_append_args;

/* For each (batch b, kv head h, new token t): position = history(b) + t with the
 * sparse_schedule rule (both totals read as u32); K rotated at that position when
 * rotary_dim > 0 (leading member own*cos - partner*sin, trailing own*cos +
 * partner*sin, fp32 math, fp16 round-to-nearest-even), V copied; written to row
 * `position` of (b, h). Rows no new token lands on are untouched. position >=
 * max_cache_seq (or >= rotary_positions when rotating) skips the row and sets
 * PKV_DEV_BAD_POSITION. With query_out, the query heads are rotated the same way.
 * query_out must not overlap the source or the caches. */
int pkv_kv_append_rotary(const pkv_kv_append_args* args, void* stream);

/* ---------------------------------------------------------------------------------
 * Block-sparse partials (sparse_attention_forward.wgsl)
 * ------------------------------------------------------------------------------- */
typedef struct pkv_sparse_args {
  const void* q;               /* [num_queries, hq, head_dim], element type `dtype`;
                                  may be NULL when num_queries is 0 */
  const void* k_pages;         /* [num_pages, hkv, page_size, head_dim], `dtype` */
  const void* v_pages;
  const int32_t* edge_meta;    /* [num_edges, 5]: q_idx, h (kv head), blk, batch, block_len */
  const int32_t* block_tables; /* [num_seqs, max_pages]: page id or -1 (unmapped) */
  float* o_partial;            /* [num_edges*qhead, head_dim]; 16-byte aligned (the
                                  fp16 path stores 32 bytes a lane when it is 32-byte
                                  aligned, which is faster) */
  float* m_partial;            /* [num_edges*qhead] */
  float* l_partial;            /* [num_edges*qhead] */
  int32_t* device_status;      /* optional */
  int64_t num_queries;
  int64_t num_edges;
  int64_t num_seqs;
  int64_t max_pages;
  int64_t num_pages;
  int64_t qhead;               /* query heads per kv head; hq = hkv * qhead */
  int64_t hq;
  int64_t hkv;
  int64_t head_dim;
  int64_t block_size;          /* keys per block (<= page_size * pages_per_block) */
  int64_t page_size;
  int64_t pages_per_block;
  float softmax_scale;
  /* element type of q, k_pages, v_pages: PKV_F32 (0 is taken as PKV_F32) or PKV_F16.
     The partials are fp32 either way. */
  int32_t dtype;
  /* optional [num_queries] int32: absolute position of each query in its sequence
     (right-aligned causal; the page leaves it unimplemented). Key t of block blk takes
     part only when blk*block_size + t <= position; right-aligned queries of a sequence
     with n queries and used length u sit at u - n + i. NULL: no causal mask. */
  const int32_t* query_positions;
} pkv_sparse_args;

/* Host only: workspace bytes of pkv_sparse_attention_partials: the edge grouping and,
 * for fp32 calls whose shape runs on the tensor core (head_dim 64/128, block_size <= 64,
 * page_size a multiple of 8 with pages_per_block * page_size <= 64), the Q rows split
 * into fp16 (hi, lo) pairs: 4 * head_dim + 4 bytes per (query, head) row. */
int pkv_sparse_attention_partials_workspace_size(const pkv_sparse_args* args,
                                                 size_t* bytes);

/* One partial per (edge e, lane qh), index e*qhead + qh: query row q[q_idx, h*qhead+qh];
 * key t < block_len of block blk lives in page slot blk*pages_per_block + t/page_size
 * of the sequence's table row, row t % page_size; unmapped page -> score -1e30.
 * s = softmax_scale * <q, k>; m = max s (>= -1e30); weights exp(s - m) for s > -5e29
 * else 0; l = sum of weights; o = weighted sum of value rows (unnormalised).
 * block_len <= 0 -> (o = 0, m = -1e30, l = 0). No causal mask unless query_positions
 * is given. fp32 throughout for dtype PKV_F32.
 * The GPU form groups edges by (batch, kv head, block) so each K/V block is read
 * once for all edges that name it. Supported: head_dim in {64, 128}, block_size
 * <= 128, qhead <= 64.
 * dtype PKV_F16 (the page computes in fp32; this is the half-precision variant): scores
 * are fp16 products summed in fp32, the weights are computed in fp32 and summed into l,
 * and rounded once to fp16 for the weighted sum of value rows; the partials are fp32;
 * everything else as above.
 * fp32 on the tensor core: each Q row and each K / V block is scaled by a power of two
 * and split into fp16 (hi, lo) pairs, and every product is formed from three fp16 MMAs
 * with fp32 accumulation (hi*hi + hi*lo + lo*hi), about 2^-21 of |q||k| per score.
 * Supported for fp16: head_dim in {64, 128}, block_size <= 64, page_size a multiple of
 * 8 with pages_per_block * page_size <= 64; else PKV_ERR_UNSUPPORTED.
 * With query_positions the keys after the query's position take no part (they are not
 * read and flag nothing); an edge left with no key gets the empty partial. */
int pkv_sparse_attention_partials(const pkv_sparse_args* args, void* workspace,
                                  size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------------
 * Combine of (o, m, l) partials
 * ------------------------------------------------------------------------------- */
typedef struct pkv_combine_args {
  const float* o;              /* [num_partials, head_dim] unnormalised */
  const float* m;              /* [num_partials] running max (natural-log units) */
  const float* l;              /* [num_partials] sum of exp(s - m) */
  const int32_t* segment_offsets; /* [num_segments + 1] CSR over partial groups, or NULL */
  void* out;                   /* [num_segments*lanes, head_dim], dtype out_dtype */
  float* lse;                  /* optional [num_segments*lanes]: M + ln L, -inf if empty */
  int64_t num_segments;
  int64_t lanes;               /* partials per group (e.g. query heads per kv head) */
  int64_t head_dim;
  int64_t uniform_count;       /* groups per segment when segment_offsets == NULL */
  int32_t out_dtype;           /* PKV_F16 or PKV_F32 */
  int32_t reserved;
} pkv_combine_args;

/* Output row s*lanes + c merges partial rows e*lanes + c for groups e in
 * [off[s], off[s+1]) (or [s*uniform_count, (s+1)*uniform_count)): over partials with
 * l > 0, M = max m, w = exp(m - M), L = sum w*l, out = sum w*o / L, lse = M + ln L.
 * A partial with l == 0 is empty and its o row is not read. No non-empty partial:
 * out = 0, lse = -inf. Supported: head_dim in {64, 128}. */
int pkv_combine_partials(const pkv_combine_args* args, void* stream);

/* ---------------------------------------------------------------------------------
 * Schedule: block tables and slot maps from request lengths
 * ------------------------------------------------------------------------------- */
typedef struct pkv_schedule_args {
  const int32_t* past_seqlens;   /* [batch] tokens of each row already in the cache */
  const int32_t* new_seqlens;    /* [batch] tokens the row takes in now (0: idle row) */
  /* [batch, max_blocks], updated in place. Row b holds its first
     ceil(past_seqlens[b] / block_size) entries: these are read (an entry of -1 is a hole,
     skipped; rows may share blocks). The entries behind them, up to
     ceil((past + new) / block_size), are written; later ones stay as they are. */
  int32_t* block_table;
  /* outputs; all but the first may be NULL */
  int32_t* cumulative_sequence_length;  /* [batch + 1] granted tokens before each row */
  int32_t* slot_mapping;         /* [num_tokens] block * block_size + offset of each token;
                                    -1 past the last granted token */
  int32_t* positions;            /* [num_tokens] past + t of each token, -1 past the last */
  int32_t* total_seqlens;        /* [batch] past + granted tokens (the next past) */
  int32_t* free_blocks;          /* [1] blocks of the pool that no row holds afterwards */
  int32_t* device_status;        /* optional */
  int64_t batch;
  int64_t max_blocks;
  int64_t num_blocks;            /* blocks of the pool */
  int64_t block_size;
  int64_t num_tokens;            /* length of slot_mapping and positions */
} pkv_schedule_args;

/* A block is in use when some row holds it; every other block of the pool is free, so a
 * finished request gives its blocks back by a past of 0. Row b needs
 * ceil((past + new) / block_size) - ceil(past / block_size) blocks; counted over the rows
 * in order, the r-th block asked for is the r-th free block by number. A row is granted all
 * of its new tokens or none:
 *   - rows are granted in order while the blocks asked for up to and including the row fit
 *     the free ones; a row behind that is granted only if it needs no block
 *     (PKV_DEV_NO_BLOCKS when one is not);
 *   - and while the tokens of the rows up to it that the pool takes fit num_tokens: from the first
 *     one that does not on, no row that brings tokens is granted any (PKV_DEV_BAD_SEQUENCE);
 *   - a negative length (PKV_DEV_BAD_SEQUENCE), a past + new beyond max_blocks *
 *     block_size (PKV_DEV_BAD_BLOCK) are granted nothing; a negative past holds nothing.
 * A row that is granted nothing keeps its table row; total_seqlens gives its past back.
 * A held entry outside the pool counts as a hole and sets PKV_DEV_BAD_BLOCK; a token
 * whose held block is a hole gets slot -1 and sets PKV_DEV_BAD_BLOCK.
 * The result depends on the inputs alone; a second call with the same inputs gives the same.
 * past_seqlens and new_seqlens must not overlap the outputs. No workspace. Supported:
 * batch <= 8192, num_blocks <= 2^20; num_blocks * block_size, batch * max_blocks and
 * num_tokens below 2^31, max_blocks * block_size below 2^31 - 16; otherwise
 * PKV_ERR_UNSUPPORTED. */
int pkv_paged_schedule(const pkv_schedule_args* args, void* stream);

/* ---------------------------------------------------------------------------------
 * Paged append with rotary positions of several axes
 * ------------------------------------------------------------------------------- */
#define PKV_MAX_ROTARY_AXES 8
#define PKV_MAX_ROTARY_PAIRS 128

typedef struct pkv_append_axes_args {
  /* rows of num_tokens tokens, `dtype`: separate mode query [num_tokens, num_heads *
     head_size] (NULL with query_out NULL: no queries), key and value [num_tokens,
     kv_num_heads * head_size]; packed mode (key == value == NULL) query holds
     [Q | K | V] rows of (num_heads + 2 * kv_num_heads) * head_size. */
  const void* query;
  const void* key;
  const void* value;
  void* query_out;               /* [num_tokens, num_heads * head_size] or NULL: queries
                                    are not rotated */
  void* key_cache;               /* [num_blocks, block_size, kv_num_heads, head_size] */
  void* value_cache;
  const int32_t* slot_mapping;   /* [num_tokens] flat pool row; negative = padding */
  const int32_t* positions;      /* [num_axes, num_tokens] (may be NULL without rotary) */
  const void* cos_cache;         /* [rotary_positions, rotary_dim / 2], `table_dtype` */
  const void* sin_cache;
  int32_t* device_status;        /* optional */
  int64_t num_tokens;
  int64_t num_heads;
  int64_t kv_num_heads;
  int64_t head_size;
  int64_t block_size;
  int64_t num_blocks;
  int64_t rotary_dim;            /* 0 = plain copy; else even, <= head_size */
  int64_t rotary_positions;
  int32_t num_axes;              /* 1 .. PKV_MAX_ROTARY_AXES when rotary_dim > 0 */
  int32_t rotary_interleaved;    /* 0: element i pairs with i + rotary_dim / 2, 1: 2i with
                                    2i + 1 */
  int32_t dtype;                 /* PKV_F16 or PKV_BF16 */
  int32_t table_dtype;           /* `dtype` or PKV_F32 */
  uint8_t pair_axis[PKV_MAX_ROTARY_PAIRS];  /* axis of pair i < rotary_dim / 2 */
} pkv_append_axes_args;

/* For token i with slot s = slot_mapping[i] >= 0: pair j of every key (and, with query_out,
 * query) head turns by the angle whose cos and sin stand in table row
 * positions[pair_axis[j]][i], column j:
 *   leading member own*cos - partner*sin, trailing member own*cos + partner*sin,
 * in 32-bit arithmetic, rounded once to `dtype`; elements from rotary_dim on are copied.
 * The key row goes to pool row s of key_cache, the value row to value_cache, the query row
 * to row i of query_out. A negative slot is padding: whatever the token's rows and
 * positions hold, nothing is written for it. A slot past the pool (PKV_DEV_BAD_SLOT): K
 * and V are not written, the query is. A position outside [0, rotary_positions) on an axis
 * that some pair uses (PKV_DEV_BAD_POSITION): K and V are not written, the query row is
 * copied unrotated. Two tokens of one slot leave there, in each 16 bytes, the one's or the
 * other's. query_out and the caches must not overlap the inputs or one another. head_size a
 * multiple of 8, <= 256; otherwise PKV_ERR_UNSUPPORTED.
 * pkv_paged_attention reads fp16 pools alone. A bf16 pool is read by pkv_paged_window_attention
 * and pkv_paged_prefix_attention, and by pkv_cross_attention, which has no causal mask. */
int pkv_paged_append_rotary_axes(const pkv_append_axes_args* args, void* stream);

/* ---------------------------------------------------------------------------------
 * Cross attention over a paged cache of encoder states
 * ------------------------------------------------------------------------------- */
typedef struct pkv_cross_attention_args {
  const void* query;             /* [num_tokens, num_heads * head_size], `dtype` */
  const void* key_cache;         /* [num_blocks, block_size, kv_num_heads, head_size] */
  const void* value_cache;
  const int32_t* cumulative_sequence_length;  /* [batch + 1] query rows of each sequence */
  const int32_t* key_seqlens;    /* [batch] encoder states of each sequence (may be 0) */
  const int32_t* block_table;    /* [batch, max_blocks], -1 (or any id outside the pool) =
                                    unmapped */
  void* output;                  /* [num_tokens, num_heads * head_size], `dtype` */
  float* lse;                    /* optional [num_tokens, num_heads] */
  int32_t* device_status;        /* optional */
  int64_t num_tokens;
  int64_t batch;
  int64_t num_heads;
  int64_t kv_num_heads;
  int64_t head_size;
  int64_t block_size;
  int64_t num_blocks;
  int64_t max_blocks;
  /* upper bound on the query rows of a sequence, 0 = num_tokens. A step of single tokens
     that says so (1) leaves out the kernel for many rows. */
  int64_t max_query_len;
  int32_t dtype;                 /* PKV_F16 or PKV_BF16 */
  float scale;                   /* softmax scale; 0 means 1/sqrt(head_size) */
} pkv_cross_attention_args;

/* Host only: workspace bytes pkv_cross_attention needs on the current device; 0 where few and
 * short sequences need none (workspace may then be NULL). */
int pkv_cross_attention_workspace_size(const pkv_cross_attention_args* args, size_t* bytes);

/* Query row i of sequence b, head hq with kv head h = hq / (num_heads / kv_num_heads), over
 * the n = key_seqlens[b] states of its table row:
 *   s_j = scale * <q, k_j>, lse = ln sum_j e^{s_j}, output = sum_j e^{s_j - lse} v_j,
 * summed in 32 bits; the weights e^{s_j - m} are rounded once to `dtype` for the product
 * with the values (in fp16 by at most 2^-11 of each and 2^-32 of the row's largest), their sum
 * is not. A state whose block is unmapped takes no part and sets
 * PKV_DEV_BAD_BLOCK (so does an n past max_blocks * block_size, which is cut there). A row
 * that sees no state gets output 0 and lse -inf. Cache rows behind a sequence's states may
 * hold anything (NaN too). Sequences whose cumulative lengths are inconsistent or exceed
 * max_query_len, or whose key_seqlens entry is negative, get zero rows (lse -inf) and set
 * PKV_DEV_BAD_SEQUENCE; so do rows that no sequence covers, without the flag. A row that
 * two sequences claim is one's or the other's, in parts.
 * The order of summation depends on the sizes, the lengths and the device's SM count alone:
 * equal calls give equal bits. Output and lse must not overlap the inputs. workspace: as in
 * pkv_paged_attention (256-byte aligned, contents need not be initialised, one per call in
 * flight). After PKV_DEV_TIMEOUT the rows of the tiles that gave up, and those joined from
 * their pieces, are not valid. Supported: head_size in {64, 128},
 * num_heads / kv_num_heads <= 16; otherwise PKV_ERR_UNSUPPORTED. */
int pkv_cross_attention(const pkv_cross_attention_args* args, void* workspace,
                        size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------------
 * Paged append with norms of the heads and rotary positions
 * ------------------------------------------------------------------------------- */
typedef struct pkv_append_norm_args {
  pkv_append_axes_args append;   /* as in pkv_paged_append_rotary_axes */
  const void* query_weight;      /* [head_size], `weight_dtype`; NULL: the heads of the
                                    queries are not normed */
  const void* key_weight;        /* the same for the keys */
  float epsilon;                 /* > 0 */
  int32_t weight_dtype;          /* append.dtype or PKV_F32 */
} pkv_append_norm_args;

/* pkv_paged_append_rotary_axes with a norm in front of the rotation: every head x of a key
 * (and, with query_out, of a query) becomes
 *   x_i * query_weight[i] / sqrt(sum_j x_j^2 / head_size + epsilon)
 * (key_weight for keys), which turns as there; in 32-bit arithmetic, rounded once behind the
 * rotation. Squares are summed in 32 bits: a bf16 head whose squares sum past 3.4e38 becomes
 * 0. What that call says of slots, positions, padding and overlaps holds here too; a query
 * whose position has no table row is normed and not rotated. At least one weight is given.
 * Same refusals and limits. Heads of other sizes than 64 and 128 (256 among them) are appended for
 * readers of the caller's own: the attention calls here take those two alone. */
int pkv_paged_append_norm_rotary(const pkv_append_norm_args* args, void* stream);

/* ---------------------------------------------------------------------------------
 * Causal paged attention with a sliding window, or behind a shared prefix
 * ------------------------------------------------------------------------------- */
typedef struct pkv_window_attention_args {
  const void* query;             /* [num_tokens, num_heads * head_size], `dtype` */
  const void* key_cache;         /* [num_blocks, block_size, kv_num_heads, head_size] */
  const void* value_cache;
  const int32_t* cumulative_sequence_length;  /* [batch + 1] query rows of each sequence */
  const int32_t* past_seqlens;   /* [batch] tokens in front of the sequence's first row */
  const int32_t* block_table;    /* [batch, max_blocks], -1 (or any id outside the pool) =
                                    unmapped */
  void* output;                  /* [num_tokens, num_heads * head_size], `dtype` */
  float* lse;                    /* optional [num_tokens, num_heads] */
  int32_t* device_status;        /* optional */
  int64_t num_tokens;
  int64_t batch;
  int64_t num_heads;
  int64_t kv_num_heads;
  int64_t head_size;
  int64_t block_size;
  int64_t num_blocks;
  int64_t max_blocks;
  int64_t max_query_len;         /* as in pkv_cross_attention */
  int64_t window;                /* keys that a row sees, its own included; 0: all */
  int64_t sinks;                 /* first keys of a sequence that stay visible (no effect
                                    without a window) */
  int32_t dtype;                 /* PKV_F16 or PKV_BF16 */
  float scale;                   /* softmax scale; 0 means 1/sqrt(head_size) */
} pkv_window_attention_args;

/* Host only: workspace bytes pkv_paged_window_attention needs on the current device (may be 0). */
int pkv_paged_window_attention_workspace_size(const pkv_window_attention_args* args,
                                              size_t* bytes);

/* Causal attention over the paged cache; the new tokens' keys and values are in it already (an
 * append call put them there). Query row i of sequence b stands at t = past_seqlens[b] + i and
 * sees key j <= t when window is 0, when j > t - window, or when j < sinks:
 *   s_j = scale * <q, k_j>, lse = ln sum_j e^{s_j}, output = sum_j e^{s_j - lse} v_j
 * in the arithmetic of pkv_cross_attention. A key whose block is unmapped takes no part, and
 * sets PKV_DEV_BAD_BLOCK if a row sees it (so do keys from max_blocks * block_size on); blocks that
 * no row sees any more may be given back. Cache rows that no row of the sequence sees may hold
 * anything (NaN too); a key or value that is not finite can reach all rows of its sequence.
 * A row that sees no mapped key gets output 0 and lse -inf. Sequences whose cumulative lengths
 * are inconsistent or exceed max_query_len, or whose past_seqlens entry is negative or beyond
 * max_blocks * block_size, get zero rows (lse -inf) and set PKV_DEV_BAD_SEQUENCE; so do rows
 * that no sequence covers, without the flag. Equal calls give equal bits; output, lse, workspace, PKV_DEV_TIMEOUT and the sizes
 * supported: as in pkv_cross_attention. */
int pkv_paged_window_attention(const pkv_window_attention_args* args, void* workspace,
                               size_t workspace_bytes, void* stream);

typedef struct pkv_prefix_attention_args {
  const void* query;             /* as in pkv_window_attention_args, down to device_status */
  const void* key_cache;
  const void* value_cache;
  const int32_t* cumulative_sequence_length;
  const int32_t* past_seqlens;
  const int32_t* block_table;
  const int32_t* group_offsets;  /* [num_groups + 1] group g: sequences group_offsets[g] ..
                                    group_offsets[g + 1] - 1; ascending, within 0 .. batch */
  const int32_t* shared_seqlens; /* [num_groups] first keys that all of a group's sequences
                                    have in common: the same blocks in their table rows */
  void* output;
  float* lse;
  int32_t* device_status;
  int64_t num_tokens;
  int64_t batch;
  int64_t num_groups;
  int64_t num_heads;
  int64_t kv_num_heads;
  int64_t head_size;
  int64_t block_size;
  int64_t num_blocks;
  int64_t max_blocks;
  int64_t max_query_len;
  int32_t dtype;
  float scale;
} pkv_prefix_attention_args;

/* Host only: workspace bytes pkv_paged_prefix_attention needs on the current device (may be 0). It
 * holds one output in 32 bits (num_tokens * num_heads * (head_size + 1) * 4 bytes; two where every
 * sequence has few tokens, max_query_len * num_heads / kv_num_heads <= 16) and what the kernels
 * need, where these sizes may have something to share. */
int pkv_paged_prefix_attention_workspace_size(const pkv_prefix_attention_args* args,
                                              size_t* bytes);

/* What pkv_paged_window_attention computes without a window, for sequences of which some begin
 * alike: the keys that a group shares are read through the table row of its first sequence with
 * new tokens, once for the rows of all of them, and joined in 32 bits with what each row sees
 * behind them. A group shares shared_seqlens[g] keys, or fewer where one of its sequences with new
 * tokens has a shorter past. Sequences outside all groups and groups with fewer than two
 * sequences that have new tokens share nothing, nor does a group of which one sequence is bad; and
 * where sharing would save less time than its kernels take, as the lengths tell, nothing is shared
 * (the results then differ by rounding). A negative shared_seqlens entry is taken as 0 and
 * sets PKV_DEV_BAD_SEQUENCE; group offsets that descend or leave 0 .. batch set it too, and then
 * nothing is shared at all. The table entries that a group is said to share have to be equal: where
 * they are not, a sequence's output is that of its own or of the first one's. A shared block that is
 * unmapped sets PKV_DEV_BAD_BLOCK. Equal calls give equal bits. */
int pkv_paged_prefix_attention(const pkv_prefix_attention_args* args, void* workspace,
                               size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------------
 * Fork: rows of the block table copied, reordered and freed
 * ------------------------------------------------------------------------------- */
#define PKV_MAX_FORK_CACHES 256

typedef struct pkv_fork_args {
  const int32_t* parents;        /* [batch] row that each row becomes a copy of: itself (it
                                    stays), another one, or negative (it is freed) */
  const int32_t* past_seqlens;   /* [batch] tokens of each row */
  const int32_t* block_table;    /* [batch, max_blocks] */
  int32_t* new_past_seqlens;     /* [batch] */
  int32_t* new_block_table;      /* [batch, max_blocks], written whole */
  int32_t* free_blocks;          /* optional [1] blocks of the pool that no row holds now */
  void* const* caches;           /* HOST array of num_caches device pointers: pools of
                                    num_blocks * block_size rows (keys and values of every
                                    layer, any type) */
  const int64_t* cache_row_bytes;  /* HOST array: bytes of a token's row in each */
  int32_t* device_status;        /* optional */
  int64_t batch;
  int64_t max_blocks;
  int64_t num_blocks;
  int64_t block_size;
  int64_t num_caches;            /* 0: tables only */
} pkv_fork_args;

/* Host only: workspace bytes pkv_paged_fork needs. */
int pkv_paged_fork_workspace_size(const pkv_fork_args* args, size_t* bytes);

/* New row b takes over the n = past_seqlens[p] tokens of old row p = parents[b]: its first
 * n / block_size entries are p's (whole blocks are shared), and where n ends inside a block
 * one of p's copies (row p itself if it stays, else the first) keeps that block, the others
 * get one of their own, whose first n % block_size rows are copied from it in every cache.
 * Entries behind are -1. A block of the pool that no new row holds is free, so what freed and
 * replaced rows alone held is given back; the r-th row that needs a block gets the r-th free
 * one by number. A row for which there is none is freed (PKV_DEV_NO_BLOCKS), as is one whose
 * parent is no row, or has a negative length (PKV_DEV_BAD_SEQUENCE) or one beyond max_blocks *
 * block_size (PKV_DEV_BAD_BLOCK). A freed row has length 0 and entries of -1. An entry outside
 * the pool is copied as it is (any but -1 sets PKV_DEV_BAD_BLOCK); where it stands for the
 * block that would be copied, nothing is. Rows that shared a partly filled block before go on
 * sharing it. Rows of the caches other than those copied to are not written; the result
 * depends on the inputs alone. The outputs must not overlap the inputs. The host arrays are read during
 * the call. Supported: cache_row_bytes and cache pointers multiples of 16, num_caches <=
 * PKV_MAX_FORK_CACHES, the sizes of pkv_paged_schedule and rows of a cache below 2^31 / block_size
 * bytes; otherwise PKV_ERR_UNSUPPORTED (pointers: PKV_ERR_ALIGN). */
int pkv_paged_fork(const pkv_fork_args* args, void* workspace, size_t workspace_bytes,
                   void* stream);

/* ---------------------------------------------------------------------------------
 * Runtime utilities
 * ------------------------------------------------------------------------------- */
int pkv_abi_version(void);
const char* pkv_status_string(int status);
/* sizeof of each argument struct, so a binding can check its layout. */
size_t pkv_sizeof_struct(const char* name);
/* Kernels this library has launched since load (all entry points, all streams). */
int64_t pkv_launch_count(void);
/* Per-kernel timing: when enabled, every launch is bracketed by CUDA events on its own
 * stream; pkv_profiler_query synchronises those events and returns the summed device
 * time (ms) and launch count of `kernel` ("scatter", "append", "plan", "decode",
 * "prefill", "combine", "sparse_group", "sparse_partials", "schedule", "append_axes",
 * "cross_decode", "cross_tiles", "cross_combine", "append_norm", "window_decode",
 * "window_tiles", "window_combine", "prefix_plan", "prefix_decode", "prefix_tiles",
 * "prefix_combine", "fork_plan", "fork_copy"). Not thread-safe. */
void pkv_profiler_enable(int on);

/* Testing hook for the give-up path of the tensor-core kernels' bounded waits (the
 * tcgen05 prefill, the two block-sparse partial kernels and the kernel for many rows of the
 * cross, window and prefix attention). The pages have no
 * counterpart. max_polls replaces the default poll bound of every such wait (0 restores
 * the default); with withhold_first_copy != 0 (which needs max_polls > 0) every CTA of
 * those kernels announces its first bulk copy (the first K box of its first prefill
 * tile, or its first K/V staging) on the copy's barrier but never issues it, so the wait
 * for it gives up with no copy or MMA of that data in flight. A CTA whose wait gave up
 * ORs PKV_DEV_TIMEOUT into device_status, waits (bounded) for what it did issue, frees
 * its tensor memory and returns; outputs it had not written stay unwritten. Applies to
 * calls made after it, process-wide; not thread-safe; for tests only. Returns PKV_OK,
 * or PKV_ERR_SHAPE for withhold_first_copy without a bound. */
int pkv_testing_wait_limit(uint32_t max_polls, int32_t withhold_first_copy);
/* Testing hook for pkv_paged_prefix_attention: mode 1 shares whatever can be shared, 2 shares
 * nothing, whether it saves anything or not; 0 restores the rule. The workspace size follows it.
 * Applies to calls made after it, process-wide; for tests only. Returns PKV_OK, or PKV_ERR_SHAPE
 * for another mode. */
int pkv_testing_prefix_sharing(int32_t mode);
void pkv_profiler_reset(void);
int pkv_profiler_query(const char* kernel, double* total_ms, int64_t* launches);

#ifdef __cplusplus
}
#endif

#endif /* PAGEDKV_H */
