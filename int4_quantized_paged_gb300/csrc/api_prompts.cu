// C ABI of the operators for long and shared prompts: argument validation,
// workspaces and dispatch; everything here runs on the host.
#include <cuda_runtime.h>
#include <stdint.h>

#include "api_common.h"
#include "kvq.h"
#include "kvq_internal.h"

using namespace kvq;

namespace {

size_t align16(size_t n) { return (n + 15) & ~(size_t)15; }

// Whether two arrays of ints have an entry in common.
bool overlap(const int* a, int na, const int* b, int nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + (uintptr_t)nb * sizeof(int) && y < x + (uintptr_t)na * sizeof(int);
}

// Bytes of the decode kernel's partials and of the items' offsets in its tile list.
size_t partial_bytes(const kvq_config& c, int batch, int workers) {
  const size_t items = (size_t)batch * c.num_kv_heads, slots = items + (size_t)workers;
  const size_t G = c.num_q_heads / c.num_kv_heads;
  return align16(slots * G * (c.head_dim + 2) * sizeof(float) + (items + 1) * sizeof(long long));
}

// The partials' places in a workspace of partial_bytes.
void place_partials(const kvq_config& c, DecodeArgs* a, uint8_t* at) {
  const size_t slots = (size_t)a->B * c.num_kv_heads + (size_t)a->workers;
  const size_t rows = slots * (c.num_q_heads / c.num_kv_heads);
  a->ws_o = reinterpret_cast<float*>(at);
  a->ws_ml = a->ws_o + rows * c.head_dim;
  a->item_tiles = reinterpret_cast<long long*>(a->ws_ml + rows * 2);
}

// The arguments that the decode calls of this file have in common: checked, and put
// into *a.
kvq_status decode_args(const kvq_ctx* ctx, int layer, const void* q, const void* k_cache,
                       const void* v_cache, const float* k_scale, const float* v_scale,
                       const float* k_cache_scale, const float* v_cache_scale,
                       const int* block_table, int max_blocks_per_seq, const int* context_lens,
                       int batch, int max_context, void* out, DecodeArgs* a) {
  const kvq_config& c = ctx->cfg;
  const int mode = ctx->mode[layer];
  if ((long long)max_context > (long long)max_blocks_per_seq * c.block_size)
    return KVQ_ERR_INVALID_ARG;
  if (!q || !k_cache || !v_cache || !block_table || !context_lens || !out)
    return KVQ_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) ||
      !aligned4(block_table) || !aligned4(context_lens))
    return KVQ_ERR_ALIGNMENT;
  if ((mode == KVQ_FP8_PER_TENSOR || mode == KVQ_FP8_PER_HEAD) && (!k_scale || !v_scale))
    return KVQ_ERR_INVALID_ARG;
  if (is_dynamic(mode)) {
    if (!k_cache_scale || !v_cache_scale) return KVQ_ERR_INVALID_ARG;
    // the kernels fetch 16 scales at a time by bulk copies
    if (!aligned16(k_cache_scale) || !aligned16(v_cache_scale)) return KVQ_ERR_ALIGNMENT;
  }
  *a = {};
  a->q = static_cast<const uint16_t*>(q);
  a->k_cache = static_cast<const uint8_t*>(k_cache);
  a->v_cache = static_cast<const uint8_t*>(v_cache);
  a->k_scale = k_scale;
  a->v_scale = v_scale;
  a->k_cs = k_cache_scale;
  a->v_cs = v_cache_scale;
  a->block_table = block_table;
  a->context_lens = context_lens;
  a->out_bf16 = static_cast<uint16_t*>(out);
  a->B = batch;
  a->Hq = c.num_q_heads;
  a->Hkv = c.num_kv_heads;
  a->bs = c.block_size;
  a->bs_shift = __builtin_ctz((unsigned)c.block_size);
  a->max_blocks = max_blocks_per_seq;
  a->cap = (long long)max_blocks_per_seq * c.block_size;
  a->num_blocks = c.num_blocks;
  a->qk_scale = ctx->softmax_scale * 1.4426950408889634f;
  return KVQ_OK;
}

// Pages that cannot stay in L2 until the next step are streamed evict-first.  `positions`
// of every row count: a prefix that rows share counts for each of them (counting it once
// made no difference of more than 2 % on groups of 2 to 64 rows, L2 warm or cold).
int stream_once(const kvq_ctx* ctx, int layer, int batch, long long positions) {
  const kvq_config& c = ctx->cfg;
  const int mode = ctx->mode[layer];
  const double bytes = (double)batch * c.num_kv_heads * (double)positions *
                       (2.0 * (double)row_bytes(mode, c.head_dim) + (is_dynamic(mode) ? 8 : 0));
  return bytes > 64.0 * 1024 * 1024;
}

constexpr long long kMostWorkers = 4LL * 65535 * 64;

// Sizes of a call behind shared prefixes: splits of a prefix at most (0 in: the plan's
// choice), workers of the rows' own positions, and the parts of the workspace.
struct SharedPlan {
  int splits, workers;
  int units, unit_rows;          // as in SharedArgs
  size_t rows;                   // partial rows of the prefixes
  size_t index_bytes, unit_bytes, prefix_bytes, own_bytes;
  size_t bytes() const { return index_bytes + unit_bytes + prefix_bytes + own_bytes; }
};

kvq_status plan_shared(const kvq_ctx* ctx, int layer, int batch, int num_groups, int max_group,
                       int max_shared, int max_own, int num_splits, SharedPlan* p) {
  kvq_status st = check_layer(ctx, layer);
  if (st != KVQ_OK) return st;
  if (ctx->window[layer] != 0) return KVQ_ERR_UNSUPPORTED;
  if (batch < 0 || num_groups < 0 || max_group < 0 || max_shared < 0 || max_own < 0 ||
      max_shared >= (1 << 30) || max_own >= (1 << 30) || num_splits < 0 || num_splits > 1024)
    return KVQ_ERR_INVALID_ARG;
  const kvq_config& c = ctx->cfg;
  if (max_group > batch) max_group = batch;
  *p = {};
  bool share = num_groups > 0 && max_group > 1 && max_shared >= 16;
  // nothing to gain, were every row to share the longest prefix (the device's own test
  // would only find so behind the launch of the pass, some 4 us)
  if (num_splits == 0 && 2.0 * batch * ((max_shared + 63) / 64) * c.num_kv_heads <
                             5.0 * (SHARED_PASS + 4) * sm_count())
    share = false;
  if (share) {
    const int tile = cross_query_tile(c.head_dim, c.num_q_heads / c.num_kv_heads);
    // units of one split, in steps whose products fit 64 bits
    const long long base = ((long long)max_group + tile - 1) / tile * num_groups;
    if (base >= (1LL << 31)) return KVQ_ERR_INVALID_ARG;
    const int tiles = (int)(((long long)max_shared + CROSS_KEYS - 1) / CROSS_KEYS);
    // one wave over the SMs, or two units for each group where they are more than that
    const long long wave = (sm_count() + c.num_kv_heads - 1) / c.num_kv_heads;
    p->splits = num_splits > 0 ? num_splits : (int)(tiles < wave ? tiles : wave);
    long long units = base * p->splits;
    const long long most = 2 * base > wave ? 2 * base : wave;
    if (units > most) units = most;
    if (units >= (1LL << 31) / c.num_kv_heads) return KVQ_ERR_INVALID_ARG;
    p->units = (int)units;
    p->unit_rows = max_group < tile ? max_group : tile;
    if (units >= (1LL << 34) / p->unit_rows / c.num_q_heads) return KVQ_ERR_INVALID_ARG;
    p->rows = (size_t)units * p->unit_rows * c.num_q_heads;
  }
  // a row that reads its prefix alone has all of its positions as its own
  int workers = 0;
  st = kvq_decode_plan(ctx, layer, batch, max_shared + max_own, &workers, nullptr);
  if (st != KVQ_OK) return st;
  p->workers = workers;
  p->index_bytes = align16(((size_t)batch * 2 + (size_t)num_groups * 3 + 1) * sizeof(int));
  p->unit_bytes = (size_t)p->units * sizeof(int4);
  p->prefix_bytes = align16(p->rows * (c.head_dim + 1) * sizeof(float));
  p->own_bytes = partial_bytes(c, batch, workers);
  return KVQ_OK;
}

}  // namespace

extern "C" {

kvq_status kvq_prompt_attention(const kvq_ctx* ctx, int layer, const void* q,
                                long long q_token_stride, const void* k, const void* v,
                                long long kv_token_stride, const int* seq_start, int batch,
                                int max_seq_len, long long num_tokens, void* out, void* stream) {
  kvq_status st = check_layer(ctx, layer);
  if (st != KVQ_OK) return st;
  if (batch < 0 || max_seq_len < 0 || num_tokens < 0 || num_tokens >= (1LL << 31) - 256)
    return KVQ_ERR_INVALID_ARG;
  if (batch == 0 || max_seq_len == 0 || num_tokens == 0) return KVQ_OK;
  const kvq_config& c = ctx->cfg;
  const long long QD = (long long)c.num_q_heads * c.head_dim;
  const long long KD = (long long)c.num_kv_heads * c.head_dim;
  const long long qs = q_token_stride == 0 ? QD : q_token_stride;
  const long long ks = kv_token_stride == 0 ? KD : kv_token_stride;
  // a tensor map's stride stays below 2^40 bytes
  if (!q || !k || !v || !seq_start || !out || qs < QD || ks < KD || qs >= (1LL << 39) ||
      ks >= (1LL << 39))
    return KVQ_ERR_INVALID_ARG;
  if (qs % 8 != 0 || ks % 8 != 0 || !aligned16(q) || !aligned16(k) || !aligned16(v) ||
      !aligned16(out) || !aligned4(seq_start))
    return KVQ_ERR_ALIGNMENT;
  const int G = c.num_q_heads / c.num_kv_heads;
  const long long most = max_seq_len < num_tokens ? max_seq_len : num_tokens;
  if (prompt_items(c.head_dim, G, num_tokens, most, batch, 1) >= (1LL << 31) / c.num_kv_heads)
    return KVQ_ERR_INVALID_ARG;
  unsigned* err = error_word();
  if (!err) return KVQ_ERR_CUDA;
  PromptArgs a = {};
  a.q = static_cast<const uint16_t*>(q);
  a.seq_start = seq_start;
  a.out = static_cast<uint16_t*>(out);
  a.err = err;
  a.T = num_tokens;
  a.B = batch;
  a.Hq = c.num_q_heads;
  a.Hkv = c.num_kv_heads;
  a.g_shift = __builtin_ctz((unsigned)G);
  a.max_len = (int)most;
  a.window = ctx->window[layer];
  a.qk_scale = ctx->softmax_scale * 1.4426950408889634f;
  return cuda_status(
      launch_prompt(c.head_dim, a, qs, k, v, ks, static_cast<cudaStream_t>(stream)));
}

// ---------------------------------------------------------------- shared prefixes
kvq_status kvq_shared_prefix_plan(const kvq_ctx* ctx, int layer, int batch, int num_groups,
                                  int max_group, int max_shared, int max_own, int* num_splits,
                                  size_t* workspace_bytes) {
  if (!num_splits) return KVQ_ERR_INVALID_ARG;
  SharedPlan p;
  const kvq_status st = plan_shared(ctx, layer, batch, num_groups, max_group, max_shared, max_own,
                                    *num_splits, &p);
  if (st != KVQ_OK) return st;
  if (p.units == 0) *num_splits = 0;
  if (workspace_bytes) *workspace_bytes = p.bytes();
  return KVQ_OK;
}

kvq_status kvq_shared_prefix_attention(const kvq_ctx* ctx, int layer, const void* q,
                                       const void* k_cache, const void* v_cache,
                                       const float* k_scale, const float* v_scale,
                                       const float* k_cache_scale, const float* v_cache_scale,
                                       const int* block_table, int max_blocks_per_seq,
                                       const int* context_lens, int batch, const int* group_start,
                                       const int* shared_lens, int num_groups, int max_group,
                                       int max_shared, int max_own, void* out, int num_splits,
                                       void* workspace, size_t workspace_bytes, void* stream) {
  SharedPlan p;
  kvq_status st = plan_shared(ctx, layer, batch, num_groups, max_group, max_shared, max_own,
                              num_splits, &p);
  if (st != KVQ_OK) return st;
  if (max_blocks_per_seq < 0) return KVQ_ERR_INVALID_ARG;
  if (batch == 0) return KVQ_OK;
  const kvq_config& c = ctx->cfg;
  DecodeArgs a;
  st = decode_args(ctx, layer, q, k_cache, v_cache, k_scale, v_scale, k_cache_scale, v_cache_scale,
                   block_table, max_blocks_per_seq, context_lens, batch, 0, out, &a);
  if (st != KVQ_OK) return st;
  if ((long long)max_blocks_per_seq * c.block_size >= (1LL << 31)) return KVQ_ERR_INVALID_ARG;
  if (num_groups > 0 && (!group_start || !shared_lens)) return KVQ_ERR_INVALID_ARG;
  if (!aligned4(group_start) || !aligned4(shared_lens)) return KVQ_ERR_ALIGNMENT;
  if ((long long)batch * c.num_kv_heads >= (1LL << 31) || p.workers > kMostWorkers)
    return KVQ_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < p.bytes()) return KVQ_ERR_WORKSPACE;
  if (!aligned16(workspace)) return KVQ_ERR_ALIGNMENT;
  a.err = error_word();
  if (!a.err) return KVQ_ERR_CUDA;
  a.workers = p.workers;
  a.stream_once = stream_once(ctx, layer, batch, (long long)max_shared + max_own);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  SharedArgs x = {};
  x.group_start = group_start;
  x.shared_lens = shared_lens;
  x.groups = num_groups;
  x.max_group = max_group < batch ? max_group : batch;
  x.max_splits = p.splits;
  x.always = num_splits > 0;
  x.max_units = p.units;
  x.unit_rows = p.unit_rows;
  x.tile = cross_query_tile(c.head_dim, c.num_q_heads / c.num_kv_heads);
  x.sms = sm_count();
  // index: (first unit, splits) of each group, which want 8-byte alignment, lead
  x.at = reinterpret_cast<int2*>(ws);
  x.first = reinterpret_cast<int*>(x.at + num_groups);
  x.group_of = x.first + batch;
  x.prefix = x.group_of + batch;
  x.num_units = x.prefix + num_groups;
  x.units = reinterpret_cast<int4*>(ws + p.index_bytes);
  x.o = reinterpret_cast<float*>(ws + p.index_bytes + p.unit_bytes);
  x.lse = x.o + p.rows * c.head_dim;
  a.first = x.first;
  place_partials(c, &a, ws + p.index_bytes + p.unit_bytes + p.prefix_bytes);
  return cuda_status(launch_shared(ctx->mode[layer], c.head_dim, c.num_q_heads / c.num_kv_heads, a,
                                   x, static_cast<cudaStream_t>(stream)));
}

// ---------------------------------------------------------------- accumulated weights
kvq_status kvq_decode_weights_plan(const kvq_ctx* ctx, int layer, int batch, int max_context,
                                   int* num_workers, size_t* workspace_bytes) {
  kvq_status st = check_layer(ctx, layer);
  if (st != KVQ_OK) return st;
  if (ctx->window[layer] != 0) return KVQ_ERR_UNSUPPORTED;
  if (!num_workers || *num_workers < 0) return KVQ_ERR_INVALID_ARG;
  st = kvq_decode_plan(ctx, layer, batch, max_context, num_workers, nullptr);
  if (st != KVQ_OK) return st;
  const kvq_config& c = ctx->cfg;
  if ((double)batch * c.num_q_heads * (double)max_context >= 0x1p60) return KVQ_ERR_INVALID_ARG;
  // partials, the rows' log2 sums, and the scores
  if (workspace_bytes)
    *workspace_bytes = partial_bytes(c, batch, *num_workers) +
                       align16((size_t)batch * c.num_q_heads * sizeof(float)) +
                       (size_t)batch * c.num_q_heads * (size_t)max_context * sizeof(float);
  return KVQ_OK;
}

kvq_status kvq_decode_attention_weights(const kvq_ctx* ctx, int layer, const void* q,
                                        const void* k_cache, const void* v_cache,
                                        const float* k_scale, const float* v_scale,
                                        const float* k_cache_scale, const float* v_cache_scale,
                                        const int* block_table, int max_blocks_per_seq,
                                        const int* context_lens, int batch, int max_context,
                                        void* out, float decay, float* weights,
                                        long long weights_stride, int num_workers,
                                        void* workspace, size_t workspace_bytes, void* stream) {
  int workers = num_workers;
  size_t need = 0;
  kvq_status st = kvq_decode_weights_plan(ctx, layer, batch, max_context, &workers, &need);
  if (st != KVQ_OK) return st;
  if (max_blocks_per_seq < 0 || weights_stride < max_context || !(decay >= 0.f && decay <= 1.f))
    return KVQ_ERR_INVALID_ARG;
  if (batch == 0) return KVQ_OK;
  const kvq_config& c = ctx->cfg;
  // the second pass has a grid of (parts of the context, KV heads, sequences)
  if (batch > 65535 || c.num_kv_heads > 65535 || workers > kMostWorkers) return KVQ_ERR_INVALID_ARG;
  DecodeArgs a;
  st = decode_args(ctx, layer, q, k_cache, v_cache, k_scale, v_scale, k_cache_scale, v_cache_scale,
                   block_table, max_blocks_per_seq, context_lens, batch, max_context, out, &a);
  if (st != KVQ_OK) return st;
  if (!weights) return KVQ_ERR_INVALID_ARG;
  if (!aligned4(weights)) return KVQ_ERR_ALIGNMENT;
  if (!workspace || workspace_bytes < need) return KVQ_ERR_WORKSPACE;
  if (!aligned16(workspace)) return KVQ_ERR_ALIGNMENT;
  a.err = error_word();
  if (!a.err) return KVQ_ERR_CUDA;
  a.workers = workers;
  a.cap = max_context;                          // the scores' rows
  a.stream_once = stream_once(ctx, layer, batch, max_context);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  place_partials(c, &a, ws);
  ws += partial_bytes(c, batch, workers);
  a.lse = reinterpret_cast<float*>(ws);
  a.scores = reinterpret_cast<float*>(ws + align16((size_t)batch * c.num_q_heads * sizeof(float)));
  return cuda_status(launch_decode_weights(ctx->mode[layer], c.head_dim,
                                           c.num_q_heads / c.num_kv_heads, a, weights,
                                           weights_stride, decay, static_cast<cudaStream_t>(stream)));
}

// ---------------------------------------------------------------- eviction
kvq_status kvq_evict_cells(const kvq_ctx* ctx, int layer, const int* rows, const int* keep_lens,
                           int num_rows, int first_kept, int last_kept, const int* ref_count,
                           const int* block_table, int table_rows, int max_blocks_per_seq,
                           const int* context_lens, int max_context, float* weights,
                           long long weights_stride, int* new_lens, void* k_cache, void* v_cache,
                           float* k_cache_scale, float* v_cache_scale, void* stream) {
  kvq_status st = check_layer(ctx, layer);
  if (st != KVQ_OK) return st;
  if (ctx->window[layer] != 0) return KVQ_ERR_UNSUPPORTED;
  if (num_rows < 0 || first_kept < 0 || last_kept < 0 || max_context < 0 || table_rows < 0 ||
      max_blocks_per_seq < 0 || weights_stride < max_context)
    return KVQ_ERR_INVALID_ARG;
  if (num_rows == 0) return KVQ_OK;
  const kvq_config& c = ctx->cfg;
  const int mode = ctx->mode[layer];
  if ((long long)max_blocks_per_seq * c.block_size >= (1LL << 31) ||
      (long long)max_context > (long long)max_blocks_per_seq * c.block_size)
    return KVQ_ERR_INVALID_ARG;
  if (!rows || !keep_lens || !block_table || !context_lens || !weights || !new_lens || !k_cache ||
      !v_cache)
    return KVQ_ERR_INVALID_ARG;
  if (!aligned4(rows) || !aligned4(keep_lens) || !aligned4(ref_count) || !aligned4(block_table) ||
      !aligned4(context_lens) || !aligned4(weights) || !aligned4(new_lens) || !aligned16(k_cache) ||
      !aligned16(v_cache))
    return KVQ_ERR_ALIGNMENT;
  if (is_dynamic(mode)) {
    if (!k_cache_scale || !v_cache_scale) return KVQ_ERR_INVALID_ARG;
    if (!aligned4(k_cache_scale) || !aligned4(v_cache_scale)) return KVQ_ERR_ALIGNMENT;
  }
  const long long items = (long long)num_rows * c.num_kv_heads;
  const int cluster = evict_cluster(max_context, items);
  if (cluster == 0) return KVQ_ERR_UNSUPPORTED;
  if (items * cluster >= (1LL << 31)) return KVQ_ERR_INVALID_ARG;
  // written while other CTAs of the row still read these
  if (overlap(new_lens, num_rows, context_lens, table_rows) ||
      overlap(new_lens, num_rows, rows, num_rows) ||
      (keep_lens != new_lens && overlap(new_lens, num_rows, keep_lens, num_rows)))
    return KVQ_ERR_INVALID_ARG;
  unsigned* err = error_word();
  if (!err) return KVQ_ERR_CUDA;
  EvictArgs a = {};
  a.t = page_tables(ctx, const_cast<int*>(ref_count), const_cast<int*>(block_table), table_rows,
                    max_blocks_per_seq, const_cast<int*>(context_lens), err);
  a.rows = rows;
  a.keep_lens = keep_lens;
  a.new_lens = new_lens;
  a.weights = weights;
  a.stride = weights_stride;
  a.code[0] = static_cast<uint8_t*>(k_cache);
  a.code[1] = static_cast<uint8_t*>(v_cache);
  if (is_dynamic(mode)) {
    a.scale[0] = k_cache_scale;
    a.scale[1] = v_cache_scale;
  }
  a.Hkv = c.num_kv_heads;
  a.first = first_kept;
  a.last = last_kept;
  a.max_len = max_context;
  a.chunk_shift = __builtin_ctz((unsigned)(row_bytes(mode, c.head_dim) / 16));
  return cuda_status(launch_evict(a, num_rows, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
