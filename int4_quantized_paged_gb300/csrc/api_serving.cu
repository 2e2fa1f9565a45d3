// C ABI of the operators around the cache: rotary positions, the pages of the
// pool and cross attention.  Argument validation, the split plan and dispatch;
// everything here runs on the host.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <new>
#include <vector>

#include "api_common.h"
#include "kvq.h"
#include "kvq_internal.h"

struct kvq_rope {
  int head_dim, rotary_dim, layout;
  double frequency[kvq::ROPE_MAX_PAIRS];
  kvq::RopeTable table;
};

using namespace kvq;

namespace {

bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }

bool positive(double x) { return x > 0.0 && isfinite(x); }

constexpr double kTwoPi = 6.283185307179586476925;

// f / (2 pi) modulo one turn, as a 64-bit fraction of a turn.  A double carries
// 53 bits of it, so p f is off by p f 2^-53 radians at most, as a product in
// double would be.
unsigned long long turn_fraction(double f) {
  double turns = f / kTwoPi;
  turns -= floor(turns);
  return turns >= 1.0 ? 0ull : (unsigned long long)ldexp(turns, 64);
}

kvq_status check_tables(const kvq_ctx* ctx, const int* ref_count, const int* block_table, int rows,
                        int max_blocks, const int* context_lens) {
  if (!ctx || rows < 0 || max_blocks < 0) return KVQ_ERR_INVALID_ARG;
  if ((long long)max_blocks * ctx->cfg.block_size >= (1LL << 31)) return KVQ_ERR_INVALID_ARG;
  if (!ref_count || !block_table || !context_lens) return KVQ_ERR_INVALID_ARG;
  if (!aligned4(ref_count) || !aligned4(block_table) || !aligned4(context_lens))
    return KVQ_ERR_ALIGNMENT;
  return KVQ_OK;
}

// Splits of the keys for `base` CTAs (query tiles x sequences x KV heads) over
// `tiles` key tiles: the count whose waves over the SMs take the least time, in
// units of a key tile (about 1 us): a CTA costs its tiles and about three more
// for its queries, barriers and epilogue; joining splits costs about three and
// a little per split.
int plan_splits(long long base, int tiles) {
  const int sms = sm_count();
  int best = 1;
  double best_cost = 1e300;
  for (int s = 1; s <= tiles && s <= 128; ++s) {
    const int per = (tiles + s - 1) / s;
    if (s > 1 && (tiles + per - 1) / per != s) continue;     // fewer splits do the same
    const double waves = (double)((base * s + sms - 1) / sms);
    const double cost = waves * (per + 3.0) + (s > 1 ? 3.0 + 0.05 * s : 0.0);
    if (cost < best_cost) {
      best_cost = cost;
      best = s;
    }
  }
  return best;
}

// Splits (0 in: the plan's choice) and workspace bytes of a cross attention call
// with query_start, or with max_query_len 0 of the one without.
kvq_status plan_cross(const kvq_ctx* ctx, int layer, int batch, int max_query_len,
                      int max_encoder_len, int* num_splits, size_t* need) {
  kvq_status st = check_layer(ctx, layer);
  if (st != KVQ_OK) return st;
  if (!num_splits || *num_splits < 0 || batch < 0 || max_query_len < 0 || max_encoder_len < 0 ||
      max_encoder_len > (1 << 30))
    return KVQ_ERR_INVALID_ARG;
  if (max_query_len == 0)                       // one query per sequence: the decode's plan
    return kvq_decode_plan(ctx, layer, batch, max_encoder_len, num_splits, need);
  const kvq_config& c = ctx->cfg;
  const int tile = cross_query_tile(c.head_dim, c.num_q_heads / c.num_kv_heads);
  // CTAs of one split, in steps whose products fit 64 bits
  long long base = ((long long)max_query_len + tile - 1) / tile * batch;
  if (base >= (1LL << 31)) return KVQ_ERR_INVALID_ARG;
  base *= c.num_kv_heads;
  if (base >= (1LL << 31)) return KVQ_ERR_INVALID_ARG;
  const int tiles = (int)(((long long)max_encoder_len + CROSS_KEYS - 1) / CROSS_KEYS);
  if (*num_splits == 0) *num_splits = plan_splits(base, tiles);
  if (*num_splits > 1024 || base * *num_splits >= (1LL << 31)) return KVQ_ERR_INVALID_ARG;
  // the grid of the kernel that joins the splits
  if (*num_splits > 1 && (long long)*num_splits * batch * max_query_len * c.num_q_heads >= (1LL << 34))
    return KVQ_ERR_INVALID_ARG;
  *need = *num_splits <= 1 ? 0
                           : (size_t)*num_splits * batch * (size_t)max_query_len * c.num_q_heads *
                                 (c.head_dim + 1) * sizeof(float);
  return KVQ_OK;
}

}  // namespace

extern "C" {

// ---------------------------------------------------------------- rotary
kvq_status kvq_rope_create(const kvq_rope_config* cfg, kvq_rope** out) {
  if (!cfg || !out) return KVQ_ERR_INVALID_ARG;
  *out = nullptr;
  if (cfg->head_dim != 64 && cfg->head_dim != 128 && cfg->head_dim != 256)
    return KVQ_ERR_UNSUPPORTED;
  const int r = cfg->rotary_dim;
  if (r < 16 || r > cfg->head_dim) return KVQ_ERR_INVALID_ARG;
  if (r % 16 != 0) return KVQ_ERR_UNSUPPORTED;
  if (cfg->layout != KVQ_ROPE_HALF && cfg->layout != KVQ_ROPE_INTERLEAVED)
    return KVQ_ERR_INVALID_ARG;
  if (cfg->scaling < KVQ_ROPE_PLAIN || cfg->scaling > KVQ_ROPE_PARTS) return KVQ_ERR_INVALID_ARG;
  if (cfg->frequencies ? cfg->scaling != KVQ_ROPE_PLAIN : !positive(cfg->base))
    return KVQ_ERR_INVALID_ARG;
  if (cfg->scaling != KVQ_ROPE_PLAIN && !positive(cfg->factor)) return KVQ_ERR_INVALID_ARG;
  if (cfg->scaling == KVQ_ROPE_PARTS &&
      (!positive(cfg->original_context) || !(cfg->low_rotations >= 0.0) ||
       !(cfg->high_rotations > cfg->low_rotations) || !isfinite(cfg->high_rotations)))
    return KVQ_ERR_INVALID_ARG;
  const float m = cfg->magnitude == 0.f ? 1.f : cfg->magnitude;
  // The range keeps a rotated vector's scale away from fp32 underflow for every
  // bf16 input: its amax is at least 2^-133 / (16 sqrt 2).
  if (!(m >= 0.0625f && m <= 16.f)) return KVQ_ERR_INVALID_ARG;
  kvq_rope* p = new (std::nothrow) kvq_rope;
  if (!p) return KVQ_ERR_INVALID_ARG;
  memset(p, 0, sizeof(*p));
  p->head_dim = cfg->head_dim;
  p->rotary_dim = r;
  p->layout = cfg->layout;
  p->table.magnitude = m;
  double base = cfg->base;
  if (cfg->scaling == KVQ_ROPE_BASE) base *= pow(cfg->factor, r / (r - 2.0));
  for (int i = 0; i < r / 2; ++i) {
    double f = cfg->frequencies ? cfg->frequencies[i] : pow(base, -2.0 * i / r);
    if (cfg->scaling == KVQ_ROPE_LINEAR) f /= cfg->factor;
    if (cfg->scaling == KVQ_ROPE_PARTS) {
      const double turns = cfg->original_context * f / kTwoPi;
      double g = (turns - cfg->low_rotations) / (cfg->high_rotations - cfg->low_rotations);
      g = g < 0.0 ? 0.0 : (g > 1.0 ? 1.0 : g);
      f = g * f + (1.0 - g) * f / cfg->factor;
    }
    if (!isfinite(f)) {
      delete p;
      return KVQ_ERR_INVALID_ARG;
    }
    p->frequency[i] = f;
    p->table.phase[i] = turn_fraction(f);
  }
  *out = p;
  return KVQ_OK;
}

void kvq_rope_destroy(kvq_rope* rope) { delete rope; }

kvq_status kvq_rope_frequencies(const kvq_rope* rope, double* frequencies, float* magnitude) {
  if (!rope) return KVQ_ERR_INVALID_ARG;
  if (frequencies) memcpy(frequencies, rope->frequency, sizeof(double) * (rope->rotary_dim / 2));
  if (magnitude) *magnitude = rope->table.magnitude;
  return KVQ_OK;
}

kvq_status kvq_rope_apply(const kvq_rope* rope, const void* x, long long x_token_stride,
                          const long long* positions, long long num_tokens, int num_heads,
                          void* out, long long out_token_stride, int inverse, void* stream) {
  if (!rope || num_tokens < 0 || num_heads <= 0) return KVQ_ERR_INVALID_ARG;
  if (num_tokens == 0) return KVQ_OK;
  const long long HD = (long long)num_heads * rope->head_dim;
  const long long xs = x_token_stride == 0 ? HD : x_token_stride;
  const long long os = out_token_stride == 0 ? HD : out_token_stride;
  if (!x || !out || !positions || xs < HD || os < HD) return KVQ_ERR_INVALID_ARG;
  if (x == out && xs != os) return KVQ_ERR_INVALID_ARG;
  if (num_tokens >= (1LL << 31) / num_heads) return KVQ_ERR_INVALID_ARG;
  if (xs % 8 != 0 || os % 8 != 0 || !aligned16(x) || !aligned16(out) || !aligned8(positions))
    return KVQ_ERR_ALIGNMENT;
  unsigned* err = error_word();
  if (!err) return KVQ_ERR_CUDA;
  RopeArgs a = {};
  a.w.T = num_tokens;
  a.w.err = err;
  a.w.bs = 1;
  a.q = static_cast<const uint16_t*>(x);
  a.q_out = static_cast<uint16_t*>(out);
  a.q_stride = xs;
  a.q_out_stride = os;
  a.positions = positions;
  a.Hq = num_heads;
  a.rotary = rope->rotary_dim;
  a.sin_magnitude = inverse ? -rope->table.magnitude : rope->table.magnitude;
  return cuda_status(launch_rope(KVQ_BF16, rope->head_dim, rope->layout, a, rope->table,
                                 static_cast<cudaStream_t>(stream)));
}

kvq_status kvq_rope_cache_write(const kvq_ctx* ctx, const kvq_rope* rope, int layer, const void* q,
                                long long q_token_stride, void* q_out,
                                long long q_out_token_stride, const void* k_new,
                                const void* v_new, long long kv_token_stride,
                                const long long* positions, const long long* slot_mapping,
                                long long num_tokens, const float* k_scale, const float* v_scale,
                                void* k_cache, void* v_cache, float* k_cache_scale,
                                float* v_cache_scale, void* stream) {
  kvq_status st = check_layer(ctx, layer);
  if (st != KVQ_OK) return st;
  const kvq_config& c = ctx->cfg;
  if (!rope || rope->head_dim != c.head_dim || num_tokens < 0) return KVQ_ERR_INVALID_ARG;
  if (num_tokens == 0) return KVQ_OK;
  if (num_tokens >= (1LL << 31) / (c.num_q_heads + 2 * c.num_kv_heads)) return KVQ_ERR_INVALID_ARG;
  const int mode = ctx->mode[layer];
  const long long KD = (long long)c.num_kv_heads * c.head_dim;
  const long long QD = (long long)c.num_q_heads * c.head_dim;
  const long long ks = kv_token_stride == 0 ? KD : kv_token_stride;
  const long long qs = q_token_stride == 0 ? QD : q_token_stride;
  const long long os = q_out_token_stride == 0 ? QD : q_out_token_stride;
  if (!k_new || !v_new || !positions || !slot_mapping || !k_cache || !v_cache || ks < KD)
    return KVQ_ERR_INVALID_ARG;
  if ((q == nullptr) != (q_out == nullptr)) return KVQ_ERR_INVALID_ARG;
  if (q && (qs < QD || os < QD || (q == q_out && qs != os))) return KVQ_ERR_INVALID_ARG;
  if (ks % 8 != 0 || !aligned16(k_new) || !aligned16(v_new) || !aligned16(k_cache) ||
      !aligned16(v_cache) || !aligned8(slot_mapping) || !aligned8(positions))
    return KVQ_ERR_ALIGNMENT;
  if (q && (qs % 8 != 0 || os % 8 != 0 || !aligned16(q) || !aligned16(q_out)))
    return KVQ_ERR_ALIGNMENT;
  if ((mode == KVQ_FP8_PER_TENSOR || mode == KVQ_FP8_PER_HEAD) && (!k_scale || !v_scale))
    return KVQ_ERR_INVALID_ARG;
  if (is_dynamic(mode)) {
    if (!k_cache_scale || !v_cache_scale) return KVQ_ERR_INVALID_ARG;
    if (!aligned4(k_cache_scale) || !aligned4(v_cache_scale)) return KVQ_ERR_ALIGNMENT;
  }
  unsigned* err = error_word();
  if (!err) return KVQ_ERR_CUDA;
  RopeArgs a = {};
  a.w.k_new = static_cast<const uint16_t*>(k_new);
  a.w.v_new = static_cast<const uint16_t*>(v_new);
  a.w.token_stride = ks;
  a.w.slots = slot_mapping;
  a.w.T = num_tokens;
  a.w.Hkv = c.num_kv_heads;
  a.w.bs = c.block_size;
  a.w.bs_shift = __builtin_ctz((unsigned)c.block_size);
  a.w.num_blocks = c.num_blocks;
  a.w.k_scale = k_scale;
  a.w.v_scale = v_scale;
  a.w.k_cache = static_cast<uint8_t*>(k_cache);
  a.w.v_cache = static_cast<uint8_t*>(v_cache);
  a.w.k_cs = k_cache_scale;
  a.w.v_cs = v_cache_scale;
  a.w.err = err;
  a.q = static_cast<const uint16_t*>(q);
  a.q_out = static_cast<uint16_t*>(q_out);
  a.q_stride = qs;
  a.q_out_stride = os;
  a.positions = positions;
  a.Hq = q ? c.num_q_heads : 0;
  a.rotary = rope->rotary_dim;
  a.sin_magnitude = rope->table.magnitude;
  return cuda_status(launch_rope(mode, c.head_dim, rope->layout, a, rope->table,
                                 static_cast<cudaStream_t>(stream)));
}

// ---------------------------------------------------------------- pages
kvq_status kvq_extend_sequences(const kvq_ctx* ctx, const int* rows, const int* new_tokens,
                                int num_rows, int* ref_count, int* block_table, int table_rows,
                                int max_blocks_per_seq, int* context_lens, long long max_tokens,
                                int* query_start, long long* positions, long long* slot_mapping,
                                int* copies, void* stream) {
  if (!ctx || num_rows < 0 || max_tokens < 0 || max_tokens >= (1LL << 31) - 1)
    return KVQ_ERR_INVALID_ARG;
  if (num_rows == 0) return KVQ_OK;
  kvq_status st =
      check_tables(ctx, ref_count, block_table, table_rows, max_blocks_per_seq, context_lens);
  if (st != KVQ_OK) return st;
  if (num_rows > EXTEND_MAX_ROWS) return KVQ_ERR_UNSUPPORTED;
  if (!rows || !new_tokens || !query_start || !copies) return KVQ_ERR_INVALID_ARG;
  if (max_tokens > 0 && (!positions || !slot_mapping)) return KVQ_ERR_INVALID_ARG;
  if (!aligned4(rows) || !aligned4(new_tokens) || !aligned4(query_start) || !aligned4(copies) ||
      !aligned8(positions) || !aligned8(slot_mapping))
    return KVQ_ERR_ALIGNMENT;
  unsigned* err = error_word();
  if (!err) return KVQ_ERR_CUDA;
  ExtendArgs x;
  x.rows = rows;
  x.new_tokens = new_tokens;
  x.n = num_rows;
  x.max_tokens = max_tokens;
  x.query_start = query_start;
  x.positions = positions;
  x.slots = slot_mapping;
  x.copies = copies;
  return cuda_status(launch_extend(
      page_tables(ctx, ref_count, block_table, table_rows, max_blocks_per_seq, context_lens, err), x,
      static_cast<cudaStream_t>(stream)));
}

kvq_status kvq_fork_sequences(const kvq_ctx* ctx, const int* parents, const int* children,
                              int num_forks, int* ref_count, int* block_table, int table_rows,
                              int max_blocks_per_seq, int* context_lens, void* stream) {
  if (!ctx || num_forks < 0) return KVQ_ERR_INVALID_ARG;
  if (num_forks == 0) return KVQ_OK;
  kvq_status st =
      check_tables(ctx, ref_count, block_table, table_rows, max_blocks_per_seq, context_lens);
  if (st != KVQ_OK) return st;
  if (!parents || !children) return KVQ_ERR_INVALID_ARG;
  if (!aligned4(parents) || !aligned4(children)) return KVQ_ERR_ALIGNMENT;
  unsigned* err = error_word();
  if (!err) return KVQ_ERR_CUDA;
  return cuda_status(launch_fork(
      page_tables(ctx, ref_count, block_table, table_rows, max_blocks_per_seq, context_lens, err),
      parents, children, num_forks, static_cast<cudaStream_t>(stream)));
}

kvq_status kvq_truncate_sequences(const kvq_ctx* ctx, const int* rows, const int* keep_lens,
                                  int num_rows, int* ref_count, int* block_table, int table_rows,
                                  int max_blocks_per_seq, int* context_lens, void* stream) {
  if (!ctx || num_rows < 0) return KVQ_ERR_INVALID_ARG;
  if (num_rows == 0) return KVQ_OK;
  kvq_status st =
      check_tables(ctx, ref_count, block_table, table_rows, max_blocks_per_seq, context_lens);
  if (st != KVQ_OK) return st;
  if (!rows) return KVQ_ERR_INVALID_ARG;
  if (!aligned4(rows) || !aligned4(keep_lens)) return KVQ_ERR_ALIGNMENT;
  unsigned* err = error_word();
  if (!err) return KVQ_ERR_CUDA;
  return cuda_status(launch_truncate(
      page_tables(ctx, ref_count, block_table, table_rows, max_blocks_per_seq, context_lens, err),
      rows, keep_lens, num_rows, static_cast<cudaStream_t>(stream)));
}

kvq_status kvq_compact_blocks(const kvq_ctx* ctx, int* ref_count, int* block_table,
                              int table_rows, int max_blocks_per_seq, int* context_lens,
                              int* moves, int* num_moves, void* stream) {
  kvq_status st =
      check_tables(ctx, ref_count, block_table, table_rows, max_blocks_per_seq, context_lens);
  if (st != KVQ_OK) return st;
  if (!num_moves || (!moves && ctx->cfg.num_blocks > 1)) return KVQ_ERR_INVALID_ARG;
  if (!aligned4(moves) || !aligned4(num_moves)) return KVQ_ERR_ALIGNMENT;
  unsigned* err = error_word();
  if (!err) return KVQ_ERR_CUDA;
  return cuda_status(launch_compact(
      page_tables(ctx, ref_count, block_table, table_rows, max_blocks_per_seq, context_lens, err),
      moves, num_moves, static_cast<cudaStream_t>(stream)));
}

kvq_status kvq_copy_blocks(const kvq_ctx* ctx, int first_layer, int num_layers, const int* pairs,
                           int max_pairs, const int* num_pairs, void* const* k_caches,
                           void* const* v_caches, float* const* k_cache_scales,
                           float* const* v_cache_scales, void* stream) {
  if (!ctx || max_pairs < 0 || num_layers < 0 || first_layer < 0 ||
      num_layers > ctx->cfg.num_layers - first_layer)
    return KVQ_ERR_INVALID_ARG;
  if (max_pairs == 0 || num_layers == 0) return KVQ_OK;
  if (!pairs || !k_caches || !v_caches) return KVQ_ERR_INVALID_ARG;
  if (!aligned4(pairs) || !aligned4(num_pairs)) return KVQ_ERR_ALIGNMENT;
  const kvq_config& c = ctx->cfg;
  const long long cells = (long long)c.num_kv_heads * c.block_size;
  for (int l = 0; l < num_layers; ++l) {        // all of them before anything is launched
    const int mode = ctx->mode[first_layer + l];
    if (!k_caches[l] || !v_caches[l]) return KVQ_ERR_INVALID_ARG;
    if (!aligned16(k_caches[l]) || !aligned16(v_caches[l])) return KVQ_ERR_ALIGNMENT;
    if (cells * row_bytes(mode, c.head_dim) / 16 >= (1LL << 28)) return KVQ_ERR_UNSUPPORTED;
    if (is_dynamic(mode)) {
      if (!k_cache_scales || !v_cache_scales || !k_cache_scales[l] || !v_cache_scales[l])
        return KVQ_ERR_INVALID_ARG;
      if (!aligned16(k_cache_scales[l]) || !aligned16(v_cache_scales[l])) return KVQ_ERR_ALIGNMENT;
    }
  }
  unsigned* err = error_word();
  if (!err) return KVQ_ERR_CUDA;
  for (int l0 = 0; l0 < num_layers; l0 += COPY_MAX_LAYERS) {
    CopyArgs a = {};
    a.layers = num_layers - l0 < COPY_MAX_LAYERS ? num_layers - l0 : COPY_MAX_LAYERS;
    for (int l = 0; l < a.layers; ++l) {
      const int mode = ctx->mode[first_layer + l0 + l];
      CopyLayer& y = a.layer[l];
      y.buf[0] = k_caches[l0 + l];
      y.buf[1] = v_caches[l0 + l];
      y.code_chunks = (unsigned)(cells * row_bytes(mode, c.head_dim) / 16);
      if (is_dynamic(mode)) {
        y.buf[2] = k_cache_scales[l0 + l];
        y.buf[3] = v_cache_scales[l0 + l];
        y.scale_chunks = (unsigned)(cells * 4 / 16);
      }
    }
    a.pairs = pairs;
    a.num_pairs = num_pairs;
    a.max_pairs = max_pairs;
    a.num_blocks = c.num_blocks;
    a.err = err;
    const kvq_status st = cuda_status(launch_copy_blocks(a, static_cast<cudaStream_t>(stream)));
    if (st != KVQ_OK) return st;
  }
  return KVQ_OK;
}

// ---------------------------------------------------------------- cross attention
kvq_status kvq_cross_plan(const kvq_ctx* ctx, int layer, int batch, int max_query_len,
                          int max_encoder_len, int* num_splits, size_t* workspace_bytes) {
  size_t need = 0;
  kvq_status st =
      plan_cross(ctx, layer, batch, max_query_len, max_encoder_len, num_splits, &need);
  if (st != KVQ_OK) return st;
  if (max_query_len == 1) {                     // the call may have no query_start: the decode's
    int workers = 0;                            // own plan then fits the same workspace
    size_t step = 0;
    st = kvq_decode_plan(ctx, layer, batch, max_encoder_len, &workers, &step);
    if (st != KVQ_OK) return st;
    if (step > need) need = step;
  }
  if (workspace_bytes) *workspace_bytes = need;
  return KVQ_OK;
}

kvq_status kvq_cross_attention(const kvq_ctx* ctx, int layer, const void* q, const void* k_cache,
                               const void* v_cache, const float* k_scale, const float* v_scale,
                               const float* k_cache_scale, const float* v_cache_scale,
                               const int* block_table, int max_blocks_per_seq,
                               const int* query_start, const int* encoder_lens, int batch,
                               int max_query_len, int max_encoder_len, void* out, int num_splits,
                               void* workspace, size_t workspace_bytes, void* stream) {
  kvq_status st = check_layer(ctx, layer);
  if (st != KVQ_OK) return st;
  if (ctx->window[layer] != 0) return KVQ_ERR_UNSUPPORTED;
  if (batch < 0 || max_query_len < 0 || max_encoder_len < 0 || max_blocks_per_seq < 0 || num_splits < 0)
    return KVQ_ERR_INVALID_ARG;
  if (!query_start) {
    if (max_query_len > 1) return KVQ_ERR_INVALID_ARG;
    int workers = num_splits;
    if (max_query_len == 1) {
      // num_splits may count splits of the keys (kvq_cross_plan of 1), of which a
      // single one would leave the batch to one warp: the decode's own plan, where
      // the workspace holds it
      int own = 0;
      size_t step = 0;
      st = kvq_decode_plan(ctx, layer, batch, max_encoder_len, &own, &step);
      if (st != KVQ_OK) return st;
      if (workspace_bytes >= step) workers = 0;
    }
    return kvq_decode_attention_bf16(ctx, layer, q, k_cache, v_cache, k_scale, v_scale,
                                     k_cache_scale, v_cache_scale, block_table, max_blocks_per_seq,
                                     encoder_lens, batch, max_encoder_len, out, workers, workspace,
                                     workspace_bytes, stream);
  }
  if (batch == 0 || max_query_len == 0) return KVQ_OK;
  const kvq_config& c = ctx->cfg;
  const int mode = ctx->mode[layer];
  if ((long long)max_encoder_len > (long long)max_blocks_per_seq * c.block_size)
    return KVQ_ERR_INVALID_ARG;
  if (!q || !k_cache || !v_cache || !block_table || !encoder_lens || !out)
    return KVQ_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) ||
      !aligned4(block_table) || !aligned4(query_start) || !aligned4(encoder_lens))
    return KVQ_ERR_ALIGNMENT;
  if ((mode == KVQ_FP8_PER_TENSOR || mode == KVQ_FP8_PER_HEAD) && (!k_scale || !v_scale))
    return KVQ_ERR_INVALID_ARG;
  if (is_dynamic(mode)) {
    if (!k_cache_scale || !v_cache_scale) return KVQ_ERR_INVALID_ARG;
    // the kernel fetches 16 scales at a time by bulk copies
    if (!aligned16(k_cache_scale) || !aligned16(v_cache_scale)) return KVQ_ERR_ALIGNMENT;
  }
  int splits = num_splits;
  size_t need = 0;
  st = plan_cross(ctx, layer, batch, max_query_len, max_encoder_len, &splits, &need);
  if (st != KVQ_OK) return st;
  if (splits > 1 && (!workspace || workspace_bytes < need)) return KVQ_ERR_WORKSPACE;
  if (splits > 1 && !aligned16(workspace)) return KVQ_ERR_ALIGNMENT;
  const size_t rows = (size_t)splits * batch * (size_t)max_query_len * c.num_q_heads;
  unsigned* err = error_word();
  if (!err) return KVQ_ERR_CUDA;
  DecodeArgs a = {};
  a.q = static_cast<const uint16_t*>(q);
  a.k_cache = static_cast<const uint8_t*>(k_cache);
  a.v_cache = static_cast<const uint8_t*>(v_cache);
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.k_cs = k_cache_scale;
  a.v_cs = v_cache_scale;
  a.block_table = block_table;
  a.context_lens = encoder_lens;
  a.out_bf16 = static_cast<uint16_t*>(out);
  if (splits > 1) {
    a.ws_o = static_cast<float*>(workspace);
    a.ws_ml = a.ws_o + rows * c.head_dim;
  }
  a.err = err;
  a.B = batch;
  a.Hq = c.num_q_heads;
  a.Hkv = c.num_kv_heads;
  a.bs = c.block_size;
  a.bs_shift = __builtin_ctz((unsigned)c.block_size);
  a.max_blocks = max_blocks_per_seq;
  a.num_blocks = c.num_blocks;
  a.qk_scale = ctx->softmax_scale * 1.4426950408889634f;
  const int tiles = (max_encoder_len + CROSS_KEYS - 1) / CROSS_KEYS;
  const int per = tiles == 0 ? 1 : (tiles + splits - 1) / splits;
  return cuda_status(launch_cross(mode, c.head_dim, c.num_q_heads / c.num_kv_heads, a, query_start,
                                  max_query_len, splits, per, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
