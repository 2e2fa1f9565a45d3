// C ABI of the operators for long and shared prompts: argument validation,
// workspaces and dispatch; everything here runs on the host.
#include <cuda_runtime.h>
#include <stdint.h>

#include "api_common.h"
#include "kvq.h"
#include "kvq_internal.h"

using namespace kvq;

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
  const int per = prompt_positions_per_cta(c.head_dim, G);
  if ((most + per - 1) / per * batch >= (1LL << 31) / c.num_kv_heads) return KVQ_ERR_INVALID_ARG;
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
