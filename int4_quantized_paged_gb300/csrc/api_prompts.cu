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

}  // extern "C"
