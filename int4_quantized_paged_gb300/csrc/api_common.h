// Host-side pieces shared by the C-ABI translation units: the context and the
// argument checks.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <vector>

#include "kvq.h"

struct kvq_ctx {
  kvq_config cfg;
  std::vector<int> mode;
  std::vector<int> window;
  float softmax_scale;
};

namespace kvq {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

inline bool is_dynamic(int mode) {
  return mode == KVQ_FP8_PER_TOKEN_HEAD || mode == KVQ_INT4_PER_TOKEN_HEAD;
}

inline double elem_bytes(int mode) {
  return mode == KVQ_BF16 ? 2.0 : (mode == KVQ_INT4_PER_TOKEN_HEAD ? 0.5 : 1.0);
}

inline long long row_bytes(int mode, int D) {
  return mode == KVQ_BF16 ? 2LL * D : (mode == KVQ_INT4_PER_TOKEN_HEAD ? D / 2 : D);
}

inline kvq_status check_layer(const kvq_ctx* ctx, int layer) {
  if (!ctx) return KVQ_ERR_INVALID_ARG;
  if (layer < 0 || layer >= ctx->cfg.num_layers) return KVQ_ERR_INVALID_ARG;
  return KVQ_OK;
}

inline kvq_status cuda_status(cudaError_t e) { return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA; }

}  // namespace kvq
