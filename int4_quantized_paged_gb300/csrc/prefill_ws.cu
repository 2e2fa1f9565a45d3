// Prefill (chunked multi-query) attention over a quantized paged cache (FP8 or
// INT4 codes at head_dim 64, 128 or 256; BF16 layers at 64 and 128),
// warp-specialised on the fifth-generation tensor cores.  It computes what the single-role prefill kernel computes
// (causal attention of each new token's query over the retained positions,
// the scales folded into score and weight: "Per-tensor vs per-head FP8 KV
// cache scales", section "Use a three-stage decision"; "FP8 KV cache layer
// skipping vs per-head scales", section "Run a four-way ablation") with the
// work of one key tile spread over warps with their own roles, so that the
// tensor cores, the code conversion and the softmax run at the same time.
//
// A CTA owns two query tiles of M = 128 rows each (128/G consecutive new
// positions times the G query heads of one KV head; tile 1 follows tile 0),
// and streams the keys of both in tiles of 64 positions.  At head_dim 256 a
// CTA owns one query tile (its O takes 256 tensor-memory columns) and keeps
// Q in tensor memory, the A operand of S; the roles below then have one
// softmax warpgroup and the other warps move down by four.  Roles (15 warps; with
// a scale per key one more, which completes the last warpgroup, and the softmax
// warpgroups take registers that the others give up):
//  * warp 12, producer: 2-D TMA copies of the key tile's K and V page tiles
//    (and 64-byte bulk copies of their dynamic scales) into a ring of raw
//    stages, issued by an elected lane; the block ids of 32 page tiles are
//    loaded at once, a round ahead.
//  * warps 8-11, converters: raw codes -> f16, K and V alike as 64 rows (keys)
//    of D in 64-d blocks of 128-byte rows with the 128-byte swizzle: the
//    K-major operand of S and the MN-major operand of PV, so nothing is
//    transposed; K and V scales (a masking one and zero for a key outside the
//    CTA's range or on a page that was not fetched) and the tile's largest V-scale exponent.  Three
//    operand buffers.  BF16 layers:
//    K stays bf16 (S is a bf16 MMA; at head_dim 128 the producer copies it
//    straight into its operand buffer), and the converters give each V row
//    the power-of-two V scale that maps its largest exponent to 2^14,
//    converting it to f16 exactly; the rest then runs as for dynamic scales.
//  * warps 13 and 14, MMA issuers (one thread each): S_j = Q_j K^T (M 128, N 64)
//    into tensor memory for each query tile j, and O_j += P'_j V with P'_j read
//    from tensor memory, every term of its f16 hi + lo split.  Each query
//    tile has two S/P' buffers (key tile t uses buffer t & 1; P' replaces S
//    there): S_j(t+2) is issued once the PV that last read its buffer, PV_j(t),
//    has completed, so a softmax warpgroup finds the scores of its next tile
//    ready and the tensor cores work on one query tile while the other's
//    softmax runs.
//  * warps 0-3 and 4-7, softmax of query tile 0 and 1: one thread per row
//    (its tensor-memory lane) loads the row's 64 scores, applies the K scale
//    and masks (pairs of fp32 per instruction), keeps a lazily moved reference
//    max (moved only when a tile's max exceeds it by more than 8 in log2 units),
//    rescales the row of O in tensor memory
//    when it moves, and stores P' = p x v_scale x 2^k (f16 hi + lo) over the
//    scores it has read.
// Tensor memory: two S/P' buffers per query tile (64 columns each), O_0, O_1
// (D each).
// Every wait is bounded; a wait that runs out flags TIMEOUT and sets a
// shared abort flag that ends every role's loop, the work already issued is
// waited for (bounded again), and tensor memory is freed before the CTA exits.
//
// Measured (FP8 per-token-head, 1,024 new tokens a sequence at the end of
// contexts of 4,096): 621 TFLOP/s at head_dim 128 (0.32 of the bf16 peak), 430 at 64;
// 676 at 256 (8,192 new tokens after 8,192).
#include <cuda.h>
#include <cuda_runtime.h>

#include "kvq_internal.h"
#include "prefill_common.cuh"
#include "prefill_ws.cuh"

namespace kvq {
namespace {

template <int MODE, int D, int G>
cudaError_t wslaunch3(const PrefillArgs& pa0, int max_query_len, cudaStream_t st) {
  using C = WCfg<MODE, D, false>;
  const DecodeArgs& a = pa0.d;
  const long long total = a.num_blocks * a.Hkv * a.bs * (long long)C::RB;
  CUtensorMap km, vm;
  if (total > 0) {
    const bool kok = C::KDIRECT ? make_kblock_map(&km, a.k_cache, total, C::RB)
                                : make_tile_map(&km, a.k_cache, total, C::TB);
    if (!kok || !make_tile_map(&vm, a.v_cache, total, C::TB)) return cudaErrorInvalidValue;
  }
  static bool attr_set[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  auto kern = prefill_ws_kernel<MODE, D, G>;
  if (!attr_set[dev]) {
    const cudaError_t e = ws_prepare<WRoles<MODE, D, false>>(kern, C::SMEM);
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  PrefillArgs pa = pa0;
  const int qp2 = WRoles<MODE, D, false>::NQ * (WROWS / G);      // query positions per CTA
  pa.qtiles = (max_query_len + qp2 - 1) / qp2;
  const long long grid = (long long)pa.qtiles * a.B * a.Hkv;
  if (grid <= 0) return cudaSuccess;
  kern<<<(unsigned)grid, WRoles<MODE, D, false>::THREADS, C::SMEM, st>>>(pa, km, vm);
  return cudaGetLastError();
}

template <int MODE, int D>
cudaError_t wslaunch2(int G, const PrefillArgs& pa, int mq, cudaStream_t st) {
  switch (G) {
    case 1: return wslaunch3<MODE, D, 1>(pa, mq, st);
    case 2: return wslaunch3<MODE, D, 2>(pa, mq, st);
    case 4: return wslaunch3<MODE, D, 4>(pa, mq, st);
    case 8: return wslaunch3<MODE, D, 8>(pa, mq, st);
    default: return cudaErrorInvalidValue;
  }
}

template <int MODE>
cudaError_t wslaunch1(int D, int G, const PrefillArgs& pa, int mq, cudaStream_t st) {
  switch (D) {
    case 64: return wslaunch2<MODE, 64>(G, pa, mq, st);
    case 128: return wslaunch2<MODE, 128>(G, pa, mq, st);
    case 256: return wslaunch2<MODE, 256>(G, pa, mq, st);
    default: return cudaErrorInvalidValue;
  }
}

// BF16 layers at head_dim 64 and 128 (a BF16 raw stage at 256 does not fit
// beside the operand buffers)
cudaError_t wslaunch1_bf16(int D, int G, const PrefillArgs& pa, int mq, cudaStream_t st) {
  switch (D) {
    case 64: return wslaunch2<BF16, 64>(G, pa, mq, st);
    case 128: return wslaunch2<BF16, 128>(G, pa, mq, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

bool prefill_ws_supports(int mode, int D) {
  if (mode == BF16) return D == 64 || D == 128;
  return D == 64 || D == 128 || D == 256;
}

cudaError_t launch_prefill_ws(int mode, int D, int G, const DecodeArgs& a, const int* query_start,
                              int max_query_len, cudaStream_t st) {
  if (a.B == 0 || max_query_len <= 0) return cudaSuccess;
  PrefillArgs pa;
  pa.d = a;
  pa.query_start = query_start;
  pa.qtiles = 0;
  switch (mode) {
    case FP8_PER_TENSOR: return wslaunch1<FP8_PER_TENSOR>(D, G, pa, max_query_len, st);
    case FP8_PER_HEAD: return wslaunch1<FP8_PER_HEAD>(D, G, pa, max_query_len, st);
    case FP8_PER_TOKEN_HEAD: return wslaunch1<FP8_PER_TOKEN_HEAD>(D, G, pa, max_query_len, st);
    case INT4_PER_TOKEN_HEAD: return wslaunch1<INT4_PER_TOKEN_HEAD>(D, G, pa, max_query_len, st);
    case BF16: return wslaunch1_bf16(D, G, pa, max_query_len, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace kvq
