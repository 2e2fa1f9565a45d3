// Paged GQA decode attention over the quantized cache.
//
// What it computes: for each sequence b and query head hq, the softmax over
// retained positions p in [lo, L) of softmax_scale * <q, K_hat[p]> weights
// V_hat[p]; K_hat = code * K scale, V_hat = code * V scale.  The K scale
// multiplies the dot product of q with the raw codes and the V scale the
// softmax weight, so codes are never rescaled element by element.  Scale
// layouts: "Per-tensor vs per-head FP8 KV cache scales"; packed INT4:
// "Per-token-head KV cache scale overhead", section "INT4 makes the metadata
// fraction larger"; windows and BF16 (skipped) layers: "FP8 KV cache layer
// skipping vs per-head scales", sections "FP8 KV cache layer skipping vs
// per-head scales" and "Layer skipping follows retained-token footprint".
//
// Work decomposition (split-K over the context, balanced over warps):
//  * A sequence's retained positions are cut into 16-position tiles (a tile
//    never straddles a page: block_size is a multiple of 16).  All tiles of
//    all (sequence, KV head) items, in that order, form one list of T tiles.
//    Worker warp w takes tiles [w T / W, (w+1) T / W): every warp gets the
//    same number of tiles whatever the context lengths, and a warp's share
//    runs across item boundaries.  For each item segment it covers, a warp
//    either writes the final output (it covered the whole item) or a partial
//    (running max m, sum l, unnormalised O) that a merge kernel combines by
//    log-sum-exp; the merge is a programmatic dependent launch, so its launch
//    overlaps this grid's tail.  Warps never wait on one another.
//  * Each warp streams its tiles through an NS-stage ring in shared memory
//    with TMA: a 2-D tensor copy each for the K and V code tile (128-byte
//    rows, 128B swizzle so the fragment loads below hit no bank conflicts)
//    and, for dynamic scales, a 64-byte bulk copy each of the tile's K and V
//    scales, completing on the stage's mbarrier.  The copies of the next
//    NS-1 tiles (of this or the next item) are in flight while one tile is
//    computed.  Pages of a layer larger than L2 are copied evict-first.
//    Every wait is bounded: a wait that runs out sets the TIMEOUT bit of the
//    device error word, drains the warp's copies and stops.
//  * QK on tensor cores: S^T[16 positions x 8 columns] = K_tile . Q^T with
//    mma.m16n8k16, fp32 accumulate.  E4M3 and INT4 codes convert exactly to
//    f16; q (bf16) times a power of two converts exactly to f16 (an FP8
//    query's E4M3 values are f16 values).  Columns are the G query heads of
//    the KV head, repeated once per term of the weight split when they fit
//    in the 8 columns, so a QK column is already the PV column it feeds.
//  * Online softmax in log2 units on the fragments, against a reference max
//    that moves (reduced over the warp, O and l rescaled) only on tiles where
//    some lane holds a score above it by more than 8 (a weight factor of
//    2^8), so the weights p stay below 2^8.  The weights that meet V are P' = p * v_scale * 2^k, with k a
//    power-of-two range factor that keeps P' below 2^14, so both f16 terms of
//    its split stay normal numbers.
//  * PV on tensor cores with d as the M dimension: O^T[d x cols] += V^T P'.
//    P' is split into two f16 terms (hi + lo, about 22 bits; three bf16
//    terms for BF16 layers) so the weighted sum keeps fp32-class accuracy;
//    for G*terms <= 8 all terms share one 8-column tile.  The P' fragment
//    comes from the S^T fragment by movmatrix (in-register 8x8 transpose).
//  * Outputs are fp32, or their round-to-nearest-even bf16 for the bf16
//    variant.
#include <cuda.h>
#include <cuda_runtime.h>

#include "decode_kernel.cuh"

namespace kvq {
namespace {

template <int MODE, int D, int G>
cudaError_t launch3(const DecodeArgs& a, cudaStream_t st) {
  using C = Cfg<MODE, D>;
  const long long total = a.num_blocks * a.Hkv * a.bs * (long long)C::RB;
  CUtensorMap km, vm;
  if (total > 0) {
    if (!make_tile_map(&km, a.k_cache, total, C::TB) || !make_tile_map(&vm, a.v_cache, total, C::TB))
      return cudaErrorInvalidValue;
  }
  int smem = 0;
  if (prepare<MODE, D, G>(&smem) <= 0) return cudaErrorInvalidConfiguration;
  const int ctas = (a.workers + WARPS - 1) / WARPS;
  decode_kernel<MODE, D, G><<<ctas, WARPS * 32, smem, st>>>(a, km, vm);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || a.workers <= 1) return e;
  // programmatic dependent launch: the merge grid's launch overlaps the
  // decode grid's tail
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.B * a.Hkv));
  cfg.blockDim = dim3(32 * G);
  cfg.dynamicSmemBytes = 0;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, merge_kernel<D, G>, a);
}

template <int MODE, int D>
int per_sm2(int G) {
  switch (G) {
    case 1: return prepare<MODE, D, 1>(nullptr);
    case 2: return prepare<MODE, D, 2>(nullptr);
    case 4:
      if constexpr (built<MODE, D, 4>()) return prepare<MODE, D, 4>(nullptr);
      else return 0;
    case 8:
      if constexpr (built<MODE, D, 8>()) return prepare<MODE, D, 8>(nullptr);
      else return 0;
    default: return 0;
  }
}

template <int MODE>
int per_sm1(int D, int G) {
  switch (D) {
    case 64: return per_sm2<MODE, 64>(G);
    case 128: return per_sm2<MODE, 128>(G);
    case 256: return per_sm2<MODE, 256>(G);
    default: return 0;
  }
}

template <int MODE, int D>
cudaError_t launch2(int G, const DecodeArgs& a, cudaStream_t st) {
  switch (G) {
    case 1: return launch3<MODE, D, 1>(a, st);
    case 2: return launch3<MODE, D, 2>(a, st);
    case 4:
      if constexpr (built<MODE, D, 4>()) return launch3<MODE, D, 4>(a, st);
      else return cudaErrorInvalidValue;
    case 8:
      if constexpr (built<MODE, D, 8>()) return launch3<MODE, D, 8>(a, st);
      else return cudaErrorInvalidValue;
    default: return cudaErrorInvalidValue;
  }
}

template <int MODE>
cudaError_t launch1(int D, int G, const DecodeArgs& a, cudaStream_t st) {
  switch (D) {
    case 64: return launch2<MODE, 64>(G, a, st);
    case 128: return launch2<MODE, 128>(G, a, st);
    case 256: return launch2<MODE, 256>(G, a, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

int decode_ctas_per_sm(int mode, int D, int G) {
  switch (mode) {
    case BF16: return per_sm1<BF16>(D, G);
    case FP8_PER_TENSOR: return per_sm1<FP8_PER_TENSOR>(D, G);
    case FP8_PER_HEAD: return per_sm1<FP8_PER_HEAD>(D, G);
    case FP8_PER_TOKEN_HEAD: return per_sm1<FP8_PER_TOKEN_HEAD>(D, G);
    case INT4_PER_TOKEN_HEAD: return per_sm1<INT4_PER_TOKEN_HEAD>(D, G);
    default: return 0;
  }
}

int decode_warps_per_cta() { return WARPS; }

bool decode_supported(int mode, int D, int G) {
  if (!(mode >= BF16 && mode <= INT4_PER_TOKEN_HEAD)) return false;
  if (!(D == 64 || D == 128 || D == 256)) return false;
  if (!(G == 1 || G == 2 || G == 4 || G == 8)) return false;
  // the PV accumulators (D/16 tiles x 4 x column tiles) must fit in registers
  if (D == 256 && (G == 8 || (mode == BF16 && G == 4))) return false;
  return true;
}

cudaError_t launch_decode(int mode, int D, int G, const DecodeArgs& a, cudaStream_t st) {
  if (a.B == 0) return cudaSuccess;
  switch (mode) {
    case BF16: return launch1<BF16>(D, G, a, st);
    case FP8_PER_TENSOR: return launch1<FP8_PER_TENSOR>(D, G, a, st);
    case FP8_PER_HEAD: return launch1<FP8_PER_HEAD>(D, G, a, st);
    case FP8_PER_TOKEN_HEAD: return launch1<FP8_PER_TOKEN_HEAD>(D, G, a, st);
    case INT4_PER_TOKEN_HEAD: return launch1<INT4_PER_TOKEN_HEAD>(D, G, a, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace kvq
