// Cross attention: the queries of each sequence attend to ALL positions of its
// cached encoder states (another length, no mask), over the quantized paged
// cache.  out[t] = sum_p softmax_p(scale <q[t], K_hat[p]>) V_hat[p].
//
// Kernel.  The warp-specialised tcgen05 kernel of the prefill in its CROSS form
// (prefill_ws.cuh): 128 rows (queries x heads of one KV head) per query tile, key
// tiles of 64, with three differences.
//  * No mask but the sequence's end, so a row's keys are the CTA's keys.
//  * The keys of a sequence are cut into splits of whole key tiles when the
//    queries alone do not fill the SMs (few decoder tokens, long encoder
//    states): each split leaves O / l in fp32 and the log2 of its weights' sum,
//    and a second kernel joins them.  A split has a fixed number of tiles, so
//    ragged lengths spread over the SMs and none waits for the longest.
//  * The output is bf16, and the weight P' that meets V is one f16 term (11
//    bits: off by 2^-11 of its value at most) where the fp32 prefill splits it in
//    two.  That is an eighth of the output's own rounding (2^-8) while P' is a normal
//    f16 number, that is for p x V scale above 2^-20 of the largest V scale seen;
//    below, P' is off by 2^-31 of that scale.  The errors of many weights average,
//    and the PV product costs one MMA instead of two.
//
//  * At most 128 rows (head_dim 64 and 128) take the FEW form: one query tile with
//    Q in tensor memory, two converter groups, and 64 rows or fewer standing in
//    the tile two or four times, each copy with its share of a key tile's keys.
//
// What bounds it.  Many queries: 4 D flops per row and key on the tensor cores; six
// sequences of 900-1,024 queries x 3,000-4,096 states, 32 heads of 128, FP8 (and one
// without states, one without queries): 400 us, 870 TFLOP/s (0.45 of the cuBLAS bf16
// rate); a softmax thread's chain of dependent
// steps takes about 1,880 cycles a key tile, the MMAs of the two query tiles
// about 1,300 (those of S read Q from shared memory again for every 64 keys).
// Few queries: the pages' bytes; six sequences of 1-5 queries x 20,000-32,768 states,
// 64 heads, likewise: 133 us, 2.6 TB/s (0.39); a key tile's 16 KB pass an SM in 770 cycles at the copy
// rate and take about 1,450, in which its roles issue about half of the
// instructions that the SM could: conversion and softmax cost the same for 5
// rows as for 64.
#include <cuda.h>
#include <cuda_runtime.h>

#include "kvq_internal.h"
#include "prefill_common.cuh"
#include "prefill_ws.cuh"

namespace kvq {
namespace {

static_assert(CROSS_KEYS == WKT, "keys per tile");

// Joins the splits of a (query, head) row: weights 2^(lse - max).  WPR warps take
// a row's splits in turn, so that all of them are in flight at once (19 splits
// by one warp took 5 us of dependent loads), and meet in shared memory.  Rows of
// sequences that one split covers were written by it.
constexpr int MERGE_WARPS = 8;

template <int D>
__global__ void __launch_bounds__(MERGE_WARPS * 32) cross_merge_kernel(const PrefillArgs pa, int wpr) {
  // launched as a programmatic dependent: the splits' results are visible below
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const DecodeArgs& a = pa.d;
  constexpr int DL = D / 64;                   // float2 pairs per lane
  __shared__ float2 s_o[MERGE_WARPS][DL][32];
  __shared__ float s_ml[MERGE_WARPS][2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = warp % wpr;
  const long long item = (long long)blockIdx.x * (MERGE_WARPS / wpr) + warp / wpr;
  const long long rows = (long long)a.B * pa.max_query;
  const int h = (int)(item % a.Hq);
  const long long r = item / a.Hq;
  int ns = 0, q0 = 0, i = 0;
  if (r < rows) {
    const int b = (int)(r / pa.max_query);
    i = (int)(r - (long long)b * pa.max_query);
    q0 = pa.query_start[b];
    const int n_b = pa.query_start[b + 1] - q0;
    const int L = a.context_lens[b];
    if (i < n_b && L > 0 && (long long)L <= ((long long)a.max_blocks << a.bs_shift)) {
      const int tiles = (L + CROSS_KEYS - 1) / CROSS_KEYS;
      ns = min(pa.splits, (tiles + pa.split_tiles - 1) / pa.split_tiles);
    }
  }
  const bool here = ns > 1;                    // the same for the row's warps
  const long long step = rows * a.Hq;          // partial rows between splits
  const long long p0 = r * a.Hq + h;
  float2 acc[DL];
#pragma unroll
  for (int k = 0; k < DL; ++k) acc[k] = make_float2(0.f, 0.f);
  float top = -INFINITY, sum = 0.f;
  if (here) {
    // the running maximum and sum of this warp's splits, eight at a time
    for (int s0 = part; s0 < ns; s0 += 8 * wpr) {
      float e[8];
      float2 v[8][DL];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int s = s0 + u * wpr;
        e[u] = -INFINITY;
#pragma unroll
        for (int k = 0; k < DL; ++k) v[u][k] = make_float2(0.f, 0.f);
        if (s < ns) {
          const long long p = p0 + s * step;
          e[u] = a.ws_ml[p];
          const float2* o = reinterpret_cast<const float2*>(a.ws_o + p * D) + lane;
#pragma unroll
          for (int k = 0; k < DL; ++k) v[u][k] = o[32 * k];
        }
      }
      float m = top;
#pragma unroll
      for (int u = 0; u < 8; ++u) m = fmaxf(m, e[u]);
      const float ref = m == -INFINITY ? 0.f : m;
      const float old = ex2(top - ref);
      sum *= old;
#pragma unroll
      for (int k = 0; k < DL; ++k) { acc[k].x *= old; acc[k].y *= old; }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const float w = ex2(e[u] - ref);
        sum += w;
#pragma unroll
        for (int k = 0; k < DL; ++k) {
          acc[k].x = fmaf(w, v[u][k].x, acc[k].x);
          acc[k].y = fmaf(w, v[u][k].y, acc[k].y);
        }
      }
      top = m;
    }
  }
  if (wpr > 1) {
#pragma unroll
    for (int k = 0; k < DL; ++k) s_o[warp][k][lane] = acc[k];
    if (lane == 0) { s_ml[warp][0] = top; s_ml[warp][1] = sum; }
    __syncthreads();
    if (part == 0) {
      float m = top;
      for (int w = 1; w < wpr; ++w) m = fmaxf(m, s_ml[warp + w][0]);
      const float ref = m == -INFINITY ? 0.f : m;
      const float own = ex2(top - ref);
      sum *= own;
#pragma unroll
      for (int k = 0; k < DL; ++k) { acc[k].x *= own; acc[k].y *= own; }
      for (int w = 1; w < wpr; ++w) {
        const float f = ex2(s_ml[warp + w][0] - ref);
        sum = fmaf(f, s_ml[warp + w][1], sum);
#pragma unroll
        for (int k = 0; k < DL; ++k) {
          const float2 v = s_o[warp + w][k][lane];
          acc[k].x = fmaf(f, v.x, acc[k].x);
          acc[k].y = fmaf(f, v.y, acc[k].y);
        }
      }
    }
  }
  if (!here || part != 0) return;
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  uint32_t* out = reinterpret_cast<uint32_t*>(a.out_bf16 + ((long long)(q0 + i) * a.Hq + h) * D) + lane;
#pragma unroll
  for (int k = 0; k < DL; ++k) out[32 * k] = pack_bf16x2(acc[k].x * inv, acc[k].y * inv);
}

template <int MODE, int D, bool FEW>
cudaError_t claunch(const PrefillArgs& pa, cudaStream_t st) {
  using C = WCfg<MODE, D, FEW>;
  const DecodeArgs& a = pa.d;
  const long long total = a.num_blocks * a.Hkv * a.bs * (long long)C::RB;
  CUtensorMap km = {}, vm = {};
  if (total > 0) {
    const bool kok = C::KDIRECT ? make_kblock_map(&km, a.k_cache, total, C::RB)
                                : make_tile_map(&km, a.k_cache, total, C::TB);
    if (!kok || !make_tile_map(&vm, a.v_cache, total, C::TB)) return cudaErrorInvalidValue;
  }
  static bool attr_set[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  auto kern = prefill_ws_kernel<MODE, D, 0, true, FEW>;
  if (!attr_set[dev]) {
    const cudaError_t e = ws_prepare<WRoles<MODE, D, FEW>>(kern, C::SMEM);
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  const long long grid = pa.units ? (long long)pa.splits * a.Hkv : (long long)pa.qtiles * pa.splits * a.B * a.Hkv;
  kern<<<(unsigned)grid, WRoles<MODE, D, FEW>::THREADS, C::SMEM, st>>>(pa, km, vm);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || pa.splits <= 1 || pa.units) return e;
  const long long items = (long long)a.B * pa.max_query * a.Hq;
  // its launch overlaps the attention's tail
  const int wpr = pa.splits <= 8 ? 1 : (pa.splits <= 16 ? 2 : (pa.splits <= 32 ? 4 : 8));
  const int per_cta = MERGE_WARPS / wpr;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((items + per_cta - 1) / per_cta));
  cfg.blockDim = dim3(MERGE_WARPS * 32);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cross_merge_kernel<D>, pa, wpr);
}

template <int MODE>
cudaError_t claunch_d(int D, const PrefillArgs& pa, cudaStream_t st) {
  // one query tile's rows at most: the form with two converter groups (at head_dim
  // 256, which has one query tile anyway, it measured 20 % slower: its operand
  // buffers leave no room for the second group to work ahead)
  const bool few = ((long long)pa.max_query << pa.g_shift) <= WROWS;
  switch (D) {
    case 64: return few ? claunch<MODE, 64, true>(pa, st) : claunch<MODE, 64, false>(pa, st);
    case 128: return few ? claunch<MODE, 128, true>(pa, st) : claunch<MODE, 128, false>(pa, st);
    case 256: return claunch<MODE, 256, false>(pa, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

int cross_query_tile(int D, int G) {
  return (D == 256 ? WRoles<BF16, 256, false>::NQ : WRoles<BF16, 128, false>::NQ) * (WROWS / G);
}

namespace {

cudaError_t launch(int mode, int D, int G, const PrefillArgs& pa, cudaStream_t st) {
  switch (mode) {
    case BF16: return claunch_d<BF16>(D, pa, st);
    case FP8_PER_TENSOR: return claunch_d<FP8_PER_TENSOR>(D, pa, st);
    case FP8_PER_HEAD: return claunch_d<FP8_PER_HEAD>(D, pa, st);
    case FP8_PER_TOKEN_HEAD: return claunch_d<FP8_PER_TOKEN_HEAD>(D, pa, st);
    case INT4_PER_TOKEN_HEAD: return claunch_d<INT4_PER_TOKEN_HEAD>(D, pa, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_cross(int mode, int D, int G, const DecodeArgs& a, const int* query_start,
                         int max_query_len, int splits, int split_tiles, cudaStream_t st) {
  PrefillArgs pa = {};
  pa.d = a;
  pa.query_start = query_start;
  const int tile = cross_query_tile(D, G);
  pa.qtiles = (max_query_len + tile - 1) / tile;
  pa.g_shift = __builtin_ctz((unsigned)G);
  pa.max_query = max_query_len;
  pa.splits = splits;
  pa.split_tiles = split_tiles;
  return launch(mode, D, G, pa, st);
}

cudaError_t launch_prefix(int mode, int D, int G, const DecodeArgs& a, const SharedArgs& x, cudaStream_t st) {
  PrefillArgs pa = {};
  pa.d = a;
  pa.query_start = x.group_start;
  pa.qtiles = 1;                               // divided by, then a unit names its query tile
  pa.g_shift = __builtin_ctz((unsigned)G);
  pa.max_query = x.max_group;
  pa.splits = x.max_units;                     // CTAs per KV head
  pa.units = x.units;
  pa.num_units = x.num_units;
  pa.unit_rows = x.unit_rows;
  return launch(mode, D, G, pa, st);
}

}  // namespace kvq
