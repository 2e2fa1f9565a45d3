// Decode attention of a batch whose rows share prefixes: each group of rows reads its
// prefix once.
//
// Mathematics.  A row's softmax over [0, L) joins its softmax over the prefix [0, P)
// with the one over its own positions [P, L) by their sums: with the log2 sums e1, e2
// and outputs o1, o2 of the parts, o = (2^(e1 - m) o1 + 2^(e2 - m) o2) / (2^(e1 - m)
// + 2^(e2 - m)), m = max(e1, e2).  The prefix's part is that of an attention without
// a mask, of all rows of the group at once.
//
// Structure.  Four launches:
//  * plan_kernel, one CTA: each group's prefix as it can be shared (cut to its
//    shortest row and to whole tiles of 16), for each row where its own begins, and the
//    units of work: the prefixes cut into splits of as many key tiles as take the
//    least time over the SMs.  The host does not know the lengths, and splits of equal
//    numbers left most SMs waiting for the longest prefix (six groups of 100-8,000
//    positions, 1-30 rows: 52 us; cut by the lengths 35);
//  * the warp-specialised attention of cross.cu over the units: rows x heads on the
//    tensor cores;
//  * the decode kernel over the rows' own positions, which begins while the prefixes'
//    last CTAs run (it does not read their results; the prefixes' launch itself gains
//    nothing from being one of that kind);
//  * join_kernel: all partials of a row.
//
// What bounds it: the prefix's bytes for few rows, 4 D flops per row, head and prefix
// position for many.  One group of 64 rows behind 32,768 positions, 64 heads of 128, FP8
// per head, up to 1,000 positions of their own: 112 us (prefix 72, 930 TFLOP/s; own
// positions 31, partly beside it; join 9; plan 5).
#include <cuda.h>
#include <cuda_runtime.h>

#include "decode_kernel.cuh"
#include "join.cuh"

namespace kvq {
namespace {

constexpr int PT = 1024;
// What sharing costs and saves, in the time that a CTA takes for a key tile (64 keys of
// one KV head against a query tile, about 0.9 us).  The decode kernel reads 160 keys of
// a row and KV head for an SM in that time, so a group gains from three rows on (times
// its keys: 1 against 0.4 a row); the pass itself, and the join of its splits, cost
// about ten more (SHARED_PASS).  Measured, FP8, 32 heads of 128, 64 rows, shared / each row for
// itself: 32 groups of 2 behind 4,096 positions 134 / 91 us, 16 of 4 85 / 90, 8 of 8
// 58 / 90; 8 groups of 8 behind 512 positions 36 / 27; one group of 64 behind 32,768
// (64 heads, scales per head) 114 / 570.
constexpr int MIN_ROWS = 3;

__global__ void __launch_bounds__(PT) plan_kernel(const DecodeArgs a, const SharedArgs x) {
  __shared__ unsigned long long s_best, s_alone;
  __shared__ int s_most;
  for (int b = threadIdx.x; b < a.B; b += PT) {
    x.first[b] = 0;
    x.group_of[b] = -1;
  }
  if (threadIdx.x == 0) {
    s_best = ~0ull;
    s_alone = 0;
    s_most = 0;
  }
  // starts that do not ascend within the batch might put a row into two groups
  bool astray = false;
  for (int g = threadIdx.x; g < x.groups; g += PT) {
    const int r0 = x.group_start[g], r1 = x.group_start[g + 1];
    astray |= r0 < 0 || r1 < r0 || r1 > a.B;
  }
  astray = __syncthreads_or(astray);
  if (astray && threadIdx.x == 0) atomicOr(a.err, ERR_BAD_INDEX);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int least_rows = x.always ? 2 : MIN_ROWS;
  for (int g = warp; g < x.groups; g += PT / 32) {
    const int r0 = x.group_start[g], r1 = x.group_start[g + 1], P = x.shared_lens[g];
    if (P < 0 && lane == 0) atomicOr(a.err, ERR_BAD_INDEX);
    int shared = 0;
    // rows past the caller's bound, and few rows, read their prefix alone
    if (!astray && P > 0 && x.max_units > 0 && r1 - r0 >= least_rows && r1 - r0 <= x.max_group) {
      shared = P;
      for (int b = r0 + lane; b < r1; b += 32) shared = min(shared, ctx_len(a, b));
      shared = __reduce_min_sync(0xffffffffu, shared) & ~(TILE - 1);
    }
    if (lane == 0) {
      const int tiles = (shared + CROSS_KEYS - 1) / CROSS_KEYS;
      x.prefix[g] = shared;
      atomicMax(&s_most, tiles);
      atomicAdd(&s_alone, (unsigned long long)tiles * (unsigned)max(r1 - r0, 0));
    }
  }
  __syncthreads();
  const int most = s_most;
  if (most == 0) {                             // nothing to share
    if (threadIdx.x == 0) *x.num_units = 0;
    return;
  }
  // Query tiles and key tiles of a group.
  auto sizes = [&](int g, int* tiles) {
    *tiles = (x.prefix[g] + CROSS_KEYS - 1) / CROSS_KEYS;
    return *tiles > 0 ? (x.group_start[g + 1] - x.group_start[g] + x.tile - 1) / x.tile : 0;
  };
  // Key tiles per split: a CTA costs its tiles and about three more, and CTAs come in
  // waves over the SMs.  Each thread prices its own counts; of equal ones the larger
  // splits win.
  const int least = (most + x.max_splits - 1) / x.max_splits;
  for (int t = least + threadIdx.x; t <= most; t += PT) {
    long long units = 0;
    for (int g = 0; g < x.groups; ++g) {
      int tiles;
      const int q = sizes(g, &tiles);
      units += (long long)q * ((tiles + t - 1) / t);
    }
    if (units > x.max_units && t < most) continue;
    const unsigned long long waves = (unsigned long long)((units * a.Hkv + x.sms - 1) / x.sms);
    atomicMin(&s_best, (waves * (unsigned)(t + 3)) << 31 | (unsigned)(0x7fffffff - t));
  }
  __syncthreads();
  const int per = 0x7fffffff - (int)(s_best & 0x7fffffffu);
  // 5 (cost + SHARED_PASS) SMs < 2 KV heads x rows x key tiles: 0.4 of a tile each
  if (!x.always && 5 * ((s_best >> 31) + SHARED_PASS) * (unsigned)x.sms >= 2 * s_alone * (unsigned)a.Hkv) {
    if (threadIdx.x == 0) *x.num_units = 0;
    return;
  }
  for (int g = warp; g < x.groups; g += PT / 32) {
    const int shared = x.prefix[g];
    if (shared > 0)
      for (int b = x.group_start[g] + lane; b < x.group_start[g + 1]; b += 32) {
        x.first[b] = shared;
        x.group_of[b] = g;
      }
  }
  // The list of units: a group's query tiles are neighbours, so that they read its pages
  // from L2.
  if (warp == 0) {
    int base = 0;
    for (int g0 = 0; g0 < x.groups; g0 += 32) {
      const int g = g0 + lane;
      int tiles = 0, q = 0, splits = 0;
      if (g < x.groups) {
        q = sizes(g, &tiles);
        splits = (tiles + per - 1) / per;
      }
      int incl = q * splits;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      const int first = base + incl - q * splits;
      if (g < x.groups) x.at[g] = make_int2(first, splits);
      base += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) *x.num_units = base;
  }
  __syncthreads();
  for (int g = warp; g < x.groups; g += PT / 32) {
    int tiles;
    const int q = sizes(g, &tiles);
    const int2 at = x.at[g];
    for (int i = lane; i < q * at.y; i += 32) x.units[at.x + i] = make_int4(g, i / q, i % q, per);
  }
}

struct OwnOp {
  const DecodeArgs& a;
  const SharedArgs& x;
  bool behind_prefix;                          // launched behind the prefixes' kernel
  cudaStream_t st;

  template <int MODE, int D, int G>
  cudaError_t run() const {
    using C = Cfg<MODE, D>;
    const long long total = a.num_blocks * a.Hkv * a.bs * (long long)C::RB;
    CUtensorMap km = {}, vm = {};
    if (total > 0) {
      if (!make_tile_map(&km, a.k_cache, total, C::TB) || !make_tile_map(&vm, a.v_cache, total, C::TB))
        return cudaErrorInvalidValue;
    }
    int smem = 0;
    if (prepare<MODE, D, G, DECODE_OWN>(&smem) <= 0) return cudaErrorInvalidConfiguration;
    const int ctas = (a.workers + WARPS - 1) / WARPS;
    auto kern = decode_kernel<MODE, D, G, DECODE_OWN>;
    cudaError_t e;
    if (behind_prefix) {
      e = launch_dependent(kern, dim3((unsigned)ctas), WARPS * 32, smem, st, a, km, vm);
    } else {
      kern<<<ctas, WARPS * 32, smem, st>>>(a, km, vm);
      e = cudaGetLastError();
    }
    if (e != cudaSuccess) return e;
    return launch_dependent(join_kernel<D, G, true>, dim3((unsigned)(a.B * a.Hkv)), JT, 0, st, a, x);
  }
};

}  // namespace

cudaError_t launch_shared(int mode, int D, int G, const DecodeArgs& a, const SharedArgs& x, cudaStream_t st) {
  plan_kernel<<<1, PT, 0, st>>>(a, x);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const bool prefix = x.max_units > 0;
  if (prefix) {
    DecodeArgs p = a;
    p.B = x.groups;
    p.context_lens = x.prefix;
    p.ws_o = x.o;
    p.ws_ml = x.lse;
    e = launch_prefix(mode, D, G, p, x, st);
    if (e != cudaSuccess) return e;
  }
  return with_layer(mode, D, G, OwnOp{a, x, prefix, st});
}

}  // namespace kvq
