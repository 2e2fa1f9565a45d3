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
//    shortest row and to whole tiles of 16), and for each row where its own begins;
//  * the warp-specialised attention of cross.cu, the groups as its sequences: rows x
//    heads on the tensor cores, the prefix cut into splits that fill the SMs;
//  * the decode kernel over the rows' own positions, which begins while the prefixes'
//    last CTAs run (it does not read their results);
//  * join_kernel: all partials of a row.
//
// What bounds it: the prefix's bytes for few rows, 4 D flops per row, head and prefix
// position for many.
#include <cuda.h>
#include <cuda_runtime.h>

#include "decode_kernel.cuh"

namespace kvq {
namespace {

constexpr int PT = 1024;
constexpr int MIN_ROWS = 2;                    // rows of a group that are worth a shared pass

__global__ void __launch_bounds__(PT) plan_kernel(const DecodeArgs a, const SharedArgs x) {
  for (int b = threadIdx.x; b < a.B; b += PT) {
    x.first[b] = 0;
    x.group_of[b] = -1;
  }
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int g = warp; g < x.groups; g += PT / 32) {
    const int r0 = x.group_start[g], r1 = x.group_start[g + 1], P = x.shared_lens[g];
    const bool bad = r0 < 0 || r1 < r0 || r1 > a.B || P < 0;
    if (bad && lane == 0) atomicOr(a.err, ERR_BAD_INDEX);
    int shared = 0;
    // rows past the caller's bound, and a row by itself, read their prefix alone
    if (!bad && r1 - r0 >= MIN_ROWS && r1 - r0 <= x.max_group) {
      shared = P;
      for (int b = r0 + lane; b < r1; b += 32) shared = min(shared, ctx_len(a, b));
      shared = __reduce_min_sync(0xffffffffu, shared) & ~(TILE - 1);
    }
    if (lane == 0) x.prefix[g] = shared;
    if (shared > 0)
      for (int b = r0 + lane; b < r1; b += 32) {
        x.first[b] = shared;
        x.group_of[b] = g;
      }
  }
}

// One CTA per (row, query head): JW warps take its partials in turn, and meet in
// shared memory.
constexpr int JW = 4;

template <int D>
__global__ void __launch_bounds__(JW * 32) join_kernel(const DecodeArgs a, const SharedArgs x) {
  constexpr int DL = D / 64;                   // float2 pairs per lane
  __shared__ float2 s_o[JW][DL][32];
  __shared__ float s_top[JW], s_sum[JW];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.x % a.Hq, b = blockIdx.x / a.Hq;
  const int G = a.Hq / a.Hkv, kvh = h / G, j = h - kvh * G;
  // launched as a programmatic dependent: all partials are visible below
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // the prefix's splits: O / l, and the log2 of the weights' sum
  const int grp = x.group_of[b];
  int ns = 0;
  long long p0 = 0;
  if (grp >= 0) {
    const int tiles = (x.prefix[grp] + CROSS_KEYS - 1) / CROSS_KEYS;
    ns = min(x.splits, (tiles + x.split_tiles - 1) / x.split_tiles);
    p0 = ((long long)grp * x.max_group + (b - x.group_start[grp])) * a.Hq + h;
  }
  const long long step = (long long)x.groups * x.max_group * a.Hq;
  // the workers of the row's own positions: O, running maximum and sum
  const int item = b * a.Hkv + kvh;
  long long w0 = 0, nw = 0;
  const long long W = a.workers, T = a.item_tiles[(long long)a.B * a.Hkv];
  {
    const long long first = a.item_tiles[item], n = a.item_tiles[item + 1] - first;
    if (n > 0) {
      w0 = ((first + 1) * W - 1) / T;
      nw = ((first + n) * W - 1) / T - w0 + 1;
    }
  }
  float top = -INFINITY, sum = 0.f;
  float2 acc[DL];
#pragma unroll
  for (int k = 0; k < DL; ++k) acc[k] = make_float2(0.f, 0.f);
  // parts 0 .. ns - 1 are splits, the others workers; four in flight a warp
  for (long long s0 = warp; s0 < ns + nw; s0 += 4 * JW) {
    float e[4], f[4];                          // log2 of a part's weight, and its sum over it
    float2 v[4][DL];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const long long s = s0 + u * JW;
      e[u] = -INFINITY;
      f[u] = 0.f;
#pragma unroll
      for (int k = 0; k < DL; ++k) v[u][k] = make_float2(0.f, 0.f);
      const float* o = nullptr;
      if (s < ns) {
        const long long p = p0 + s * step;
        e[u] = x.lse[p];
        f[u] = 1.f;
        o = x.o + p * D;
      } else if (s < ns + nw) {
        const long long w = w0 + (s - ns);
        // a worker whose share is empty wrote nothing
        if ((w * T) / W != ((w + 1) * T) / W) {
          const long long part = (item + w) * G + j;
          e[u] = a.ws_ml[2 * part];
          f[u] = a.ws_ml[2 * part + 1];
          o = a.ws_o + part * D;
        }
      }
      if (o && e[u] != -INFINITY) {
#pragma unroll
        for (int k = 0; k < DL; ++k) v[u][k] = reinterpret_cast<const float2*>(o)[lane + 32 * k];
      }
    }
    float m = top;
#pragma unroll
    for (int u = 0; u < 4; ++u) m = fmaxf(m, e[u]);
    const float ref = m == -INFINITY ? 0.f : m;
    const float old = ex2(top - ref);
    sum *= old;
#pragma unroll
    for (int k = 0; k < DL; ++k) { acc[k].x *= old; acc[k].y *= old; }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float w = ex2(e[u] - ref);
      sum = fmaf(w, f[u], sum);
#pragma unroll
      for (int k = 0; k < DL; ++k) {
        acc[k].x = fmaf(w, v[u][k].x, acc[k].x);
        acc[k].y = fmaf(w, v[u][k].y, acc[k].y);
      }
    }
    top = m;
  }
#pragma unroll
  for (int k = 0; k < DL; ++k) s_o[warp][k][lane] = acc[k];
  if (lane == 0) { s_top[warp] = top; s_sum[warp] = sum; }
  __syncthreads();
  float m = -INFINITY;
#pragma unroll
  for (int w = 0; w < JW; ++w) m = fmaxf(m, s_top[w]);
  const float ref = m == -INFINITY ? 0.f : m;
  float f[JW], all = 0.f;
#pragma unroll
  for (int w = 0; w < JW; ++w) {
    f[w] = ex2(s_top[w] - ref);
    all = fmaf(f[w], s_sum[w], all);
  }
  const float inv = all > 0.f ? 1.f / all : 0.f;   // a row without positions: zeros
  uint32_t* out = reinterpret_cast<uint32_t*>(a.out_bf16 + ((long long)b * a.Hq + h) * D);
  for (int k = warp; k < DL; k += JW) {
    float2 r = make_float2(0.f, 0.f);
#pragma unroll
    for (int w = 0; w < JW; ++w) {
      const float2 v = s_o[w][k][lane];
      r.x = fmaf(f[w], v.x, r.x);
      r.y = fmaf(f[w], v.y, r.y);
    }
    out[lane + 32 * k] = pack_bf16x2(r.x * inv, r.y * inv);
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
    return launch_dependent(join_kernel<D>, dim3((unsigned)((long long)a.B * a.Hq)), JW * 32, 0, st, a, x);
  }
};

}  // namespace

cudaError_t launch_shared(int mode, int D, int G, const DecodeArgs& a, const SharedArgs& x, cudaStream_t st) {
  plan_kernel<<<1, PT, 0, st>>>(a, x);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const bool prefix = x.groups > 0 && x.max_group >= MIN_ROWS && x.splits > 0;
  if (prefix) {
    DecodeArgs p = a;
    p.B = x.groups;
    p.context_lens = x.prefix;
    p.ws_o = x.o;
    p.ws_ml = x.lse;
    e = launch_prefix(mode, D, G, p, x.group_start, x.max_group, x.splits, x.split_tiles, st);
    if (e != cudaSuccess) return e;
  }
  return with_layer(mode, D, G, OwnOp{a, x, prefix, st});
}

}  // namespace kvq
