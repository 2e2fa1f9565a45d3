// Joins the partial results of a row: those of the decode kernel's workers and, behind
// a shared prefix, those of the prefix's splits.
#pragma once

#include "decode_kernel.cuh"

namespace kvq {
namespace {

// One CTA per (row, KV head): JT / 32 / G warps take the parts of each of its G query
// heads in turn, JU in flight a warp, and meet in shared memory.  (A warp for a query
// head, as the decode's own merge has, took 15 us over 57 parts; here 5.)
constexpr int JT = 512;
constexpr int JU = 4;

// BEHIND: the rows' prefixes are in *x.  With a.lse the log2 of each row's weight sum
// is left there.
template <int D, int G, bool BEHIND>
__global__ void __launch_bounds__(JT) join_kernel(const DecodeArgs a, const SharedArgs x) {
  constexpr int DL = D / 64;                   // float2 pairs per lane
  constexpr int JW = JT / 32 / G;              // warps of a query head
  __shared__ float2 s_o[JT / 32][DL][32];
  __shared__ float s_top[JT / 32], s_sum[JT / 32];
  __shared__ long long s_w0, s_T;
  __shared__ int s_n[2];                       // splits, workers
  __shared__ long long s_p0, s_step;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int j = warp / JW, part = warp - j * JW;
  const int item = blockIdx.x, b = item / a.Hkv, kvh = item - b * a.Hkv;
  const long long W = a.workers;
  // launched as a programmatic dependent: all partials are visible below
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (threadIdx.x == 0) {
    // the workers that own tiles of this item (64-bit divisions: by one thread)
    const long long first = a.item_tiles[item], n = a.item_tiles[item + 1] - first;
    const long long T = a.item_tiles[(long long)a.B * a.Hkv];
    s_T = T;
    s_w0 = n > 0 ? ((first + 1) * W - 1) / T : 0;
    s_n[1] = n > 0 ? (int)(((first + n) * W - 1) / T - s_w0) + 1 : 0;
    if (!BEHIND) s_n[0] = 0;
  }
  if (BEHIND && threadIdx.x == 32) {
    const int grp = x.group_of[b];
    s_n[0] = 0;
    if (grp >= 0) {
      const int2 at = x.at[grp];
      s_n[0] = at.y;
      const int r0 = x.group_start[grp], rows = x.group_start[grp + 1] - r0;
      const int qt = (b - r0) / x.tile, tiles = (rows + x.tile - 1) / x.tile;
      s_p0 = ((long long)(at.x + qt) * x.unit_rows + (b - r0 - qt * x.tile)) * a.Hq;
      s_step = (long long)tiles * x.unit_rows * a.Hq;
    }
  }
  __syncthreads();
  const int ns = s_n[0], nw = s_n[1];
  const long long w0 = s_w0, T = s_T;
  float top = -INFINITY, sum = 0.f;
  float2 acc[DL];
#pragma unroll
  for (int k = 0; k < DL; ++k) acc[k] = make_float2(0.f, 0.f);
  // parts 0 .. ns - 1 are splits, the others workers
  for (int s0 = part; s0 < ns + nw; s0 += JU * JW) {
    float e[JU], f[JU];                        // log2 of a part's weight, and its sum over it
    float2 v[JU][DL];
#pragma unroll
    for (int u = 0; u < JU; ++u) {
      const int s = s0 + u * JW;
      e[u] = -INFINITY;
      f[u] = 0.f;
      const float* o = nullptr;
      if (BEHIND && s < ns) {
        const long long p = s_p0 + s * s_step + kvh * G + j;
        e[u] = x.lse[p];
        f[u] = 1.f;
        o = x.o + p * D;
      } else if (s < ns + nw) {
        const long long w = w0 + (s - ns);
        // with more workers than tiles some have none, and wrote nothing
        if (T >= W || (w * T) / W != ((w + 1) * T) / W) {
          const long long p = (item + w) * G + j;
          e[u] = a.ws_ml[2 * p];
          f[u] = a.ws_ml[2 * p + 1];
          o = a.ws_o + p * D;
        }
      }
#pragma unroll
      for (int k = 0; k < DL; ++k)
        v[u][k] = o ? reinterpret_cast<const float2*>(o)[lane + 32 * k] : make_float2(0.f, 0.f);
    }
    float m = top;
#pragma unroll
    for (int u = 0; u < JU; ++u) m = fmaxf(m, e[u]);
    const float ref = m == -INFINITY ? 0.f : m;
    const float old = ex2(top - ref);
    sum *= old;
#pragma unroll
    for (int k = 0; k < DL; ++k) { acc[k].x *= old; acc[k].y *= old; }
#pragma unroll
    for (int u = 0; u < JU; ++u) {
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
  for (int w = 0; w < JW; ++w) m = fmaxf(m, s_top[j * JW + w]);
  const float ref = m == -INFINITY ? 0.f : m;
  float f[JW], all = 0.f;
#pragma unroll
  for (int w = 0; w < JW; ++w) {
    f[w] = ex2(s_top[j * JW + w] - ref);
    all = fmaf(f[w], s_sum[j * JW + w], all);
  }
  const float inv = all > 0.f ? 1.f / all : 0.f;   // a row without positions: zeros
  const long long row = (long long)b * a.Hq + kvh * G + j;
  if (a.lse && part == 0 && lane == 0) a.lse[row] = m + log2f(all);
  uint32_t* out = reinterpret_cast<uint32_t*>(a.out_bf16 + row * D);
  for (int k = part; k < DL; k += JW) {
    float2 r = make_float2(0.f, 0.f);
#pragma unroll
    for (int w = 0; w < JW; ++w) {
      const float2 v = s_o[j * JW + w][k][lane];
      r.x = fmaf(f[w], v.x, r.x);
      r.y = fmaf(f[w], v.y, r.y);
    }
    out[lane + 32 * k] = pack_bf16x2(r.x * inv, r.y * inv);
  }
}

}  // namespace
}  // namespace kvq
