// Rotary positions: the rotation of query (and any other) head vectors, and
// its fused form, the cache write that rotates q and k, quantizes k and v and
// scatters them into pages in one launch.
//
// Mathematics.  Pair i of a head vector (elements i and i + r/2, or 2i and
// 2i + 1) at position p turns by the angle p f_i and is multiplied by a
// magnitude m:  (x, y) -> m (x cos - y sin, x sin + y cos); elements from r on
// pass through.  With -sin the map is the transpose, which is the rotation's
// gradient and, where m = 1, its inverse.
//
// Angles.  p f_i reaches 10^5 radians and more, where a 32-bit product keeps no
// fraction of a turn.  The frequency is therefore held as a 64-bit fixed-point
// fraction of a turn per position, F_i = f_i / (2 pi) 2^64: the product p F_i
// wraps modulo one turn by itself, exactly, for any 64-bit p.  The nearest quarter
// turn comes off in integers too, so only the rest, an eighth of a turn at most, is
// rounded to fp32, relative to its own size: sines and cosines near zero keep their
// bits.  (Of the whole turn, fp32 is off by up to 9e-8 radians.)  What is left is
// F_i's own rounding, a double's: about p f_i 2^-53 radians.  The table comes with
// the launch as a parameter (128 entries at most), so the handle owns no device
// memory.
//
// What bounds it: HBM.  Per token the kernel reads 2 D bytes for each q, k and
// v head and writes 2 D for each q head and the codes and scales of k and v;
// about 3 flop a byte.  A warp takes one token (or a slice of its vectors, when
// there are too few tokens to fill the SMs), so the r/2 cosines and sines of the
// token are computed once by its 32 lanes and shared through shared memory by
// all of its heads; D/16 lanes then hold one vector, 16 elements each, both
// elements of a pair in the same lane, and the amax of a dynamic scale is a
// shuffle reduction in the group.
//
// Rounding: everything up to the result is fp32.  k goes into its quotient and
// code without a rounding to bf16 in between (one rounding fewer than a
// rotation followed by the cache write); a BF16 layer rounds once.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "kvq_internal.h"
#include "quantize.cuh"

namespace kvq {
namespace {

using namespace quant;

constexpr int RWARPS = 4;                      // warps per CTA, independent of one another

// fp32 pair -> bf16x2, round to nearest even; `lo` in the low half.
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(bf16x2(x[0], x[1]), bf16x2(x[2], x[3]), bf16x2(x[4], x[5]), bf16x2(x[6], x[7]));
}

// The same for values that are bf16 already: their upper halves, so that what passes
// through keeps its bits (the conversion makes every NaN the same).  Keeping the raw
// words instead took 8 registers more: 194 -> 218 us for the 32,768 tokens below.
__device__ __forceinline__ uint4 join8(const float* x) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    w[j] = __byte_perm(__float_as_uint(x[2 * j]), __float_as_uint(x[2 * j + 1]), 0x7632);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Rotates the lane's 16 elements: pair j is (x[j], x[8 + j]) in the half layout
// and (x[2j], x[2j + 1]) in the interleaved one.
template <int LAYOUT>
__device__ __forceinline__ void rotate(float* x, const float* c, const float* s) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int i0 = LAYOUT == ROPE_HALF ? j : 2 * j;
    const int i1 = LAYOUT == ROPE_HALF ? 8 + j : 2 * j + 1;
    const float a = x[i0], b = x[i1];
    x[i0] = fmaf(a, c[j], -b * s[j]);
    x[i1] = fmaf(a, s[j], b * c[j]);
  }
}

// Sine and cosine of u 2^-64 of a turn.
__device__ __forceinline__ void turn_sincos(unsigned long long u, float* sn, float* cn) {
  const unsigned quarter = (unsigned)((u + (1ull << 61)) >> 62);        // modulo 4
  const long long rest = (long long)(u - ((unsigned long long)quarter << 62));
  float s, c;
  sincospif((float)rest * 0x1p-63f, &s, &c);
  const float s1 = quarter & 1u ? c : s, c1 = quarter & 1u ? -s : c;
  *sn = quarter & 2u ? -s1 : s1;
  *cn = quarter & 2u ? -c1 : c1;
}

// Vectors a lane has in flight.  Measured, 32,768 tokens x 80 heads of 128: 2: 217 us,
// 3: 202, 4: 192 (99 % of the copy rate), 5: 191; 2,053 x 32 heads of 256: 2: 17.2,
// 4: 18.2 (a vector takes 16 lanes, and registers end the occupancy).
__host__ __device__ constexpr int in_flight(int D) { return D == 256 ? 2 : 4; }

template <int MODE, int D, int LAYOUT>
__global__ void __launch_bounds__(RWARPS * 32)
    rope_kernel(const RopeArgs a, const __grid_constant__ RopeTable tab) {
  constexpr int LPV = D / 16;                  // lanes per vector
  constexpr int GP = 32 / LPV;                 // vectors a warp holds at once
  constexpr int U = in_flight(D);              // and has in flight per lane
  constexpr int NP = D / 64;                   // pairs a lane computes the angle of
  __shared__ __align__(16) float2 cs_all[RWARPS][D / 2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane % LPV, gi = lane / LPV;
  float2* cs = cs_all[warp];
  const int pairs = a.rotary / 2;
  unsigned long long ph[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int p = lane + 32 * i;
    ph[i] = p < pairs ? tab.phase[p] : 0ull;
  }
  // the lane's two 8-element chunks: the two halves of its 8 pairs in the half
  // layout, neighbours otherwise (and where the head passes through)
  const bool rot = 8 * sub < pairs;
  int c0 = 2 * sub, c1 = 2 * sub + 1;
  if (LAYOUT == ROPE_HALF && rot) {
    c0 = sub;
    c1 = sub + a.rotary / 16;
  }
  const WriteArgs& w = a.w;
  const int hk = a.Hq + w.Hkv, nv = a.Hq + 2 * w.Hkv;
  const long long cells = w.num_blocks * w.bs;
  const unsigned items = (unsigned)w.T * (unsigned)a.slices;     // < 2^31 (host)
  for (unsigned it = blockIdx.x * RWARPS + warp; it < items; it += gridDim.x * RWARPS) {
    const unsigned t = it / (unsigned)a.slices;
    const int v0 = (int)(it - t * (unsigned)a.slices) * a.per_slice;
    const int v1 = min(nv, v0 + a.per_slice);
    const long long pos = a.positions[t];
    const long long slot = w.slots ? w.slots[t] : -1;
    const bool store = slot >= 0 && slot < cells;
    if (slot >= cells && v0 == 0 && lane == 0) atomicOr(w.err, ERR_BAD_INDEX);
    uint4 r0[U], r1[U];
    // the group's next vectors (the whole group agrees on `v`)
    auto load = [&](int v) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int vv = v + GP * u;
        if (vv >= v1 || (vv >= a.Hq && !store)) continue;
        const uint16_t* src =
            vv < a.Hq ? a.q + (long long)t * a.q_stride + (long long)vv * D
                      : (vv < hk ? w.k_new + (long long)t * w.token_stride + (long long)(vv - a.Hq) * D
                                 : w.v_new + (long long)t * w.token_stride + (long long)(vv - hk) * D);
        r0[u] = reinterpret_cast<const uint4*>(src)[c0];
        r1[u] = reinterpret_cast<const uint4*>(src)[c1];
      }
    };
    load(v0 + gi);                             // in flight while the angles are computed
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int p = lane + 32 * i;
      if (p < pairs) {
        float sn, cn;
        turn_sincos((unsigned long long)pos * ph[i], &sn, &cn);
        cs[p] = make_float2(cn * tab.magnitude, sn * a.sin_magnitude);
      }
    }
    __syncwarp();
    float c[8], s[8];
    if (rot) {
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const float4 q = *reinterpret_cast<const float4*>(cs + 8 * sub + j);
        c[j] = q.x; s[j] = q.y; c[j + 1] = q.z; s[j + 1] = q.w;
      }
    }
    __syncwarp();                              // cs may be overwritten by the next item
    const unsigned blk = (unsigned)((store ? slot : 0) >> w.bs_shift);
    const unsigned off = (unsigned)(store ? slot : 0) & (unsigned)(w.bs - 1);
    for (int v = v0 + gi; v < v1; v += GP * U) {
      if (v != v0 + gi) load(v);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int vv = v + GP * u;
        if (vv >= v1 || (vv >= a.Hq && !store)) continue;        // whole group agrees
        float x[16];
        unpack8(x, r0[u]);
        unpack8(x + 8, r1[u]);
        const bool turned = rot && vv < hk;
        if (turned) rotate<LAYOUT>(x, c, s);
        if (vv < a.Hq) {
          uint4* dst = reinterpret_cast<uint4*>(a.q_out + (long long)t * a.q_out_stride +
                                                (long long)vv * D);
          dst[c0] = turned ? pack8(x) : join8(x);
          dst[c1] = turned ? pack8(x + 8) : join8(x + 8);
          continue;
        }
        const int is_v = vv >= hk;
        const int h = vv - (is_v ? hk : a.Hq);
        const unsigned cell = ((blk * (unsigned)w.Hkv + (unsigned)h) << w.bs_shift) | off;
        uint8_t* cache = is_v ? w.v_cache : w.k_cache;
        if constexpr (MODE == BF16) {
          uint4* dst = reinterpret_cast<uint4*>(cache + (size_t)cell * (2 * D));
          dst[c0] = turned ? pack8(x) : join8(x);
          dst[c1] = turned ? pack8(x + 8) : join8(x + 8);
        } else {
          float sc;
          if constexpr (MODE == FP8_PER_TENSOR) {
            sc = __ldg(is_v ? w.v_scale : w.k_scale);
          } else if constexpr (MODE == FP8_PER_HEAD) {
            sc = __ldg((is_v ? w.v_scale : w.k_scale) + h);
          } else {
            float m = 0.f;
#pragma unroll
            for (int e = 0; e < 16; ++e) m = fmaxf(m, fabsf(x[e]));
            sc = dynamic_scale<MODE>(group_max<LPV>(m));
            if (sub == 0) (is_v ? w.v_cs : w.k_cs)[cell] = sc;
          }
          float y[16];
          divide_rn<MODE, 16>(y, x, sc);
          uint32_t code[4];
          encode<MODE, 16>(code, y);
          if constexpr (MODE == INT4_PER_TOKEN_HEAD) {
            uint32_t* dst = reinterpret_cast<uint32_t*>(cache + (size_t)cell * (D / 2));
            dst[c0] = code[0];
            dst[c1] = code[1];
          } else {
            uint2* dst = reinterpret_cast<uint2*>(cache + (size_t)cell * D);
            dst[c0] = make_uint2(code[0], code[1]);
            dst[c1] = make_uint2(code[2], code[3]);
          }
        }
      }
    }
  }
}

template <int MODE, int D, int LAYOUT>
cudaError_t launch_l(RopeArgs& a, const RopeTable& tab, cudaStream_t st) {
  // Work per warp: a token, or a slice of its vectors (GP at least, so that no lane
  // idles).  A warp's item costs its rounds of loads and about one more for the
  // angles; the cut that takes the fewest of them over the waves of resident warps
  // wins, the finer one where two cost the same (a decode step: one round per warp).
  // Measured, 2,053 tokens x 32 heads of 256, one slice (a wave): 17.1 us, two or
  // three (a second, partly filled wave): 18.8; 8,192 x 80 heads of 64: 30.4 and 32.3.
  constexpr int GP = 32 / (D / 16);
  const int nv = a.Hq + 2 * a.w.Hkv;
  constexpr int ROUND = GP * in_flight(D);                     // vectors a warp loads at once
  const long long warps = (long long)sm_count() * 16;          // resident (97-117 registers)
  // more than two waves of slices of a vector group never win
  const int most = (int)std::min((long long)(nv + GP - 1) / GP, 2 * warps / a.w.T + 1);
  int per = 0;
  long long best = 0;
  for (int s = most; s >= 1; --s) {
    const int p = ((nv + s - 1) / s + GP - 1) / GP * GP;
    const long long items = a.w.T * ((nv + p - 1) / p);
    const long long cost = (items + warps - 1) / warps * ((p + ROUND - 1) / ROUND + 1);
    if (per == 0 || cost < best) {
      best = cost;
      per = p;
    }
  }
  a.per_slice = per;
  a.slices = (nv + per - 1) / per;
  const long long items = a.w.T * a.slices;
  if (items >= (1LL << 31)) return cudaErrorInvalidValue;
  long long grid = (items + RWARPS - 1) / RWARPS;
  // two waves of CTAs and no more: a warp then carries its frequencies over several
  // items (16 or 64 per SM measured 1 to 4 % slower)
  const long long cap = (long long)sm_count() * 8;
  if (grid > cap) grid = cap;
  rope_kernel<MODE, D, LAYOUT><<<(unsigned)grid, RWARPS * 32, 0, st>>>(a, tab);
  return cudaGetLastError();
}

template <int MODE, int D>
cudaError_t launch_d(RopeArgs& a, const RopeTable& tab, int layout, cudaStream_t st) {
  return layout == ROPE_HALF ? launch_l<MODE, D, ROPE_HALF>(a, tab, st)
                             : launch_l<MODE, D, ROPE_INTERLEAVED>(a, tab, st);
}

template <int MODE>
cudaError_t launch_m(int D, RopeArgs& a, const RopeTable& tab, int layout, cudaStream_t st) {
  switch (D) {
    case 64: return launch_d<MODE, 64>(a, tab, layout, st);
    case 128: return launch_d<MODE, 128>(a, tab, layout, st);
    case 256: return launch_d<MODE, 256>(a, tab, layout, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_rope(int mode, int D, int layout, RopeArgs a, const RopeTable& tab,
                        cudaStream_t st) {
  if (a.w.T == 0) return cudaSuccess;
  switch (mode) {
    case BF16: return launch_m<BF16>(D, a, tab, layout, st);
    case FP8_PER_TENSOR: return launch_m<FP8_PER_TENSOR>(D, a, tab, layout, st);
    case FP8_PER_HEAD: return launch_m<FP8_PER_HEAD>(D, a, tab, layout, st);
    case FP8_PER_TOKEN_HEAD: return launch_m<FP8_PER_TOKEN_HEAD>(D, a, tab, layout, st);
    case INT4_PER_TOKEN_HEAD: return launch_m<INT4_PER_TOKEN_HEAD>(D, a, tab, layout, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace kvq
