// Quantization of one head vector held by a group of lanes, shared by the cache
// write and its rotary form: bf16 unpacking, the group's amax, the dynamic
// scale, the correctly rounded quotient and the E4M3 / INT4 codes.
#pragma once

#include <stdint.h>

#include "kvq_internal.h"

namespace kvq {
namespace quant {

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Two fp32 -> two E4M3 codes, round to nearest even, saturating to +-448
// (hardware cvt with .satfinite).  `lo` lands in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Max over the LPV lanes of one vector group.  Groups of one warp may take
// different paths (a skipped slot, the end of the grid-stride loop), so the
// shuffle names only the group's own lanes.
template <int LPV>
__device__ __forceinline__ float group_max(float v) {
  const unsigned lane = threadIdx.x & 31u;
  const unsigned mask = (LPV == 32) ? 0xffffffffu
                                    : (((1u << LPV) - 1u) << (lane & ~(unsigned)(LPV - 1)));
#pragma unroll
  for (int o = LPV / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(mask, v, o));
  return v;
}

// Unpacks 8 bf16 (one 16-byte word group) to fp32.
__device__ __forceinline__ void unpack8(float* x, const uint4 raw) {
  x[0] = bf16_lo(raw.x); x[1] = bf16_hi(raw.x);
  x[2] = bf16_lo(raw.y); x[3] = bf16_hi(raw.y);
  x[4] = bf16_lo(raw.z); x[5] = bf16_hi(raw.z);
  x[6] = bf16_lo(raw.w); x[7] = bf16_hi(raw.w);
}

// Dynamic scale from the vector's amax: s = RN32(amax / qmax), 1.0 for a zero
// vector.  Computed by the reciprocal correction below (exact for every bf16
// amax >= 2^-100); IEEE division under that.
template <int MODE>
__device__ __forceinline__ float dynamic_scale(float m) {
  constexpr float qmax = (MODE == INT4_PER_TOKEN_HEAD) ? 7.0f : 448.0f;
  constexpr float rq = 1.0f / qmax;                         // RN(1/qmax)
  if (m >= 0x1p-100f) {
    const float q0 = __fmul_rn(m, rq);
    return __fmaf_rn(__fmaf_rn(-q0, qmax, m), rq, q0);
  }
  return (m == 0.f) ? 1.0f : __fdiv_rn(m, qmax);
}

// y = RN32(x / s).  One correctly rounded reciprocal per vector, then per
// element q0 = RN(x r) and the FMA correction q1 = RN(q0 + RN(x - q0 s) r),
// which is the correctly rounded quotient while the remainder x - q0 s is
// exact (Markstein's theorem: r within half an ulp of 1/s, q0 within an ulp).
// That holds away from fp32 underflow; below the guard the kernel divides.
// Verified equal to IEEE division over every dynamic scale (every bf16 amax,
// /448 and /7, every bf16 |x| <= amax) where the result decides a code, and
// over random static scales.  With a static scale the quotient can be huge;
// past 1e30 it saturates either way, so the correction is skipped there.
// With a dynamic scale |x/s| <= qmax (1 + 2^-23), so no guard is needed.
template <int MODE, int N>
__device__ __forceinline__ void divide_rn(float* y, const float* x, float s) {
  constexpr bool DYN = (MODE == FP8_PER_TOKEN_HEAD || MODE == INT4_PER_TOKEN_HEAD);
  constexpr float kLo = DYN ? 0x1p-100f : 0x1p-60f;
  if (s >= kLo && s <= 0x1p100f) {
    const float r = __frcp_rn(s);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float q0 = __fmul_rn(x[i], r);
      const float q1 = __fmaf_rn(__fmaf_rn(-q0, s, x[i]), r, q0);
      y[i] = (DYN || fabsf(q0) < 1e30f) ? q1 : q0;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) y[i] = __fdiv_rn(x[i], s);
  }
}

// Codes of N quotients: E4M3 bytes (N/4 words) or packed INT4 nibbles, even
// element in the low nibble (N/8 words).
//
// INT4: for |y| < 2^22, RN(y + 1.5 * 2^23) = 1.5 * 2^23 + RNE(y) exactly (the
// sum's ulp is 1, ties go to the even significand, i.e. to even RNE(y)), and
// the bit pattern of that float is the pattern of 1.5 * 2^23 (low bits 0)
// plus RNE(y), so its low four bits are RNE(y) as a two's-complement nibble.
// The per-token-head scale keeps |y| <= 7 (1 + 2^-23) (s = RN(amax / 7),
// |x| <= amax, and the scale's rounding error is far below 1/14 down to the
// smallest bf16 amax), so RNE(y) already lies in [-7, 7] and needs no clamp.
template <int MODE, int N>
__device__ __forceinline__ void encode(uint32_t* w, const float* y) {
  if constexpr (MODE == INT4_PER_TOKEN_HEAD) {
    constexpr float kRound = 12582912.0f;                     // 1.5 * 2^23
#pragma unroll
    for (int k = 0; k < N / 8; ++k) {
      uint32_t b[4];                                          // byte j in the low 8 bits
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t lo = __float_as_uint(__fadd_rn(y[8 * k + 2 * j], kRound));
        const uint32_t hi = __float_as_uint(__fadd_rn(y[8 * k + 2 * j + 1], kRound));
        b[j] = (lo & 0x0Fu) | ((hi << 4) & 0xF0u);
      }
      w[k] = __byte_perm(__byte_perm(b[0], b[1], 0x0040u), __byte_perm(b[2], b[3], 0x0040u),
                         0x5410u);
    }
  } else {
#pragma unroll
    for (int k = 0; k < N / 4; ++k)
      w[k] = e4m3x2(y[4 * k], y[4 * k + 1]) | (e4m3x2(y[4 * k + 2], y[4 * k + 3]) << 16);
  }
}

}  // namespace quant
}  // namespace kvq
