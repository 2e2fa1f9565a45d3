// The warp-specialised attention kernel over the paged cache, shared by the
// prefill (causal) and the cross attention (CROSS): its tile shapes and the
// kernel.  The file that launches the prefill describes its roles.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "async_copy.cuh"
#include "kvq_internal.h"
#include "prefill_common.cuh"
#include "tcgen05.cuh"
#include "tile_math.cuh"

namespace kvq {
namespace {

constexpr int WS_CONV = 4;                          // warps of a converter group
constexpr int WROWS = 128;                          // rows per query tile (the MMA's M)

// A 16-byte shared-memory load that stays after the tensor-memory stores
// issued before it (both are volatile asm): the softmax reads the
// scales of 16 keys ahead of their use, instead of the compiler hoisting all
// sixteen loads of a tile to its start, where their 64 registers pushed the
// thread past its 128-register share and spilled.
__device__ __forceinline__ float4 lds_v4_ordered(const float4* p) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"((uint32_t)__cvta_generic_to_shared(p)));
  return v;
}

// 32 values of an output row: rounded to bf16, or as they are.
__device__ __forceinline__ void store_row_bf16(uint16_t* row, const float (&v)[32]) {
  uint4* dst = reinterpret_cast<uint4*>(row);
#pragma unroll
  for (int e = 0; e < 4; ++e)
    dst[e] = make_uint4(pack_bf16x2(v[8 * e], v[8 * e + 1]), pack_bf16x2(v[8 * e + 2], v[8 * e + 3]),
                        pack_bf16x2(v[8 * e + 4], v[8 * e + 5]), pack_bf16x2(v[8 * e + 6], v[8 * e + 7]));
}

__device__ __forceinline__ void store_row_f32(float* row, const float (&v)[32]) {
  float4* dst = reinterpret_cast<float4*>(row);
#pragma unroll
  for (int e = 0; e < 8; ++e) dst[e] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
}

// A warpgroup's registers a thread, from here on.
template <int N>
__device__ __forceinline__ void give_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void take_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// Warp roles: NQ query tiles per CTA (two at head_dim 64 and 128; one at 256,
// whose O needs 256 tensor-memory columns), a softmax warpgroup per query
// tile, then the converters, the producer and two MMA issuers, of S and of PV
// (FEW: one of both).
// FEW (at most 128 rows): one query tile, built at head_dim 64 and 128, and two converter
// groups that take key tiles in turn.  With one query tile a key tile's
// conversion (1,500 cycles by one group) is a longer step than its MMAs, so the
// second softmax warpgroup's place goes to a second converter.
template <int MODE, int D, bool FEW>
struct WRoles {
  static constexpr int NQ = (D == 256 || FEW) ? 1 : 2;
  static constexpr int CG = FEW ? 2 : 1;             // converter groups
  static constexpr int SOFT = 4 * NQ;                // softmax warps
  static constexpr int PROD = SOFT + CG * WS_CONV;   // producer warp
  static constexpr int MMA_S = PROD + 1;             // warp that issues S
  static constexpr int MMA_PV = FEW ? MMA_S : PROD + 2;   // and the one that issues PV
  // Two query tiles and a scale per key: four warpgroups (warp 15 only completes
  // the fourth), whose registers move to the softmax: its 64 scores, the scales
  // ahead and its sums spilled in an even share of 128, and the other roles need
  // fewer.  Cross attention of 8 x 900-1,024 queries to 3,000-4,096 states, 32 heads
  // of 128: 412 -> 398 us; prefill per token and head 603 -> 621 TFLOP/s, INT4 583 ->
  // 588; without scales per key the softmax has room, and the same split measured
  // 727 -> 712 (per head) and 574 -> 568 (BF16).
  // The shares add up to what the block is launched with, or the softmax would
  // wait for registers that nobody gives up.
  static constexpr bool SPLIT_REGS =
      NQ == 2 && (MODE == FP8_PER_TOKEN_HEAD || MODE == INT4_PER_TOKEN_HEAD);
  static constexpr int THREADS = SPLIT_REGS ? 512 : (MMA_PV + 1) * 32;   // 512, 480, 448 or 352
  static constexpr int REGS = 128;                   // a thread at launch (SPLIT_REGS)
  static constexpr int REGS_SOFT = 168, REGS_CONV = 112, REGS_REST = 64;
  static_assert(!SPLIT_REGS || 2 * REGS_SOFT + REGS_CONV + REGS_REST == 4 * REGS, "register shares");
  static_assert(!SPLIT_REGS || (SOFT == 8 && PROD == 12 && THREADS == 16 * 32), "whole warpgroups");
};
constexpr int WKT = 64;                             // keys per tile
constexpr float NO_KEY = -INFINITY;                 // K scale that masks a key (0 is a scale: its scores are 0)
constexpr int WKP = 6;                              // P' = p v_scale 2^(WKP - vexp) < 2^15 (p <= 2^8)
constexpr float WLAZY = 8.f;                        // the reference max moves when exceeded by this
// static FP8 scales: P' = p x 2^6 (< 2^14)
constexpr int CONV_BAR = 1;                         // named barriers of the converter groups (1, 2)
constexpr int JOIN_BAR = 3;                         // and of the softmax warps (FEW's epilogue)
constexpr int Q_BAR = 4;                            // the queries are in place

template <int MODE, int D, bool FEW>
struct WCfg {
  static constexpr int RB = row_bytes<MODE>(D);
  static constexpr int TB = 16 * RB;                       // one page tile (16 positions)
  static constexpr int TBP = (TB + 1023) / 1024 * 1024;
  // scales copied from the cache with the codes (dynamic FP8, INT4)
  static constexpr bool FETCH = (MODE == FP8_PER_TOKEN_HEAD || MODE == INT4_PER_TOKEN_HEAD);
  // BF16 layers: K stays bf16 (S is a bf16 MMA against bf16 queries); each V
  // row is scaled by the power of two that maps its largest exponent to 2^14
  // and converted to f16 exactly, and its V scale is that power's inverse
  static constexpr bool BFK = (MODE == BF16);
  // per-key V scales in the scale buffer, followed by the softmax's range factor
  static constexpr bool DYN = FETCH || BFK;
  static constexpr int SUB = WKT / 16;                      // page tiles per key tile
  // BF16 at head_dim 128: K is copied straight into its operand buffer, which
  // halves the raw stage so that three raw stages and three operand buffers
  // fit (two and two otherwise); at 256 two and two fit only so.  At 64 both
  // already fit three and four, and the producer keeps its four-stage
  // lookahead by staging K like V.
  static constexpr bool KDIRECT = BFK && D >= 128;
  // a raw stage: the K and V page tiles of a key tile (V only with KDIRECT),
  // then their scales
  static constexpr int RAW = (KDIRECT ? 1 : 2) * SUB * TBP;
  static constexpr int VOFF = KDIRECT ? 0 : SUB * TBP;      // V page tiles in a raw stage
  static constexpr int SCB = FETCH ? 2 * SUB * 64 : 0;
  static constexpr int RAWS = (RAW + SCB + 1023) / 1024 * 1024;
  static constexpr int NQ = WRoles<MODE, D, FEW>::NQ;
  static constexpr int QB = WROWS * D * 2;                  // one query tile: D/64 blocks of 128 x 128 B
  // queries in shared memory (two query tiles); with one query tile they live
  // in tensor memory instead, the A operand of S
  static constexpr int QSM = (NQ == 2) ? 2 * QB : 0;
  static constexpr int KB = WKT * D * 2;                    // one K buffer: D/64 blocks of 64 x 128 B
  static constexpr int VTB = WKT * D * 2;                   // one V buffer, as K
  // one scale buffer: K scales, V scales, then ints: V-scale exponent of
  // each 32-key half, whether every page tile was fetched
  static constexpr int SCS = 2 * WKT * 4 + 16;
  static constexpr int ROWB = 2 * 2 * WROWS * 4;            // row factor and position per row
  static constexpr int BARB = 32 * 8;                       // barriers
  static constexpr int LIMIT = 232448 - 1024;               // per-CTA shared memory, minus slack
  // operand buffers (K, V, scales): three when they fit beside two raw stages.
  // FEW: buffers and stages are even in number, so that each converter group
  // owns every second one and waits for each of their phases.
  static constexpr int fixed_of(int nb) { return QSM + nb * (KB + VTB + SCS) + ROWB + BARB + 64; }
  static constexpr bool fits(int nb, int nr) { return fixed_of(nb) + nr * RAWS <= LIMIT; }
  static constexpr int NB = FEW ? (fits(4, 2) ? 4 : 2) : (fits(3, 2) ? 3 : 2);
  static constexpr int FIXED = fixed_of(NB);
  static constexpr int NR = fits(NB, 4) ? 4 : ((!FEW && fits(NB, 3)) ? 3 : 2);
  static constexpr int SMEM = NR * RAWS + FIXED + 1024;
  // Tensor-memory columns.  S/P' buffer b of query tile j: S (fp32, 64
  // columns), then P' (f16 hi in the first 32 columns, lo in the next 32) in
  // its place.  Two query tiles: S/P' at 64 (2 j + b), O_j at 256 + D j.  One
  // query tile (D 256, FEW): O at 0, S/P' at 256 + 64 b, Q (f16, D / 2 columns)
  // at 384.
  __host__ __device__ static constexpr int scol(int j, int b) { return NQ == 2 ? 64 * (2 * j + b) : 256 + 64 * b; }
  __host__ __device__ static constexpr int ocol(int j) { return NQ == 2 ? 256 + D * j : 0; }
  static constexpr int QCOL = 384;
  static constexpr int TCOLS = 512;
  static_assert(NQ == 2 ? 256 + 2 * D <= TCOLS : QCOL + D / 2 <= TCOLS, "tensor memory");
  static_assert(SMEM <= 232448, "shared memory");
  static_assert(!FEW || WROWS * (D + 1) * 4 <= NR * RAWS + NB * (KB + VTB), "the copies' O");
};

// CROSS false: causal prefill, G query heads per KV head, fp32 output.
// CROSS true: attention to all positions of the sequence (no mask), 2^g_shift
// query heads per KV head, bf16 output, the keys cut into splits; FEW as above.
template <int MODE, int D, int G, bool CROSS = false, bool FEW = false>
__global__ void __launch_bounds__(WRoles<MODE, D, FEW>::THREADS, 1)
    prefill_ws_kernel(const PrefillArgs pa, const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap) {
  using C = WCfg<MODE, D, FEW>;
  using RL = WRoles<MODE, D, FEW>;
  constexpr int NQ = RL::NQ;
  const DecodeArgs& a = pa.d;
  constexpr int SUB = C::SUB;
  constexpr int NR = C::NR;
  constexpr int NB = C::NB;
  // positions per query tile.  Row r of a tile is head r / QP of position r % QP
  // (causal: a tile's rows then cover few positions of many heads alike) or
  // head r % heads of position r / heads (CROSS: the rows in use come first, so
  // that few queries leave whole softmax warps idle)
  const int heads = CROSS ? 1 << pa.g_shift : (G > 0 ? G : 1);
  const int QP = CROSS ? WROWS >> pa.g_shift : WROWS / (G > 0 ? G : 1);
  auto row_head = [&](int r) { return CROSS ? r & (heads - 1) : r / QP; };
  auto row_query = [&](int r) { return CROSS ? r >> pa.g_shift : r - (r / QP) * QP; };
  constexpr int PTERMS = CROSS ? 1 : 2;        // f16 terms of P' (see the softmax)
  constexpr int CPR = C::RB / 16;              // 16-byte raw chunks per position row
  constexpr int EPC = (MODE == INT4_PER_TOKEN_HEAD) ? 32 : (MODE == BF16 ? 8 : 16);   // elements per raw chunk

  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* raw = smem;                                       // NR stages
  uint8_t* q16 = raw + NR * C::RAWS;                         // 2 query tiles (none for NQ 1)
  uint8_t* k16 = q16 + C::QSM;                               // NB K buffers
  uint8_t* vt16 = k16 + NB * C::KB;                          // NB V buffers
  uint8_t* scb = vt16 + NB * C::VTB;                         // NB scale buffers
  float* rowf = reinterpret_cast<float*>(scb + NB * C::SCS); // [2][128] score factor per row
  int* rowp = reinterpret_cast<int*>(rowf + 2 * WROWS);      // [2][128] position (-1: no row)
  uint64_t* bars = reinterpret_cast<uint64_t*>(rowp + 2 * WROWS);
  uint64_t* raw_full = bars;                                 // [NR] producer -> converters
  uint64_t* raw_empty = raw_full + NR;                       // [NR] converters -> producer
  uint64_t* kv_full = raw_empty + NR;                        // [NB] converters -> MMA
  uint64_t* kv_empty = kv_full + NB;                         // [NB] MMA (commit) -> converters
  uint64_t* s_full = kv_empty + NB;                          // [2][2] MMA (commit) -> softmax j, per S buffer
  // P' of query tile j in S/P' buffer b: [2][2], 128 arrivals each.  One
  // barrier per buffer: a softmax warpgroup may finish key tile t + 1 before
  // the MMA issuer waits for its tile t, and a barrier per query tile would
  // then complete two phases ahead of its waiter.
  uint64_t* p_full = s_full + 4;
  // PV (commit) -> S issuer and softmax j, per S/P' buffer for the same reason
  uint64_t* pv_done = p_full + 4;
  uint64_t* o_fin = pv_done + 4;                             // PV (commit) -> softmax, at the end
  uint64_t* s_fin = o_fin + 1;                               // the S issuer's own end
  static_assert(2 * NR + 2 * NB + 3 * 4 + 2 <= 32, "barriers");
  int* s_have = reinterpret_cast<int*>(bars + 32);           // [NR] fetched page tiles per stage
  volatile int* s_abort = s_have + 4;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(s_have + 5);

  // the warp index through a shuffle: the compiler then knows that the role
  // branches are warp-uniform (descriptors stay in uniform registers, and the
  // softmax no longer spills)
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);

  // the kernel that joins the splits may be launched; it waits for this grid
  if constexpr (CROSS) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // ---- this CTA's (sequence, KV head, pair of query tiles); latest first.
  // CROSS: the query tiles of one (split, sequence, KV head) are neighbours, so
  // that they read its pages from L2.
  const int per_tile = a.B * a.Hkv;
  const int ct = CROSS ? (int)(blockIdx.x % pa.qtiles) : pa.qtiles - 1 - (int)(blockIdx.x / per_tile);
  const int rem = CROSS ? (int)(blockIdx.x / pa.qtiles) % per_tile : (int)(blockIdx.x % per_tile);
  const int split = CROSS ? (int)(blockIdx.x / pa.qtiles) / per_tile : 0;
  const int b = rem / a.Hkv, g = rem - b * a.Hkv;
  const int q0 = pa.query_start[b];
  int n_b = pa.query_start[b + 1] - q0;
  const int L = a.context_lens[b];
  if constexpr (CROSS) {
    if (n_b > pa.max_query) {                               // rows past the caller's bound
      if (tid == 0) atomicOr(a.err, ERR_BAD_INDEX);
      n_b = pa.max_query;
    }
  }
  if (ct * NQ * QP >= n_b || n_b <= 0) return;              // whole CTA: before any barrier
  if (L < (CROSS ? 0 : n_b) || (long long)L > ((long long)a.max_blocks << a.bs_shift)) {
    if (tid == 0) atomicOr(a.err, ERR_BAD_INDEX);
    return;
  }
  const int qbase = ct * NQ * QP;                           // query index of tile 0, row 0
  const int nq = min(NQ * QP, n_b - qbase);                 // valid query positions here
  const int nqt = (CROSS && nq <= QP) ? 1 : NQ;             // query tiles with rows in use
  // FEW: 64 rows or fewer stand in the tile two or four times (copy c in the
  // warps from 4 c / copies on), and the softmax of a copy takes its share of a
  // key tile's keys, so that every SM sub-partition works on the exponents; the
  // copies' O are joined in the epilogue like splits.
  const int copies_shift = !FEW ? 0 : (nq * heads <= 32 ? 2 : (nq * heads <= 64 ? 1 : 0));
  const int copy_rows = WROWS >> copies_shift;
  int first, pmax, kmin;                                    // first query's position; keys [kmin, pmax]
  bool whole = true;                                        // this CTA sees every key (CROSS)
  if constexpr (CROSS) {
    const int tiles = (L + WKT - 1) / WKT;
    if (tiles == 0) {                                       // no keys: zeros
      if (split == 0)
        for (int i = tid; i < nq * heads * (D / 8); i += RL::THREADS) {
          const int row = i / (D / 8), c = i - row * (D / 8);
          reinterpret_cast<uint4*>(a.out_bf16 + ((long long)(q0 + qbase + row_query(row)) * a.Hq +
                                                 g * heads + row_head(row)) * D)[c] =
              make_uint4(0u, 0u, 0u, 0u);
        }
      return;
    }
    const int ts = split * pa.split_tiles;
    if (ts >= tiles) return;
    const bool last = split == pa.splits - 1;
    whole = pa.splits <= 1 || tiles <= pa.split_tiles;
    kmin = ts * WKT;
    pmax = (last ? L : min(L, (ts + pa.split_tiles) * WKT)) - 1;
    first = pmax;                                           // every row sees the same keys
  } else {
    first = L - n_b + qbase;
    pmax = first + nq - 1;
    kmin = (a.window > 0) ? max(0, first + 1 - a.window) : 0;
  }
  const int t0 = kmin / WKT, t1 = pmax / WKT;               // key tiles, inclusive
  const int ntl = t1 - t0 + 1;

  if (warp == RL::PROD && elect_one()) {
    prefetch_map(&kmap);
    prefetch_map(&vmap);
  }
  if (tid == 0) {
    for (int s = 0; s < NR; ++s) {
      mbar_init(&raw_full[s], 1);
      mbar_init(&raw_empty[s], 1);
    }
    for (int s = 0; s < NB; ++s) {
      mbar_init(&kv_full[s], 1);
      mbar_init(&kv_empty[s], 1);
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&p_full[s], 4 * 32);
    }
    for (int s = 0; s < 4; ++s) mbar_init(&pv_done[s], 1);
    mbar_init(o_fin, 1);
    mbar_init(s_fin, 1);
    mbar_init_fence();
    *s_abort = 0;
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(s_tmem)),
                 "r"(C::TCOLS));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;

  // ---- queries: row R = 128 j + r of query tile j -> query index
  // qbase + j * QP + row_query(r), head g * heads + row_head(r), prescaled
  // by a power of two so the bf16 values are exact in f16 (BF16 layers: the bf16
  // values as they are).
  float ks_static = 1.f;
  if constexpr (MODE == FP8_PER_TENSOR) ks_static = a.k_scale[0];
  if constexpr (MODE == FP8_PER_HEAD) ks_static = a.k_scale[g];
  // The producer needs none of this and starts its copies at once; converters
  // take their share of the rows and go on.  Several rows are loaded at a time:
  // one after the other, their latencies added up to 7 us of a CTA.
  if constexpr (NQ == 2) {
    // into shared memory (K-major, 128-byte swizzle); lane l holds elements
    // l D / 32 ... of a row
    if (warp != RL::PROD) {
      constexpr int QW = RL::THREADS / 32 - 1;               // warps that load
      constexpr int W = D / 64;                              // words (bf16 pairs) per lane
      constexpr int UR = 8;                                  // rows in flight per warp
      const int w0 = warp - (warp > RL::PROD ? 1 : 0);
      for (int Rb = w0; Rb < nqt * WROWS; Rb += UR * QW) {
        uint32_t x[UR][W];
#pragma unroll
        for (int u = 0; u < UR; ++u) {
          const int R = Rb + u * QW;
          const int j = R / WROWS, r = R - j * WROWS;
          const int qi = j * QP + row_query(r);              // query index within the CTA
#pragma unroll
          for (int e = 0; e < W; ++e) x[u][e] = 0u;
          if (R < nqt * WROWS && qi < nq) {
            const uint16_t* src = a.q + ((long long)(q0 + qbase + qi) * a.Hq + g * heads + row_head(r)) * D;
            if constexpr (W == 2) {
              const uint2 v = reinterpret_cast<const uint2*>(src)[lane];
              x[u][0] = v.x;
              x[u][W - 1] = v.y;
            } else {
              x[u][0] = reinterpret_cast<const uint32_t*>(src)[lane];
            }
          }
        }
#pragma unroll
        for (int u = 0; u < UR; ++u) {
          const int R = Rb + u * QW;
          if (R >= nqt * WROWS) break;
          const int j = R / WROWS, r = R - j * WROWS;
          const int qi = j * QP + row_query(r);
          float amax = 0.f;
#pragma unroll
          for (int e = 0; e < W; ++e)
            amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(x[u][e] << 16)),
                                     fabsf(__uint_as_float(x[u][e] & 0xFFFF0000u))));
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
          int qexp = 0;
          if (amax > 0.f) qexp = max(((int)(__float_as_uint(amax) >> 23) & 0xFF) - 127, -100);
          if constexpr (C::BFK) qexp = 14;
          const float qmul = pow2i(14 - qexp);
          uint32_t y[W];
#pragma unroll
          for (int e = 0; e < W; ++e)
            y[e] = C::BFK ? x[u][e]
                          : pack_f16x2(__uint_as_float(x[u][e] << 16) * qmul,
                                       __uint_as_float(x[u][e] & 0xFFFF0000u) * qmul);
          const int d = lane * (2 * W);
          uint8_t* dst = q16 + j * C::QB + (d >> 6) * (WROWS * 128) + swc(r, (d & 63) >> 3) + (d & 7) * 2;
          if constexpr (W == 2) *reinterpret_cast<uint2*>(dst) = make_uint2(y[0], y[W - 1]);
          else *reinterpret_cast<uint32_t*>(dst) = y[0];
          if (lane == 0) {
            rowf[R] = a.qk_scale * ks_static * pow2i(qexp - 14);
            rowp[R] = qi < nq ? (CROSS ? first : first + qi) : -1;
          }
        }
      }
    }
  } else {
    // into tensor memory, the A operand of S: the softmax warps' thread r
    // owns row r (its lane) and stores its D / 2 f16 pairs as columns
    if (warp < RL::SOFT) {
      const int r = warp * 32 + lane;
      const int rr = FEW ? r & (copy_rows - 1) : r;
      const int h = row_head(rr), i = row_query(rr);
      const bool valid = i < nq;
      const uint4* src = reinterpret_cast<const uint4*>(
          a.q + ((long long)(q0 + qbase + (valid ? i : 0)) * a.Hq + g * heads + h) * D);
      constexpr int HELD = D <= 128 ? D / 8 : 16;  // chunks kept in registers between the passes
      uint4 q8[HELD];
      float amax = 0.f;
#pragma unroll
      for (int cb = 0; cb < D / 8; cb += HELD) {
#pragma unroll
        for (int c = 0; c < HELD; ++c) q8[c] = valid ? src[cb + c] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int c = 0; c < HELD; ++c) {
          const uint32_t w4[4] = {q8[c].x, q8[c].y, q8[c].z, q8[c].w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(w4[e] << 16)),
                                     fabsf(__uint_as_float(w4[e] & 0xFFFF0000u))));
        }
      }
      int qexp = 0;
      if (amax > 0.f) qexp = max(((int)(__float_as_uint(amax) >> 23) & 0xFF) - 127, -100);
      if constexpr (C::BFK) qexp = 14;
      const float qmul = pow2i(14 - qexp);
      const uint32_t trq = tmem + ((uint32_t)(warp * 32) << 16) + C::QCOL;
#pragma unroll
      for (int cb = 0; cb < D / 8; cb += HELD) {
        if constexpr (HELD < D / 8) {
#pragma unroll
          for (int c = 0; c < HELD; ++c) q8[c] = valid ? src[cb + c] : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int c4 = 0; c4 < HELD; c4 += 4) {     // 16 columns = 32 elements at a time
          uint32_t wq[16];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint32_t w4[4] = {q8[c4 + c].x, q8[c4 + c].y, q8[c4 + c].z, q8[c4 + c].w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
              wq[4 * c + e] = C::BFK ? w4[e]
                                     : pack_f16x2(__uint_as_float(w4[e] << 16) * qmul,
                                                  __uint_as_float(w4[e] & 0xFFFF0000u) * qmul);
          }
          tmem_st16_nowait(trq + (cb + c4) * 4, wq);
        }
      }
      tmem_wait_st();
      rowf[r] = a.qk_scale * ks_static * pow2i(qexp - 14);
      rowp[r] = valid ? (CROSS ? first : first + i) : -1;
    }
  }
  // Q and the rows' factors are in place for the S issuer and the softmax
  constexpr int Q_THREADS = (NQ == 2 ? RL::THREADS - 32 : (RL::SOFT + 1) * 32);
  if (warp < RL::SOFT || warp == RL::MMA_S) {
    fence_proxy_async();
    tc_fence_before();
    named_sync(Q_BAR, Q_THREADS);
    tc_fence_after();
  } else if (NQ == 2 && warp != RL::PROD) {
    fence_proxy_async();
    named_arrive(Q_BAR, Q_THREADS);
  }

  // ================================================================ roles
  // A warpgroup's registers move where its branch begins, so that its four warps run
  // one and the same setmaxnreg (it is undefined where they differ); warp 15 of
  // SPLIT_REGS only completes the last one.
  if (warp >= RL::PROD) {
    if constexpr (RL::SPLIT_REGS) give_registers<RL::REGS_REST>();
    if (warp == RL::PROD) {
      // ---- producer: key tile t into raw stage (t - t0) % NR, page tile by page
      // tile.  Page tiles wholly outside [kmin, pmax] are not fetched.  The block
      // ids of 32 page tiles are loaded at once, one per lane and a round ahead, and
      // every copy is issued by an elected lane from warp-uniform operands (copies
      // issued by the page tiles' own lanes took a loop over the lanes each).
      int last[NR];                                  // tile index last issued into each stage
#pragma unroll
      for (int s = 0; s < NR; ++s) last[s] = -1;
      // block of page tile 32 c + lane (counted from the first key tile): -1 where
      // nothing is to be fetched
      auto block_ids = [&](int c) -> int {
        const int pt = 32 * c + lane;
        const int pos = t0 * WKT + 16 * pt;
        if (pt >= SUB * ntl || pos + 16 <= kmin || pos > pmax) return -1;
        const int blk = __ldg(a.block_table + (long long)b * a.max_blocks + (pos >> a.bs_shift));
        if (blk >= 0 && blk < a.num_blocks) return blk;
        atomicOr(a.err, ERR_BAD_INDEX);
        return -1;
      };
      int ids = block_ids(0), ids_next = block_ids(1);
      unsigned live = __ballot_sync(0xffffffffu, ids >= 0);
      for (int i = 0; i < ntl; ++i) {
        const int st = i % NR;
        if (i >= NR) {
          const bool ok = mbar_wait(&raw_empty[st], (uint32_t)((i / NR - 1) & 1));
          if (!__all_sync(0xffffffffu, ok)) {
            if (lane == 0) { *s_abort = 1; atomicOr(a.err, ERR_TIMEOUT); }
            break;
          }
        }
        if constexpr (C::KDIRECT) {
          // K lands in operand buffer i % NB: wait until the MMAs of its last
          // tile are done with it
          if (i >= NB) {
            const bool ok = mbar_wait(&kv_empty[i % NB], (uint32_t)((i / NB - 1) & 1));
            if (!__all_sync(0xffffffffu, ok)) {
              if (lane == 0) { *s_abort = 1; atomicOr(a.err, ERR_TIMEOUT); }
              break;
            }
          }
        }
        if (__any_sync(0xffffffffu, *s_abort)) break;
        const int at = (SUB * i) & 31;               // the tile's page tiles among the 32
        if (at == 0 && i > 0) {
          ids = ids_next;
          live = __ballot_sync(0xffffffffu, ids >= 0);
          ids_next = block_ids(SUB * i / 32 + 1);
        }
        const unsigned fetch = (live >> at) & ((1u << SUB) - 1u);
        uint8_t* base = raw + st * C::RAWS;
        fence_proxy_async();
        if (elect_one()) {
          s_have[st] = (int)fetch;
          mbar_expect_tx(&raw_full[st], (uint32_t)__popc(fetch) * (2 * C::TB + (C::FETCH ? 128 : 0)));
        }
        __syncwarp();
#pragma unroll
        for (int s = 0; s < SUB; ++s) {
          const unsigned blk = (unsigned)__shfl_sync(0xffffffffu, ids, at + s);
          if (((fetch >> s) & 1u) && elect_one()) {
            const int pos = (t0 + i) * WKT + 16 * s;
            const unsigned cell = (blk * (unsigned)a.Hkv + (unsigned)g) * (unsigned)a.bs +
                                  (unsigned)(pos & (a.bs - 1));
            const int rowc = (int)(((unsigned long long)cell * C::RB) >> 7);
            if constexpr (C::KDIRECT) {
              // bf16 K needs no conversion: each 64-d block of the page tile's 16
              // rows goes to its rows of the K operand (K-major, 128-byte swizzle)
#pragma unroll
              for (int h = 0; h < D / 64; ++h)
                tma_tile_3d(k16 + (i % NB) * C::KB + h * (WKT * 128) + s * (16 * 128), &kmap, 0, h,
                            (int)cell, &raw_full[st]);
            } else {
              tma_tile_2d(base + s * C::TBP, &kmap, 0, rowc, &raw_full[st]);
            }
            tma_tile_2d(base + C::VOFF + s * C::TBP, &vmap, 0, rowc, &raw_full[st]);
            if constexpr (C::FETCH) {
              float* sc = reinterpret_cast<float*>(base + C::RAW);
              bulk_copy(sc + 16 * s, a.k_cs + cell, 64, &raw_full[st]);
              bulk_copy(sc + 16 * (SUB + s), a.v_cs + cell, 64, &raw_full[st]);
            }
          }
          __syncwarp();
        }
        last[st] = i;
      }
      // every copy issued has landed before the CTA exits (bounded waits)
      if (lane == 0)
#pragma unroll
        for (int s = 0; s < NR; ++s)
          if (last[s] >= 0) (void)mbar_wait(&raw_full[s], (uint32_t)((last[s] / NR) & 1));
    } else if (warp <= RL::MMA_PV) {
      // ---- MMA issuers: one elected lane issues and commits (elect.sync picks the
      // same lane each time: the warp is converged); the warp waits together.  S and
      // PV have a warp each: one warp for both that waited for the P' of a query
      // tile held up the other tile's next scores, and its waits and issues alone
      // took 1,900 cycles of a key tile's 2,700.  With one query tile (FEW) there is
      // nothing to hold up, and a second polling warp costs more (134 -> 143 us).
      constexpr uint32_t IDS = mma_idesc<C::BFK>(WROWS, WKT);   // bf16 Q and K for BF16 layers
      constexpr uint32_t IDO = mma_idesc<false>(WROWS, D) | MMA_B_MN_MAJOR;
      auto wait = [&](uint64_t* bar, uint32_t par) -> bool {
        const bool w = __all_sync(0xffffffffu, mbar_wait(bar, par));
        if (!w && lane == 0) { *s_abort = 1; atomicOr(a.err, ERR_TIMEOUT); }
        return w && !__any_sync(0xffffffffu, *s_abort);
      };
      // Descriptors of the operand buffers' starts; an operand at byte offset
      // o is the start's descriptor plus o / 16 (the 14-bit address field
      // cannot carry: shared memory ends below 2^18 bytes)
      const uint64_t dq = sw128_desc(q16), dk = sw128_desc(k16), dv = sw128_mn_desc(vt16, WKT * 128);
      // S_j = Q_j K^T from K buffer kbuf into S buffer sb of query tile j (Q
      // from shared memory with two query tiles, from tensor memory with one)
      auto issue_s = [&](int j, int kbuf, int sb) {
        const uint64_t qa = dq + (uint64_t)(j * (C::QB >> 4));
        const uint64_t kb = dk + (uint64_t)(kbuf * (C::KB >> 4));
        const uint32_t td = tmem + C::scol(j, sb);
        if (elect_one()) {
          tc_fence_after();
#pragma unroll
          for (int s2 = 0; s2 < D / 16; ++s2) {
            const uint64_t db = kb + (uint64_t)((((s2 >> 2) * (WKT * 128)) + (s2 & 3) * 32) >> 4);
            if constexpr (NQ == 2)
              umma(td, qa + (uint64_t)((((s2 >> 2) * (WROWS * 128)) + (s2 & 3) * 32) >> 4), db, IDS,
                   s2 > 0);
            else
              umma_tmem_a(td, tmem + C::QCOL + 8 * s2, db, IDS, s2 > 0);
          }
          umma_commit(&s_full[2 * j + sb]);
        }
        __syncwarp();
      };
      // O_j += P'_j V, every term of the split, P' from S/P' buffer sb, V from
      // buffer vbuf
      auto issue_pv = [&](int j, int vbuf, int sb, bool acc) {
        const uint64_t vb = dv + (uint64_t)(vbuf * (C::VTB >> 4));
        const uint32_t td = tmem + C::ocol(j);
        const uint32_t ta = tmem + C::scol(j, sb);
        if (elect_one()) {
          tc_fence_after();
#pragma unroll
          for (int h = 0; h < PTERMS; ++h)
#pragma unroll
            for (int kk = 0; kk < WKT / 16; ++kk)
              umma_tmem_a(td, ta + 32 * h + 8 * kk, vb + (uint64_t)(kk * (16 * 128 >> 4)), IDO,
                          acc || h > 0 || kk > 0);
          umma_commit(&pv_done[2 * j + sb]);
        }
        __syncwarp();
      };
      // S of key tile i goes into S/P' buffer i & 1 of each query tile, two tiles
      // ahead of the softmax that reads it: S_j(i) is issued once PV_j(i-2), the
      // last reader of that buffer's P', has completed, so the softmax of a query
      // tile finds its next scores ready when it finishes
      auto scores = [&](int i) -> bool {
        bool go = wait(&kv_full[i % NB], (uint32_t)((i / NB) & 1));
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
          if (!go || j >= nqt) break;
          if (i >= 2) go = wait(&pv_done[2 * j + (i & 1)], (uint32_t)(((i >> 1) - 1) & 1));
          if (go) issue_s(j, i % NB, i & 1);
        }
        return go;
      };
      auto values = [&](int i) -> bool {
        bool go = true;
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
          if (!go || j >= nqt) break;
          go = wait(&p_full[2 * j + (i & 1)], (uint32_t)((i >> 1) & 1));
          if (go) issue_pv(j, i % NB, i & 1, i > 0);
        }
        // every PV of this key tile has read its operands (and every S of it ended
        // before its softmax): buffer free
        if (go && elect_one()) umma_commit(&kv_empty[i % NB]);
        __syncwarp();
        return go;
      };
      bool go = true;
      if constexpr (FEW) {
        for (int i = 0; go && i < 2 && i < ntl; ++i) go = scores(i);
        for (int i = 0; go && i < ntl; ++i) go = values(i) && (i + 2 >= ntl || scores(i + 2));
      } else if (warp == RL::MMA_S) {
        for (int i = 0; go && i < ntl; ++i) go = scores(i);
      } else {
        for (int i = 0; go && i < ntl; ++i) go = values(i);
      }
      // everything that this warp issued completes before the epilogue and the exit
      uint64_t* fin = warp == RL::MMA_PV ? o_fin : s_fin;
      if (elect_one()) umma_commit(fin);
      __syncwarp();
      (void)mbar_wait(fin, 0u);
    }
  } else if (warp >= RL::SOFT) {
    if constexpr (RL::SPLIT_REGS) give_registers<RL::REGS_CONV>();
    // ---- converters (groups of 128 threads, taking key tiles in turn)
    const int cgrp = RL::CG == 1 ? 0 : (warp - RL::SOFT) / WS_CONV;
    const int ct_ = tid - (RL::SOFT + cgrp * WS_CONV) * 32;
    const int conv_bar = CONV_BAR + cgrp;
    for (int i = cgrp; i < ntl; i += RL::CG) {
      const int st = i % NR, buf = i % NB;
      const int t = t0 + i;
      bool ok = mbar_wait(&raw_full[st], (uint32_t)((i / NR) & 1));
      if (i >= NB) ok = mbar_wait(&kv_empty[buf], (uint32_t)((i / NB - 1) & 1)) && ok;
      if (!ok) { *s_abort = 1; atomicOr(a.err, ERR_TIMEOUT); }
      // every converter thread takes the same decision (a barrier reduction)
      if (named_sync_or(conv_bar, WS_CONV * 32, !ok || *s_abort)) break;
      const unsigned have = (unsigned)s_have[st];
      const uint8_t* base = raw + st * C::RAWS;
      uint8_t* kb = k16 + buf * C::KB;
      uint8_t* vb = vt16 + buf * C::VTB;
      // The conversions: K and V alike, 64 rows (keys) of D f16 each in 64-d blocks
      // of 128-byte rows (128-byte swizzle); K is the K-major operand of S, V the
      // MN-major one of PV, so neither is transposed.  Zeros where nothing was
      // fetched or the position lies outside [kmin, pmax].  Each thread takes NIT
      // chunks of each; all loads first, then conversions.  (KDIRECT: the producer
      // copied K there; rows of keys not fetched or outside the range hold whatever
      // was there, and the softmax masks their scores by their K scale NO_KEY.)
      // WHOLE: every key of the tile fetched and in range, without the test per key.
      auto convert = [&](auto whole_tile) {
        constexpr bool WHOLE = decltype(whole_tile)::value;
        constexpr int NIT = WKT * CPR / (WS_CONV * 32);
        static_assert(NIT * WS_CONV * 32 == WKT * CPR, "chunks per converter thread");
        // chunk it of this thread: neighbouring eight lanes take the low chunks of
        // one key and the high ones of the next, whose rows are swizzled apart, so
        // that the stores of both 64-d blocks meet each bank once
        auto key_of = [&](int it, int& ch) -> int {
          const int cc = ct_ + it * WS_CONV * 32;
          const int row = cc / CPR;
          ch = cc % CPR;
          return (CPR >= 8 && EPC == 16) ? (row & ~1) | ((row ^ (ch >> 2)) & 1) : row;
        };
        auto is_live = [&](int key) -> bool {
          const int pos = t * WKT + key;
          return WHOLE || (((have >> (key >> 4)) & 1u) && pos >= kmin && pos <= pmax);
        };
        auto load = [&](int off, int key, int ch) -> uint4 {
          return is_live(key) ? *reinterpret_cast<const uint4*>(
                                    base + off + (key >> 4) * C::TBP +
                                    swz((uint32_t)((key & 15) * C::RB + ch * 16)))
                              : make_uint4(0u, 0u, 0u, 0u);
        };
        auto store = [&](uint8_t* dst, int key, int d, uint4 v) {
          *reinterpret_cast<uint4*>(dst + (d >> 6) * (WKT * 128) + swc(key, (d & 63) >> 3)) = v;
        };
        if constexpr (MODE == BF16) {
          // V of a BF16 layer.  First the largest exponent e of each key row (two
          // threads per key, half a row each): the key's V scale is 2^(e - 14), and
          // the row times 2^(14 - e) has its largest value in [2^14, 2^15), so every
          // bf16 value down to 2^-28 of it converts to f16 exactly.
          float* vsm = reinterpret_cast<float*>(scb + buf * C::SCS) + WKT;
          {
            const int key = ct_ >> 1, hh = ct_ & 1;
            uint32_t em = 0;                          // exponent fields (<< 7) of both halves of a word
#pragma unroll
            for (int c = 0; c < CPR / 2; ++c) {
              const uint4 w = load(C::VOFF, key, hh * (CPR / 2) + c);
              em = __vmaxu2(em, w.x & 0x7F807F80u);
              em = __vmaxu2(em, w.y & 0x7F807F80u);
              em = __vmaxu2(em, w.z & 0x7F807F80u);
              em = __vmaxu2(em, w.w & 0x7F807F80u);
            }
            em = max(em & 0xFFFFu, em >> 16) >> 7;    // biased exponent, 0 for zeros
            em = max(em, __shfl_xor_sync(0xffffffffu, em, 1));
            const int e = em ? max((int)em - 127, -100) : 0;
            if (hh == 0) vsm[key] = is_live(key) ? pow2i(e - 14) : 0.f;
          }
          named_sync(conv_bar, WS_CONV * 32);         // every key's V scale is in place
#pragma unroll
          for (int it = 0; it < NIT; ++it) {
            int ch;
            const int key = key_of(it, ch);
            if constexpr (!C::KDIRECT) store(kb, key, 8 * ch, load(0, key, ch));
            // 2^(14 - e) from 2^(e - 14): exact; 2^127 for a key with no data (its values are 0)
            const float inv = __uint_as_float((254u - (__float_as_uint(vsm[key]) >> 23)) << 23);
            const uint4 w = load(C::VOFF, key, ch);
            const uint32_t w4[4] = {w.x, w.y, w.z, w.w};
            uint32_t y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              y[e] = pack_f16x2(__uint_as_float(w4[e] << 16) * inv,
                                __uint_as_float(w4[e] & 0xFFFF0000u) * inv);
            store(vb, key, 8 * ch, make_uint4(y[0], y[1], y[2], y[3]));
          }
        } else {
          uint4 wk[NIT], wv[NIT];
#pragma unroll
          for (int it = 0; it < NIT; ++it) {
            int ch;
            const int key = key_of(it, ch);
            wk[it] = load(0, key, ch);
            wv[it] = load(C::VOFF, key, ch);
          }
#pragma unroll
          for (int it = 0; it < NIT; ++it) {
            int ch;
            const int key = key_of(it, ch);
            uint4 o[4];
            convert16<MODE>(wk[it], o);
#pragma unroll
            for (int q = 0; q < EPC / 8; ++q) store(kb, key, ch * EPC + 8 * q, o[q]);
            convert16<MODE>(wv[it], o);
#pragma unroll
            for (int q = 0; q < EPC / 8; ++q) store(vb, key, ch * EPC + 8 * q, o[q]);
          }
        }
      };
      if (have == (1u << SUB) - 1u && t * WKT >= kmin && t * WKT + WKT - 1 <= pmax)
        convert(std::true_type{});
      else
        convert(std::false_type{});
      {
        // scales: threads 0..63 K, 64..127 V (no key: NO_KEY and 0)
        float* ksm = reinterpret_cast<float*>(scb + buf * C::SCS);
        float* vsm = ksm + WKT;
        int* tinfo = reinterpret_cast<int*>(vsm + WKT);
        const int isv = ct_ >= WKT;
        const int key = isv ? ct_ - WKT : ct_;
        const int sub = key >> 4;
        const int pos = t * WKT + key;
        const bool live = ((have >> sub) & 1u) && pos >= kmin && pos <= pmax;
        float sc = live ? 1.f : (isv ? 0.f : NO_KEY);
        if constexpr (C::FETCH)
          if (live) sc = reinterpret_cast<const float*>(base + C::RAW)[16 * (isv ? SUB + sub : sub) + (key & 15)];
        if constexpr (C::BFK) {
          if (isv) sc = vsm[key];                   // the BF16 V scale found above
          else ksm[key] = sc;
        } else {
          (isv ? vsm : ksm)[key] = sc;
        }
        if constexpr (C::DYN) {
          if (isv) {
            const int e = __reduce_max_sync(0xffffffffu, live ? f32_exp(sc) : -1000);
            if (lane == 0) tinfo[(ct_ - WKT) >> 5] = e;
          }
        }
        if (ct_ == 0) tinfo[2] = (have == (1u << SUB) - 1u) ? 1 : 0;
      }
      fence_proxy_async();
      named_sync(conv_bar, WS_CONV * 32);
      if (ct_ == 0) {
        mbar_arrive(&raw_empty[st]);                // the raw stage has been read
        mbar_arrive(&kv_full[buf]);
      }
    }
  } else if (warp < 4 * nqt) {
    // ---- softmax of query tile j: one thread per row (its tensor-memory lane)
    if constexpr (RL::SPLIT_REGS) take_registers<RL::REGS_SOFT>();
    const int j = warp >> 2;
    const int r = (warp & 3) * 32 + lane;
    const int R = j * WROWS + r;
    const int pA = rowp[R];
    const int loA = (a.window > 0) ? max(0, pA + 1 - a.window) : 0;
    const float fA = rowf[R];
    const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t tO = trow + C::ocol(j);
    // positions of this query tile's first and last rows: a key tile inside
    // [last row's window start, first row] is visible to every row
    const int firstj = CROSS ? pmax : first + j * QP;
    const int pmaxj = CROSS ? pmax : min(firstj + QP - 1, pmax);
    // CROSS: no row of this warp is in use; its P' may stay what it is (rows of
    // an MMA's A operand do not mix) and it only keeps the barriers' counts
    const bool idle = CROSS && __all_sync(0xffffffffu, pA < 0);
    // mU: the row's reference max (log2 units) the weights are taken against;
    // it moves only when a tile exceeds it by more than WLAZY, so O is
    // rescaled rarely and the weights stay below 2^WLAZY
    float mU = -INFINITY, l = 0.f;
    int vexp = -1000;
    float vs_static = 1.f;
    if constexpr (MODE == FP8_PER_TENSOR) vs_static = a.v_scale[0];
    if constexpr (MODE == FP8_PER_HEAD) vs_static = a.v_scale[g];
    bool ok = true;
    // Softmax of key tile t (local tile i, operand buffer buf, scores and P' at
    // tS): NCH chunks of 16 keys from chunk ch0 on.  False when a wait ran out.
    auto softmax_tile = [&](auto nch, int ch0, int i, int t, int buf, uint32_t tS) -> bool {
      constexpr int NCH = decltype(nch)::value;
      const uint32_t tP = tS;                   // P' replaces the scores it came from
      tc_fence_after();
      uint32_t s0[32], s1[32];
      if constexpr (NCH == 1) {
        tmem_ld16_nowait(tS + 16 * ch0, s0);
      } else {
        tmem_ld32_nowait(tS + 16 * ch0, s0);
        if constexpr (NCH == 4) tmem_ld32_nowait(tS + 32, s1);
      }
      tmem_wait_ld();
      const float* ksm = reinterpret_cast<const float*>(scb + buf * C::SCS);
      const float* vsm = ksm + WKT;
      const int* tinfo = reinterpret_cast<const int*>(vsm + WKT);
      const bool fast = tinfo[2] != 0 && t * WKT + WKT - 1 <= firstj &&
                        (a.window <= 0 || t * WKT >= pmaxj + 1 - a.window);
      // scores times the K scale (or -inf where masked); four running maxima.
      // The test for a wholly visible tile is taken once, outside the
      // unrolled loops, so neither loop branches per key.
      const float4* ks4 = reinterpret_cast<const float4*>(ksm) + 4 * ch0;
      uint64_t sv[8 * NCH];                     // pairs of scores
      float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      if (fast) {
        float4 kq4[4];                           // K scales of 16 keys, loaded ahead
#pragma unroll
        for (int k4 = 0; k4 < 4 * NCH; ++k4) {
          if constexpr (C::FETCH) {
            if (k4 % 4 == 0)
#pragma unroll
              for (int u = 0; u < 4; ++u) kq4[u] = lds_v4_ordered(ks4 + k4 + u);
          }
          float x[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int k = 4 * k4 + e;
            x[e] = __uint_as_float(k < 32 ? s0[k] : s1[k - 32]);
          }
          uint64_t x01 = pack_f32x2(x[0], x[1]), x23 = pack_f32x2(x[2], x[3]);
          if constexpr (C::FETCH) {              // else every scale here is 1
            const float4 kq = kq4[k4 % 4];
            x01 = mul_f32x2(x01, pack_f32x2(kq.x, kq.y));
            x23 = mul_f32x2(x23, pack_f32x2(kq.z, kq.w));
            unpack_f32x2(x01, x[0], x[1]);
            unpack_f32x2(x23, x[2], x[3]);
          }
          sv[2 * k4] = x01;
          sv[2 * k4 + 1] = x23;
#pragma unroll
          for (int e = 0; e < 4; ++e) m4[e] = fmaxf(m4[e], x[e]);
        }
      } else {
        // keys of this row: [loA, pA] relative to the tile; a key outside the
        // CTA's range or on a page not fetched has the scale NO_KEY
        const int kt0 = t * WKT + 16 * ch0;
        const int klo = loA - kt0, khi = pA < 0 ? -1 : pA - kt0;
#pragma unroll
        for (int k4 = 0; k4 < 4 * NCH; ++k4) {
          const float4 kq = ks4[k4];
          const float ksv[4] = {kq.x, kq.y, kq.z, kq.w};
          float x[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int k = 4 * k4 + e;
            const bool okk = k >= klo && k <= khi && ksv[e] != NO_KEY;
            x[e] = okk ? __uint_as_float(k < 32 ? s0[k] : s1[k - 32]) * ksv[e] : -INFINITY;
            m4[e] = fmaxf(m4[e], x[e]);
          }
          sv[2 * k4] = pack_f32x2(x[0], x[1]);
          sv[2 * k4 + 1] = pack_f32x2(x[2], x[3]);
        }
      }
      const float mrow = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * fA;
      float al = 1.f;
      if (mrow > mU + WLAZY || (mU == -INFINITY && mrow > -INFINITY)) {
        al = (mU == -INFINITY) ? 0.f : ex2(mU - mrow);
        mU = mrow;
      }
      if constexpr (C::DYN) {
        const int et = max(tinfo[0], tinfo[1]);     // the same for every row (same keys)
        const int vnew = max(vexp, max(et, -100));
        if (vnew != vexp) {
          al *= pow2i(vexp - vnew);                 // 0 on the first data (O is 0)
          vexp = vnew;
        }
      }
      // l and O both carry the range factor 2^(WKP - vexp) (64 for static
      // scales), so both follow the max and the V-scale exponent
      l *= al;
      // O holds data from the first PV on; it is rescaled (rarely) once the
      // previous PV has updated it.  P' needs no wait: its buffer held this
      // tile's S, and the PV that last read P' there completed before that S
      // was issued.
      if (i > 0 && __any_sync(0xffffffffu, al != 1.f)) {
        const bool w2 = __all_sync(0xffffffffu, mbar_wait(&pv_done[2 * j + ((i - 1) & 1)], (uint32_t)(((i - 1) >> 1) & 1)));
        if (!w2 && lane == 0) { *s_abort = 1; atomicOr(a.err, ERR_TIMEOUT); }
        if (!w2 || __any_sync(0xffffffffu, *s_abort)) return false;
        tc_fence_after();
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 32) {
          float v[32];
          tmem_ld32(tO + c0, v);
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] *= al;
          tmem_st32(tO + c0, v);
        }
      }
      // p x 2^k = 2^(score - (mU - k)): the power-of-two range factor k
      // (WKP - vexp, or 6 for static scales) enters the exponent, exactly
      const float mu = ((mU == -INFINITY) ? 0.f : mU) - (C::DYN ? (float)(WKP - vexp) : 6.f);
      const float4* vs4 = reinterpret_cast<const float4*>(vsm) + 4 * ch0;
      const uint64_t fA2 = pack_f32x2(fA, fA), mu2 = pack_f32x2(-mu, -mu);
      uint64_t lp01 = 0, lp23 = 0;              // four partial sums, as two pairs
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        uint32_t hw[8], lw[8];
        float4 vq4[4];                          // V scales of the chunk, loaded ahead
        if constexpr (C::DYN)
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4) vq4[q4] = lds_v4_ordered(vs4 + 4 * c + q4);
#pragma unroll
        for (int q4 = 0; q4 < 4; ++q4) {
          const int k = 16 * c + 4 * q4;
          float x[4];
          unpack_f32x2(fma_f32x2(sv[k / 2], fA2, mu2), x[0], x[1]);
          unpack_f32x2(fma_f32x2(sv[k / 2 + 1], fA2, mu2), x[2], x[3]);
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = ex2(x[e]);
          uint64_t x01 = pack_f32x2(x[0], x[1]), x23 = pack_f32x2(x[2], x[3]);
          lp01 = add_f32x2(lp01, x01);
          lp23 = add_f32x2(lp23, x23);
          if constexpr (C::DYN) {
            const float4 vq = vq4[q4];
            unpack_f32x2(mul_f32x2(x01, pack_f32x2(vq.x, vq.y)), x[0], x[1]);
            unpack_f32x2(mul_f32x2(x23, pack_f32x2(vq.z, vq.w)), x[2], x[3]);
          }
#pragma unroll
          for (int h2 = 0; h2 < 2; ++h2) {
            const uint32_t h = pack_f16x2(x[2 * h2], x[2 * h2 + 1]);
            hw[2 * q4 + h2] = h;
            if constexpr (PTERMS == 2)
              lw[2 * q4 + h2] = pack_f16x2(x[2 * h2] - f16_lo(h), x[2 * h2 + 1] - f16_hi(h));
          }
        }
        tmem_st8_nowait(tP + 8 * (ch0 + c), hw);
        if constexpr (PTERMS == 2) tmem_st8_nowait(tP + 32 + 8 * c, lw);
      }
      if constexpr (NCH < 4) {
        // the other copies' keys have no weight in this one
        const uint32_t zero[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
#pragma unroll
        for (int c = NCH; c < 4; ++c) tmem_st8_nowait(tP + 8 * ((ch0 + c) & 3), zero);
      }
      float lp[4];
      unpack_f32x2(lp01, lp[0], lp[1]);
      unpack_f32x2(lp23, lp[2], lp[3]);
      l += (lp[0] + lp[1]) + (lp[2] + lp[3]);
      return true;
    };
    for (int i = 0; i < ntl; ++i) {
      const int buf = i % NB, t = t0 + i;
      // S of this tile in S/P' buffer i & 1
      const int sb = i & 1;
      const uint32_t tS = trow + C::scol(j, sb);
      const bool w = __all_sync(0xffffffffu, mbar_wait(&s_full[2 * j + sb], (uint32_t)((i >> 1) & 1)));
      if (!w && lane == 0) { *s_abort = 1; atomicOr(a.err, ERR_TIMEOUT); }
      if (!w || __any_sync(0xffffffffu, *s_abort)) { ok = false; break; }
      if (idle) {
        mbar_arrive(&p_full[2 * j + sb]);
        continue;
      }
      if (!FEW || copies_shift == 0)
        ok = softmax_tile(std::integral_constant<int, 4>{}, 0, i, t, buf, tS);
      else if constexpr (FEW)
        ok = copies_shift == 1
                 ? softmax_tile(std::integral_constant<int, 2>{}, 2 * (warp >> 1), i, t, buf, tS)
                 : softmax_tile(std::integral_constant<int, 1>{}, warp, i, t, buf, tS);
      if (!ok) break;
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&p_full[2 * j + sb]);
    }
    // ---- epilogue: out = O x unscale / l (rows without a query store nothing)
    const bool fin = __all_sync(0xffffffffu, mbar_wait(o_fin, 0u));
    const bool good = ok && fin && !__any_sync(0xffffffffu, *s_abort) && !idle;
    tc_fence_after();
    // FEW: copies after the first leave their O / l and the log2 of their weights'
    // sum (as it was before the range factor) in shared memory, where every copy
    // and MMA is done
    float* xo = reinterpret_cast<float*>(smem);                // [D][128]
    float* xl = xo + D * WROWS;                                // [128]
    // O / l: the range factor cancels; static scales multiply by v_scale
    const float f = l > 0.f ? (C::DYN ? 1.f : vs_static) / l : 0.f;
    float lse = l > 0.f ? mU + log2f(l) + (C::DYN ? (float)(vexp - WKP) : -6.f) : -INFINITY;
    if constexpr (FEW) {
      if (copies_shift > 0) {
        if (good && r >= copy_rows) {
#pragma unroll 1
          for (int c0 = 0; c0 < D; c0 += 32) {
            float v[32];
            tmem_ld32(tO + c0, v);
#pragma unroll
            for (int e = 0; e < 32; ++e) xo[(c0 + e) * WROWS + r] = v[e] * f;
          }
          xl[r] = lse;
        }
        named_sync(JOIN_BAR, RL::SOFT * 32);
      }
    }
    if (good && !(FEW && r >= copy_rows)) {
      const int h = row_head(r), ii = row_query(r);
      if constexpr (CROSS) {
        const int qi = qbase + j * QP + ii;
        const long long orow = (long long)(q0 + qi) * a.Hq + g * heads + h;
        const long long prow = (((long long)split * a.B + b) * pa.max_query + qi) * a.Hq +
                               g * heads + h;
        // weight of this row's O, and of its copies'
        float w0 = f, wc[4] = {0.f, 0.f, 0.f, 0.f};
        const int copies = FEW ? 1 << copies_shift : 1;
        if (copies > 1) {
          float top = lse;
          for (int c = 1; c < copies; ++c) top = fmaxf(top, xl[r + c * copy_rows]);
          const float ref = top == -INFINITY ? 0.f : top;
          float sum = ex2(lse - ref);
          w0 = f * sum;
#pragma unroll
          for (int c = 1; c < 4; ++c)
            if (c < copies) {
              wc[c] = ex2(xl[r + c * copy_rows] - ref);
              sum += wc[c];
            }
          const float inv = sum > 0.f ? 1.f / sum : 0.f;
          w0 *= inv;
#pragma unroll
          for (int c = 1; c < 4; ++c) wc[c] *= inv;
          lse = sum > 0.f ? ref + log2f(sum) : -INFINITY;
        }
        if (!whole && pA >= 0) a.ws_ml[prow] = lse;
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 32) {
          float v[32];
          tmem_ld32(tO + c0, v);
          if (pA >= 0) {
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] *= w0;
            if constexpr (FEW) {
              for (int c = 1; c < copies; ++c)
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  v[e] = fmaf(c == 1 ? wc[1] : (c == 2 ? wc[2] : wc[3]),
                              xo[(c0 + e) * WROWS + r + c * copy_rows], v[e]);
            }
            if (whole) store_row_bf16(a.out_bf16 + orow * D + c0, v);
            else store_row_f32(a.ws_o + prow * D + c0, v);
          }
        }
      } else {
        float* dst = a.out + ((long long)(q0 + qbase + j * QP + ii) * a.Hq + g * heads + h) * D;
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 32) {
          float v[32];
          tmem_ld32(tO + c0, v);
          if (pA >= 0) {
#pragma unroll
            for (int i4 = 0; i4 < 8; ++i4)
              *reinterpret_cast<float4*>(dst + c0 + 4 * i4) =
                  make_float4(v[4 * i4] * f, v[4 * i4 + 1] * f, v[4 * i4 + 2] * f, v[4 * i4 + 3] * f);
          }
        }
      }
    }
  }

  // ---- tensor memory is freed once every role is done with it
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(C::TCOLS));
  }
}

// Once per kernel and device, before its first launch.
template <class RL, class Kernel>
cudaError_t ws_prepare(Kernel kern, int smem) {
  if (RL::SPLIT_REGS) {                        // the shares fit what a launch gets
    cudaFuncAttributes at;
    const cudaError_t e = cudaFuncGetAttributes(&at, kern);
    if (e != cudaSuccess) return e;
    if (at.numRegs < RL::REGS) return cudaErrorInvalidConfiguration;
  }
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
}

}  // namespace
}  // namespace kvq
