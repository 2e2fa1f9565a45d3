// Attention over whole prompts, before their keys and values are cached: packed
// sequences of different lengths, bf16 q, k and v as a projection leaves them
// (rows of any stride), causal, grouped heads, optionally a window.
//   out[t] = sum_j softmax_j(scale <q[t], k[j]>) v[j],  j in (t - W, t] of t's sequence.
//
// Mathematics.  One pass over the keys with the running maximum and sum of the
// softmax: weights p = 2^(s - m) against a reference m per row (log2 units) that
// moves only when a key tile exceeds it by more than 8, so that the sums O and l,
// which a move rescales, are rescaled rarely and p stays below 2^8.  Scores, m, l
// and O are fp32; p is rounded to bf16 for the product with v (both operands of an
// MMA have one type, and v is bf16), off by 2^-9 of itself on average and 2^-8 at
// most, like the output's own rounding.
//
// Structure.  Persistent CTAs, one per SM, take items: NQ query tiles of 128 rows (128 / G
// consecutive positions times the G heads of one KV head, so that a tile's rows see
// almost the same keys) against the keys up to their last position, in tiles of KT.
// The grid has a CTA for each item; those that run cancel the launch of others and
// take their items (cluster launch control), so that the hardware hands out the
// work and an item's first loads and scores run under the previous one's softmax and
// epilogue.  Items go by falling position: the ones with the most keys come first.
// Roles:
//  * producer warp: finds the items among the ragged sequences, loads Q, then K and V
//    tiles by TMA straight into their operand layouts (rows of 128 bytes, 128-byte
//    swizzle) through one ring of slots;
//  * two MMA warps, one elected lane each: one for S_j = Q_j K^T into tensor memory, one for
//    O_j += P_j V with P_j read from tensor memory, where it replaces S_j.  With two query
//    tiles PV_0, S_0, PV_1, S_1 follow one another, so that the tensor cores work on one tile
//    during the other's softmax; with one (head_dim 256, whose O takes half of
//    tensor memory) S has two buffers and runs a key tile ahead;
//  * a softmax warpgroup per query tile, one thread per row (its tensor-memory lane).
// MMAs with different accumulators may run in any order.  S_j(i + SB) overwrites the
// columns that PV_j(i) reads, so it is issued when that one has completed.  That is what
// S has a warp of its own for: one warp that waited between the two held back the other
// query tile's PV as well (16,384 tokens: 1,650 us; two warps 1,390-1,410).
//
// Nothing beyond an item's last position is multiplied: the last key tile's MMAs
// stop at the 16 keys that hold it, and the V rows between it and their end are set
// to zero, so that rows behind a sequence (of another one, or of none) may hold
// anything, NaN too.
// Every wait is bounded; one that runs out flags TIMEOUT and ends every role.
//
// What bounds it, and measured.  Long prompts: the tensor cores, which the softmax threads
// feed: 16,384 tokens, 32 heads of 128: 1,400 us, 1,570 TFLOP/s (0.84 of the cuBLAS bf16
// rate); 8 sequences of 500-4,096: 238 us, 1,320.  A key tile pair takes about 3,000
// cycles, of which the MMAs are 2,048 at their peak rate and a softmax warp's own part
// 1,230 (max 410, exponents and sums 750).  head_dim 256: 194 us, 1,360 TFLOP/s on 3
// sequences of 1,500-4,000; 64: the softmax (as many exponents for half of the flops),
// 960 TFLOP/s on 8,192 tokens, 64 heads.  Windows and short sequences: an item's chain
// of barriers and its epilogue, two or three key tiles long (window 128, 4 sequences of
// 3,000-4,096, 64 heads of 64: 121-128 us; 48 of 1-120 tokens: 19.5 us).
// Measured no faster: the maximum found beside exponents taken against the old
// reference; 64 keys a tile with four query tiles (head_dim 64: 580 -> 817 us on the
// long prompt, 120 -> 104 in the window); P in columns of its own, so that the next
// scores need not wait for PV (head_dim 64: 572 -> 618 us, 128 -> 139 in the window); whole
// rows written by the copy engine (121 -> 127 us in the window).
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "async_copy.cuh"
#include "kvq_internal.h"
#include "prompt_items.h"
#include "tcgen05.cuh"
#include "tile_math.cuh"

namespace kvq {
namespace {

constexpr int ROWS = 128;                      // rows per query tile (the MMA's M)
constexpr float LAZY = 8.f;

template <int D>
struct Shape {
  static constexpr int NQ = D == 256 ? 1 : 2;              // query tiles
  static constexpr int SB = D == 256 ? 2 : 1;              // S/P buffers per query tile
  static constexpr int KT = D == 256 ? 64 : 128;           // keys per tile
  static constexpr int NB = D / 64;                        // 64-d blocks of a row
  static constexpr int QB = ROWS * D * 2;                  // bytes of a query tile
  static constexpr int SLOT = KT * D * 2;                  // and of a K or V tile
  // With one query tile Q lives in tensor memory, the A operand of S: there its MMAs of
  // 64 keys would read more of Q from shared memory than of K, and its place there
  // holds two more tiles of K and V.  It passes through two slots of the ring.
  static constexpr bool QTM = NQ == 1;
  static constexpr int QSM = QTM ? 0 : NQ * QB;
  static constexpr int QCOL = 384;
  static_assert(!QTM || (QB == 2 * SLOT && QCOL + D / 2 <= 512), "queries in two slots");
  static constexpr int AUX = 512;                          // items and barriers
  static constexpr int SOFT = 4 * NQ;                      // softmax warps
  static constexpr int OUT = SOFT * 32 * 128;              // 64 elements of their rows on the way out
  static constexpr int LIMIT = 232448 - 1024 - AUX - OUT;  // shared memory, less alignment
  static constexpr int NS = (LIMIT - QSM) / SLOT < 8 ? (LIMIT - QSM) / SLOT : 8;
  static constexpr int SMEM = QSM + NS * SLOT + OUT + AUX + 1024;
  static constexpr int PROD = SOFT, MMA_S = SOFT + 1, MMA_PV = SOFT + 2;
  static constexpr int THREADS = (SOFT + 4) * 32;
  __host__ __device__ static constexpr int scol(int j, int b) { return NQ == 2 ? 128 * j : 256 + KT * b; }
  __host__ __device__ static constexpr int ocol(int j) { return NQ == 2 ? 256 + D * j : 0; }
  // Two query tiles: the softmax warpgroups, whose threads hold 128 scores, take
  // registers from the third one.  The shares are what the block is launched with.
  static constexpr bool MOVE_REGS = NQ == 2;
  static constexpr int REGS = 168, REGS_SOFT = 208, REGS_REST = 88;
  static_assert(!MOVE_REGS || (2 * REGS_SOFT + REGS_REST == 3 * REGS && THREADS == 384), "register shares");
  static_assert(NS >= 4, "K and V of one tile in use, of the next under way");
};

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

using Item = PromptItem;                       // what a CTA works on

// 32 sequences at a time, one for each lane; the first ones' lengths are kept.
struct WarpLanes {
  const PromptSeqs& s;
  int lane, first;

  __device__ __forceinline__ unsigned longer(int b0, int than) const {
    bool ignored = false;
    return __ballot_sync(0xffffffffu, (b0 == 0 ? first : prompt_length(s, b0 + lane, &ignored)) > than);
  }
  __device__ __forceinline__ int nth(unsigned m, int r) const {
    const bool me = ((m >> lane) & 1u) && __popc(m & ((1u << lane) - 1u)) == r;
    return __ffs(__ballot_sync(0xffffffffu, me)) - 1;
  }
};

// Asks for the launch of one more CTA to be cancelled in favour of this one: 16 bytes
// of answer, which complete on `bar`.
__device__ __forceinline__ void ask_for_item(void* answer, uint64_t* bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::
          "r"(smem_u32(answer)),
      "r"(smem_u32(bar))
      : "memory");
}

// The block index whose launch was cancelled, or -1: none was left.
__device__ __forceinline__ long long read_answer(const void* answer) {
  uint32_t ok, x;
  asm volatile(
      "{ .reg .b128 r; .reg .pred p; .reg .b32 y, z, w; ld.shared.b128 r, [%2];"
      " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r; selp.u32 %0, 1, 0, p; mov.u32 %1, 0;"
      " @p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, y, z, w}, r; }"
      : "=r"(ok), "=r"(x)
      : "r"(smem_u32(answer))
      : "memory");
  return ok ? (long long)x : -1;
}

template <int D>
__global__ void __launch_bounds__(Shape<D>::THREADS, 1)
    prompt_kernel(const PromptArgs a, const __grid_constant__ CUtensorMap qmap,
                  const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  using C = Shape<D>;
  constexpr int NQ = C::NQ, SB = C::SB, KT = C::KT, NS = C::NS;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* qsm = smem;                                     // NQ query tiles
  uint8_t* ring = smem + C::QSM;                           // NS slots
  uint8_t* outs = ring + NS * C::SLOT;                     // 4 KB per softmax warp
  uint8_t* answer = outs + C::OUT;                         // 16 bytes
  volatile Item* items = reinterpret_cast<volatile Item*>(answer + 16);   // [2]
  uint64_t* bars = reinterpret_cast<uint64_t*>(answer + 48);
  uint64_t* full = bars;                                   // [NS] producer -> MMA
  uint64_t* empty = full + NS;                             // [NS] MMA (commit) -> producer
  uint64_t* asked = empty + NS;                            // the answer is there
  uint64_t* item_full = asked + 1;                         // [2] producer -> MMA, softmax
  uint64_t* item_empty = item_full + 2;                    // [2] MMA, softmax -> producer
  uint64_t* q_full = item_empty + 2;                       // producer, or softmax (QTM) -> MMA
  uint64_t* q_empty = q_full + 1;                          // MMA (commit) -> producer
  uint64_t* s_full = q_empty + 1;                          // [NQ][SB] MMA (commit) -> softmax
  uint64_t* p_full = s_full + NQ * SB;                     // [NQ][SB] softmax -> MMA
  uint64_t* pv_done = p_full + NQ * SB;                    // [NQ][SB] MMA (commit) -> MMA of S, softmax
  uint64_t* o_full = pv_done + NQ * SB;                    // [NQ] MMA (commit), an item's last PV
  uint64_t* o_empty = o_full + NQ;                         // [NQ] softmax -> MMA
  uint64_t* fin = o_empty + NQ;                            // [2] the MMA warps' own ends
  static_assert(48 + (2 * NS + 8 + 3 * NQ * SB + 2 * NQ + 3) * 8 <= C::AUX, "barriers");
  volatile int* s_abort = reinterpret_cast<volatile int*>(fin + 2);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(fin + 2) + 1;

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int QP = ROWS >> a.g_shift;                        // positions per query tile
  const int per = NQ * QP;                                 // and per item

  const PromptSeqs seqs = {a.seq_start, a.T, a.B, a.max_len, a.Hkv, per};
  WarpLanes lanes = {seqs, lane, 0};
  int longest = 0;
  bool descends = false;                                   // starts do: sequences may overlap
  Item first = {0, -1, 0, 0};
  if (warp == C::PROD) {
    if (elect_one()) {
      prefetch_map(&qmap);
      prefetch_map(&kmap);
      prefetch_map(&vmap);
    }
    bool wrong = false;
    auto look = [&](int b) -> int {
      descends |= b < a.B && a.seq_start[b + 1] < a.seq_start[b];
      return prompt_length(seqs, b, &wrong);
    };
    longest = lanes.first = look(lane);
    for (int b0 = 32; b0 < a.B; b0 += 32) longest = max(longest, look(b0 + lane));
    descends = __any_sync(0xffffffffu, descends);
    // every CTA that starts tells: which ones do is not known
    if (wrong) atomicOr(a.err, ERR_BAD_INDEX);
    longest = __reduce_max_sync(0xffffffffu, longest);
  }
  PromptSearch<WarpLanes> items_of_call(seqs, lanes, longest);   // the producer's
  if (warp == C::PROD) {
    first = items_of_call.find(blockIdx.x);
    if (lane == 0) *s_abort = first.p0 < 0;
  }
  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(asked, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&item_full[s], 1);
      mbar_init(&item_empty[s], C::SOFT + 2);
    }
    mbar_init(q_full, C::QTM ? 128 : 1);
    mbar_init(q_empty, 1);
    for (int s = 0; s < NQ * SB; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&p_full[s], 128);
      mbar_init(&pv_done[s], 1);
    }
    for (int j = 0; j < NQ; ++j) {
      mbar_init(&o_full[j], 1);
      mbar_init(&o_empty[j], 4);
    }
    mbar_init(&fin[0], 1);
    mbar_init(&fin[1], 1);
    mbar_init_fence();
  }
  __syncthreads();
  if (*s_abort) return;                                    // no item here: the whole CTA
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(s_tmem)),
                 "r"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;

  // A wait of a whole warp; false when it ran out here or anywhere.
  auto wait = [&](uint64_t* bar, uint32_t par) -> bool {
    const bool ok = __all_sync(0xffffffffu, mbar_wait(bar, par));
    if (!ok && lane == 0) { *s_abort = 1; atomicOr(a.err, ERR_TIMEOUT); }
    return ok && !__any_sync(0xffffffffu, *s_abort);
  };
  // Item k of this CTA, for the MMA and softmax warps; false when there is none.
  auto take_item = [&](int k, Item& it) -> bool {
    if (!wait(&item_full[k & 1], (uint32_t)((k >> 1) & 1))) return false;
    // through shuffles: the compiler then knows what follows from an item to be
    // warp-uniform, as a role's loops and descriptors are
    volatile Item* i = items + (k & 1);
    it.t0 = __shfl_sync(0xffffffffu, i->t0, 0);
    it.p0 = __shfl_sync(0xffffffffu, i->p0, 0);
    it.end = __shfl_sync(0xffffffffu, i->end, 0);
    it.g = __shfl_sync(0xffffffffu, i->g, 0);
    __syncwarp();
    if (lane == 0) mbar_arrive(&item_empty[k & 1]);
    return it.p0 >= 0;
  };
  // Key tiles of an item: from first_tile on, tiles_of(j) for query tile j.
  auto first_tile = [&](const Item& it) { return a.window > 0 ? max(0, it.p0 + 1 - a.window) / KT : 0; };
  auto query_tiles = [&](const Item& it) { return it.end - it.p0 <= QP ? 1 : NQ; };
  auto tile_end = [&](const Item& it, int j) { return min(it.end, it.p0 + (j + 1) * QP); };
  auto tiles_of = [&](const Item& it, int j) { return (tile_end(it, j) + KT - 1) / KT - first_tile(it); };

  // ================================================================ roles
  if (warp >= C::SOFT) {
    if constexpr (C::MOVE_REGS) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_REST));
    if (warp == C::PROD) {
      // ---- producer: the ring's order is K(0 .. SB-1), then V(i), K(i + SB)
      int issued = 0, k = 0;
      Item it = first;
      auto load = [&](const CUtensorMap* map, int key) -> bool {
        const int slot = issued % NS;
        if (issued >= NS && !wait(&empty[slot], (uint32_t)((issued / NS - 1) & 1))) return false;
        if (elect_one()) {
          mbar_expect_tx(&full[slot], C::SLOT);
#pragma unroll
          for (int c = 0; c < C::NB; ++c)
            tma_tile_3d(ring + slot * C::SLOT + c * (KT * 128), map, 128 * c, it.g, it.t0 + key, &full[slot]);
        }
        __syncwarp();
        ++issued;
        return true;
      };
      auto publish = [&]() -> bool {
        if (k >= 2 && !wait(&item_empty[k & 1], (uint32_t)(((k >> 1) - 1) & 1))) return false;
        if (lane == 0) {
          volatile Item* i = items + (k & 1);
          i->t0 = it.t0;
          i->p0 = it.p0;
          i->end = it.end;
          i->g = it.g;
          mbar_arrive(&item_full[k & 1]);
        }
        __syncwarp();
        return true;
      };
      int loaded = 0;                                      // items whose Q was loaded
      int asks = 0;                                        // answers waited for
      long long w = blockIdx.x;                            // the item's number
      for (bool go = publish(); go && it.p0 >= 0; go = publish()) {
        const int nqt = query_tiles(it), kt0 = first_tile(it), ntl = tiles_of(it, nqt - 1);
        if constexpr (C::QTM) {
          for (int half = 0; go && half < 2; ++half) {
            const int slot = issued % NS;
            if (issued >= NS) go = wait(&empty[slot], (uint32_t)((issued / NS - 1) & 1));
            if (!go) break;
            if (elect_one()) {
              mbar_expect_tx(&full[slot], C::SLOT);
#pragma unroll
              for (int c = 0; c < C::NB / 2; ++c)
                tma_tile_3d(ring + slot * C::SLOT + c * (ROWS * 128), &qmap, 128 * (half * (C::NB / 2) + c),
                            it.g << a.g_shift, it.t0 + it.p0, &full[slot]);
            }
            __syncwarp();
            ++issued;
          }
        }
        for (int i = 0; go && i < SB && i < ntl; ++i) go = load(&kmap, (kt0 + i) * KT);
        if constexpr (!C::QTM) {
          if (go && k >= 1) go = wait(q_empty, (uint32_t)((k - 1) & 1));
          if (!go) break;
          if (elect_one()) {
            mbar_expect_tx(q_full, nqt * C::QB);
            for (int j = 0; j < nqt; ++j)
#pragma unroll
              for (int c = 0; c < C::NB; ++c)
                tma_tile_3d(qsm + j * C::QB + c * (ROWS * 128), &qmap, 128 * c, it.g << a.g_shift,
                            it.t0 + it.p0 + j * QP, q_full);
          }
          __syncwarp();
          ++loaded;
        }
        // Sequences that overlap can have more items than the grid has CTAs; number w then
        // goes on as w + grid
        Item behind = {0, -1, 0, 0};
        bool waiting = false;                              // for an answer
        for (int i = 0; go && i < ntl; ++i) {
          if (i == max(0, ntl - 2)) {                      // the next item, no earlier than needed
            if (descends) behind = items_of_call.find(w + gridDim.x);
            if (behind.p0 < 0) {
              if (elect_one()) {
                mbar_expect_tx(asked, 16);
                ask_for_item(answer, asked);
              }
              waiting = true;
            }
          }
          __syncwarp();
          go = load(&vmap, (kt0 + i) * KT);
          if (go && i + SB < ntl) go = load(&kmap, (kt0 + i + SB) * KT);
        }
        // the answer arrives in any case (and has to, before the CTA exits)
        if (waiting && !wait(asked, (uint32_t)(asks++ & 1))) break;
        if (!go) break;
        if (waiting) {
          w = read_answer(answer);
          fence_proxy_async();                             // read before it is written again
          __syncwarp();
          it.p0 = -1;
          if (w >= 0) it = items_of_call.find(w);
        } else {
          it = behind;
          w += gridDim.x;
        }
        ++k;
      }
      // every copy has landed before the CTA exits
      if (loaded > 0) (void)mbar_wait(q_full, (uint32_t)((loaded - 1) & 1));
      for (int x = max(0, issued - NS); x < issued; ++x)
        (void)mbar_wait(&full[x % NS], (uint32_t)((x / NS) & 1));
    } else if (warp == C::MMA_S || warp == C::MMA_PV) {
      // ---- MMA issuers: one for S, one for O
      const bool scores = warp == C::MMA_S;
      const uint64_t dq = sw128_desc(qsm), dk = sw128_desc(ring), dv = sw128_mn_desc(ring, KT * 128);
      int x = 0;                                           // the item's first entry in the ring
      int used[NQ], items_of[NQ];                          // query tile j's key tiles and items so far
#pragma unroll
      for (int j = 0; j < NQ; ++j) used[j] = items_of[j] = 0;
      auto take = [&](int entry) -> bool { return wait(&full[entry % NS], (uint32_t)((entry / NS) & 1)); };
      auto commit = [&](uint64_t* bar) {
        if (elect_one()) umma_commit(bar);
        __syncwarp();
      };
      Item it;
      bool go = true;
      for (int k = 0; go && take_item(k, it); ++k) {
        const int nqt = query_tiles(it), kt0 = first_tile(it), ntl = tiles_of(it, nqt - 1);
        // key tiles of query tile j, and the keys of its last one, a multiple of 16
        int nt[NQ], rest[NQ];
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
          nt[j] = j < nqt ? tiles_of(it, j) : 0;
          rest[j] = min(KT, (tile_end(it, j) - (kt0 + nt[j] - 1) * KT + 15) & ~15);
        }
        if (scores) {
          go = wait(q_full, (uint32_t)(k & 1));
          if constexpr (C::QTM) {                          // its slots have been read
            if (lane == 0) {
              mbar_arrive(&empty[x % NS]);
              mbar_arrive(&empty[(x + 1) % NS]);
            }
            __syncwarp();
            x += 2;
          }
          for (int i = 0; go && i < ntl; ++i) {
            const int entry = x + (i < SB ? i : 2 * i + 1 - SB), slot = entry % NS;
            go = take(entry);
#pragma unroll
            for (int j = 0; j < NQ; ++j) {
              if (!go || i >= nt[j]) continue;
              const int u = used[j] + i, sb = u % SB;
              // the PV whose P it replaces, perhaps of the item before, has read it
              if (u >= SB) go = wait(&pv_done[j * SB + sb], (uint32_t)((u / SB - 1) & 1));
              if (!go) continue;
              const uint64_t qa = dq + (uint64_t)(j * (C::QB >> 4));
              const uint64_t kb = dk + (uint64_t)(slot * (C::SLOT >> 4));
              const uint32_t td = tmem + C::scol(j, sb);
              const uint32_t id = mma_idesc<true>(ROWS, i == nt[j] - 1 ? rest[j] : KT);
              if (elect_one()) {
                tc_fence_after();
#pragma unroll
                for (int s = 0; s < D / 16; ++s) {
                  const uint64_t b = kb + (uint64_t)((((s >> 2) * (KT * 128)) + (s & 3) * 32) >> 4);
                  if constexpr (C::QTM) umma_tmem_a(td, tmem + C::QCOL + 8 * s, b, id, s > 0);
                  else umma(td, qa + (uint64_t)((((s >> 2) * (ROWS * 128)) + (s & 3) * 32) >> 4), b, id, s > 0);
                }
                umma_commit(&s_full[j * SB + sb]);
              }
              __syncwarp();
            }
            if (go) commit(&empty[slot]);
          }
          if constexpr (!C::QTM) {
            if (go) commit(q_empty);                       // behind the item's last scores
          }
        } else {
          if constexpr (C::QTM) x += 2;
          for (int i = 0; go && i < ntl; ++i) {
            const int entry = x + min(SB, ntl) + i + min(i, max(ntl - SB, 0)), slot = entry % NS;
            go = take(entry);
            if (!go) break;
            if (i == ntl - 1) {
              // rows between the item's last position and the end of its 16 keys
              const int from = it.end - (kt0 + i) * KT, to = (from + 15) & ~15;
              uint8_t* v = ring + slot * C::SLOT;
              for (int e = lane; e < (to - from) * (D / 8); e += 32) {
                const int row = from + e / (D / 8), c = e % (D / 8);
                *reinterpret_cast<uint4*>(v + (c >> 3) * (KT * 128) + row * 128 + ((c & 7) << 4)) =
                    make_uint4(0u, 0u, 0u, 0u);
              }
              fence_proxy_async();
              __syncwarp();
            }
#pragma unroll
            for (int j = 0; j < NQ; ++j) {
              if (!go || i >= nt[j]) continue;
              const int u = used[j] + i, sb = u % SB;
              // O_j of the item before has been read
              if (i == 0 && items_of[j] > 0) go = wait(&o_empty[j], (uint32_t)((items_of[j] - 1) & 1));
              if (go) go = wait(&p_full[j * SB + sb], (uint32_t)((u / SB) & 1));
              if (!go) continue;
              const uint64_t vb = dv + (uint64_t)(slot * (C::SLOT >> 4));
              const uint32_t td = tmem + C::ocol(j), ta = tmem + C::scol(j, sb);
              const bool last = i == nt[j] - 1;
              constexpr uint32_t id = mma_idesc<true>(ROWS, D) | MMA_B_MN_MAJOR;
              if (elect_one()) {
                tc_fence_after();
                if (last) {
                  for (int s = 0; s < rest[j] / 16; ++s)
                    umma_tmem_a(td, ta + 8 * s, vb + (uint64_t)(s * (16 * 128 >> 4)), id, i > 0 || s > 0);
                } else {
#pragma unroll
                  for (int s = 0; s < KT / 16; ++s)
                    umma_tmem_a(td, ta + 8 * s, vb + (uint64_t)(s * (16 * 128 >> 4)), id, i > 0 || s > 0);
                }
                umma_commit(&pv_done[j * SB + sb]);
                if (last) umma_commit(&o_full[j]);
              }
              __syncwarp();
            }
            if (go) commit(&empty[slot]);
          }
        }
        x += 2 * ntl;
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
          used[j] += nt[j];
          items_of[j] += j < nqt;
        }
      }
      // what was issued completes before the CTA exits
      commit(&fin[scores]);
      (void)mbar_wait(&fin[scores], 0u);
    }
  } else {
    if constexpr (C::MOVE_REGS) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REGS_SOFT));
    // ---- softmax of query tile j
    const int j = warp >> 2;
    const int r = (warp & 3) * 32 + lane;
    const int off = j * QP + (r >> a.g_shift);             // this row's position within the item
    const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t tO = trow + C::ocol(j);
    const float c = a.qk_scale;
    int used = 0, items_done = 0;
    bool ok = true;
    // QTM: this thread's row of Q, from the ring's entry `at` and the next into tensor
    // memory (the scores before, which read the one that was there, are complete)
    int at = 0;
    auto copy_queries = [&]() -> bool {
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        const int slot = (at + half) % NS;
        if (!wait(&full[slot], (uint32_t)(((at + half) / NS) & 1))) return false;
#pragma unroll 1
        for (int b = 0; b < C::NB / 2; ++b) {
          const uint8_t* block = ring + slot * C::SLOT + b * (ROWS * 128);
          const uint32_t to = trow + C::QCOL + (half * (C::NB / 2) + b) * 32;
#pragma unroll
          for (int e = 0; e < 8; e += 4) {
            uint32_t w[16];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const uint4 v = *reinterpret_cast<const uint4*>(block + swc(r, e + y));
              w[4 * y] = v.x; w[4 * y + 1] = v.y; w[4 * y + 2] = v.z; w[4 * y + 3] = v.w;
            }
            tmem_st16_nowait(to + 4 * e, w);
          }
        }
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(q_full);
      return true;
    };
    Item it, next;
    bool more = false;
    if constexpr (C::QTM) {
      more = take_item(0, it);
      if (more) ok = copy_queries();
    }
    for (int k = 0; ok; ++k) {
      if constexpr (C::QTM) {
        if (!more) break;
      } else {
        if (!take_item(k, it)) break;
        if (j >= query_tiles(it)) continue;
      }
      const int kt0 = first_tile(it), nt = tiles_of(it, j);
      const int pos = it.p0 + off;
      const int lo = a.window > 0 ? max(0, pos + 1 - a.window) : 0;
      const int jfirst = it.p0 + j * QP, jlast = tile_end(it, j) - 1;
      // no row of this warp is in use: its P may stay what it is (rows of an MMA's A
      // operand do not mix), and it only keeps the barriers' counts
      const bool idle = __all_sync(0xffffffffu, pos >= it.end);
      float m = -INFINITY, l = 0.f;
      for (int i = 0; i < nt; ++i) {
        const int u = used + i, sb = j * SB + u % SB;
        const uint32_t tS = trow + C::scol(j, u % SB);
        ok = wait(&s_full[sb], (uint32_t)((u / SB) & 1));
        if (!ok) break;
        if (idle) {
          mbar_arrive(&p_full[sb]);
          continue;
        }
        tc_fence_after();
        uint32_t s[KT / 32][32];
#pragma unroll
        for (int q = 0; q < KT / 32; ++q) tmem_ld32_nowait(tS + 32 * q, s[q]);
        tmem_wait_ld();
        const int k0 = (kt0 + i) * KT;
        // a tile that some row does not see whole
        if (k0 + KT - 1 > jfirst || (a.window > 0 && k0 < jlast + 1 - a.window)) {
#pragma unroll
          for (int q = 0; q < KT / 32; ++q) {
            // a bit for each of 32 keys: a test per bit instead of two comparisons
            const int klo = max(lo - k0 - 32 * q, 0), khi = min(pos - k0 - 32 * q, 31);
            const uint32_t seen = klo > khi ? 0u : (0xffffffffu >> (31 - khi)) & (0xffffffffu << klo);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!((seen >> e) & 1u)) s[q][e] = 0xFF800000u;   // -inf
          }
        }
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int q = 0; q < KT / 32; ++q)
#pragma unroll
          for (int e = 0; e < 32; e += 8)
#pragma unroll
            for (int v = 0; v < 4; ++v)
              m4[v] = max3(m4[v], __uint_as_float(s[q][e + 2 * v]), __uint_as_float(s[q][e + 2 * v + 1]));
        const float top = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * c;
        float al = 1.f;
        if (top > m + LAZY || (m == -INFINITY && top > -INFINITY)) {
          al = m == -INFINITY ? 0.f : ex2(m - top);
          m = top;
        }
        l *= al;
        if (i > 0 && __any_sync(0xffffffffu, al != 1.f)) {
          // with one S buffer S(i) was issued when PV(i - 1) was done
          if constexpr (SB > 1) {
            ok = wait(&pv_done[j * SB + (u - 1) % SB], (uint32_t)(((u - 1) / SB) & 1));
            if (!ok) break;
            tc_fence_after();
          }
#pragma unroll 1
          for (int d = 0; d < D; d += 32) {
            float v[32];
            tmem_ld32(tO + d, v);
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] *= al;
            tmem_st32(tO + d, v);
          }
        }
        const float ref = m == -INFINITY ? 0.f : m;
        const uint64_t c2 = pack_f32x2(c, c), r2 = pack_f32x2(-ref, -ref);
        uint64_t l01 = 0, l23 = 0;
#pragma unroll
        for (int q = 0; q < KT / 32; ++q) {
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            float y[4];
            unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(s[q][e]), __uint_as_float(s[q][e + 1])), c2, r2),
                         y[0], y[1]);
            unpack_f32x2(
                fma_f32x2(pack_f32x2(__uint_as_float(s[q][e + 2]), __uint_as_float(s[q][e + 3])), c2, r2), y[2],
                y[3]);
#pragma unroll
            for (int v = 0; v < 4; ++v) y[v] = ex2(y[v]);
            l01 = add_f32x2(l01, pack_f32x2(y[0], y[1]));
            l23 = add_f32x2(l23, pack_f32x2(y[2], y[3]));
            w[e / 2] = pack_bf16x2(y[0], y[1]);
            w[e / 2 + 1] = pack_bf16x2(y[2], y[3]);
          }
          tmem_st16_nowait(tS + 16 * q, w);
        }
        float y[4];
        unpack_f32x2(l01, y[0], y[1]);
        unpack_f32x2(l23, y[2], y[3]);
        l += (y[0] + y[1]) + (y[2] + y[3]);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&p_full[sb]);
      }
      used += nt;
      if constexpr (C::QTM) {                              // the next item's queries, meanwhile
        at += 2 + 2 * nt;
        if (ok) more = take_item(k + 1, next);
        if (ok && more) ok = copy_queries();
      }
      // ---- epilogue: O / l
      if (ok) ok = wait(&o_full[j], (uint32_t)(items_done & 1));
      if (!ok) break;
      ++items_done;
      tc_fence_after();
      const float f = l > 0.f ? 1.f / l : 0.f;
      // The rows go out through shared memory, 64 elements at a time, so that eight
      // lanes write 128 bytes of one row (a lane's own row is a line of its own for each
      // lane: 32 lines a store, four to eight times the time)
      uint8_t* mine = outs + warp * (32 * 128);
#pragma unroll 1
      for (int d = 0; d < D; d += 64) {
        if (!idle) {
          uint32_t v[2][32];
          tmem_ld32_nowait(tO + d, v[0]);
          tmem_ld32_nowait(tO + d + 32, v[1]);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t* x = v[e >> 2] + 8 * (e & 3);
            uint32_t w[4];
#pragma unroll
            for (int y = 0; y < 4; ++y)
              w[y] = pack_bf16x2(__uint_as_float(x[2 * y]) * f, __uint_as_float(x[2 * y + 1]) * f);
            *reinterpret_cast<uint4*>(mine + swc(lane, e)) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
        if (d + 64 == D) tc_fence_before();
        __syncwarp();
        if (d + 64 == D && lane == 0) mbar_arrive(&o_empty[j]);
        if (idle) continue;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int row = 4 * e + (lane >> 3), R = (warp & 3) * 32 + row;
          const int p = it.p0 + j * QP + (R >> a.g_shift);
          const int h = (it.g << a.g_shift) + (R & ((1 << a.g_shift) - 1));
          if (p < it.end)
            *reinterpret_cast<uint4*>(a.out + ((long long)(it.t0 + p) * a.Hq + h) * D + d + 8 * (lane & 7)) =
                *reinterpret_cast<const uint4*>(mine + swc(row, lane & 7));
        }
        __syncwarp();
      }
      if constexpr (C::QTM) it = next;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
  }
}

}  // namespace

// Sequences of n tokens have ceil(n / per) items each: at most this many in T tokens.
long long prompt_items(int D, int G, long long T, long long max_len, long long B, int Hkv) {
  const long long per = (D == 256 ? 1 : 2) * (ROWS / G);
  const long long packed = (T + B * (per - 1)) / per, each = (max_len + per - 1) / per;
  return (packed / B < each ? packed : each * B) * Hkv;
}

namespace {

template <int D>
cudaError_t plaunch(PromptArgs a, long long q_stride, const void* k, const void* v, long long kv_stride,
                    cudaStream_t st) {
  using C = Shape<D>;
  const int G = 1 << a.g_shift;
  CUtensorMap qm, km, vm;
  if (!make_rows_map(&qm, a.q, D, a.Hq, a.T, q_stride, G, ROWS / G) ||
      !make_rows_map(&km, k, D, a.Hkv, a.T, kv_stride, 1, C::KT) ||
      !make_rows_map(&vm, v, D, a.Hkv, a.T, kv_stride, 1, C::KT))
    return cudaErrorInvalidValue;
  static bool attr_set[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  auto kern = prompt_kernel<D>;
  if (!attr_set[dev]) {
    if (C::MOVE_REGS) {                        // the shares fit what a launch gets
      cudaFuncAttributes at;
      const cudaError_t e = cudaFuncGetAttributes(&at, kern);
      if (e != cudaSuccess) return e;
      if (at.numRegs < C::REGS) return cudaErrorInvalidConfiguration;
    }
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  kern<<<(unsigned)prompt_items(D, G, a.T, a.max_len, a.B, a.Hkv), C::THREADS, C::SMEM, st>>>(a, qm, km, vm);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prompt(int D, const PromptArgs& a, long long q_stride, const void* k, const void* v,
                          long long kv_stride, cudaStream_t st) {
  switch (D) {
    case 64: return plaunch<64>(a, q_stride, k, v, kv_stride, st);
    case 128: return plaunch<128>(a, q_stride, k, v, kv_stride, st);
    case 256: return plaunch<256>(a, q_stride, k, v, kv_stride, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace kvq
