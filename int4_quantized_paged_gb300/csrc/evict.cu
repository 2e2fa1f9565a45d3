// Eviction from the cache by accumulated attention weight: of the L cells of a row
// and KV head the first f and the last l stay, and between them the k - f - l that
// gathered the most weight (of equal ones the lowest); the others give their places
// to the cells that stay behind the new end, so that the row is its first k cells.
//
// Mathematics.  Attention does not ask in which order its cells stand, so only what
// stays behind the new end moves: the i-th survivor there goes to the i-th place
// that an evicted cell leaves, both in ascending order, and the last l cells keep
// their order at the new end (they are the newest ones, which the next eviction has
// to find there).  A step's eviction of a few cells thus moves a few, not the row.
// The survivors are those above the (k - f - l)-th largest weight, found by radix
// selection: four passes over 8 bits of the weights' bits in sortable order.
//
// Structure.  A cluster of CTAs per (row, KV head), each with a segment of the row's
// cells; their weights are read once, into shared memory.  Counts meet through
// distributed shared memory: histograms of the passes, then prefix counts of ties,
// free places and survivors.  The i-th place and the i-th survivor are written into
// lists that are spread over the cluster (where the weights were), so that every CTA
// moves an equal share.  Nothing depends on the order of atomics but sums of
// integers.
//
// What bounds it.  The bytes (weights once, moved cells twice) take a few us; the rest
// is the chain of barriers between the steps and the first fetch of each step's
// instructions: 64 rows of 1,900-2,176 cells, 8 KV heads, cut to 2,048: 21 us (bytes:
// 3.4); 4 rows of 20,000-36,000 cut to 4,096: 32 us (9.8), of which the moves are 8.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kvq_internal.h"

namespace kvq {
namespace {

namespace cg = cooperative_groups;

constexpr int ET = 256;                        // threads per CTA, one per bin
constexpr int EW = ET / 32;
constexpr int BINS = 256;
static_assert(BINS == ET, "a thread per bin");
constexpr int MAX_CLUSTER = 8;
constexpr int MAX_SEGMENT = 48 * 1024;         // cells of a CTA (their weights: 192 KB)
static_assert(MAX_SEGMENT < 65536, "two counts of cells in 32 bits");
constexpr int MOVE_U = 8;                      // 16-byte chunks in flight per thread

// The weight's bits in an order that unsigned integers have; NaN lowest, -0 as 0.
__device__ __forceinline__ uint32_t sortable(float w) {
  if (w != w) return 0u;
  const uint32_t b = __float_as_uint(w + 0.f);
  return (b >> 31) ? ~b : b | 0x80000000u;
}

// Exclusive prefix of v over the CTA's threads, and the total.  s_warp: EW ints.
__device__ __forceinline__ int block_prefix(int v, int* s_warp, int* total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < EW; ++w) {
    const int x = s_warp[w];
    if (w < warp) before += x;
    all += x;
  }
  __syncthreads();                             // s_warp may be written again
  *total = all;
  return before + incl - v;
}

// Bits of the word of cells [p, p + 32) that lie in [lo, hi).
__device__ __forceinline__ uint32_t range_bits(int p, int lo, int hi) {
  const int a = max(lo - p, 0), b = min(hi - p, 32);
  if (a >= b) return 0u;
  return (b == 32 ? 0xffffffffu : (1u << b) - 1u) & ~((1u << a) - 1u);
}

__global__ void __launch_bounds__(ET, 3) evict_kernel(const EvictArgs a) {
  cg::cluster_group cl = cg::this_cluster();
  const int cs = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int item = blockIdx.x / cs;
  const int i = item / a.Hkv, g = item - i * a.Hkv;
  const PageTables& t = a.t;

  extern __shared__ uint32_t dyn[];
  uint32_t* keys = dyn;                        // [seg]; later the lists of moves
  uint32_t* s_gt = dyn + a.seg_max;            // [seg / 32] above the threshold, then: stays
  uint32_t* s_eq = s_gt + a.seg_max / 32;      // [seg / 32] at the threshold, then: counts before
  __shared__ int hist[BINS];                   // this CTA's, of one pass
  __shared__ int sums[4][BINS];                // the cluster's, a row per pass
  __shared__ int s_warp[EW];
  __shared__ int s_bad, s_count[3];            // what the other CTAs read: ties, places, survivors

  // A CTA by itself needs no barrier of a cluster, which takes ten times as long.
  auto sync_all = [&] {
    if (cs > 1) cl.sync();
    else __syncthreads();
  };

  // ---- the row (every CTA of its heads comes to the same result)
  const int row = a.rows[i], keep = a.keep_lens[i];
  bool seen = false;
  for (int j = tid; j < i; j += ET) seen |= a.rows[j] == row;
  seen = __syncthreads_or(seen);
  const bool bad_row = seen || row < 0 || row >= t.rows;
  const int L = bad_row ? 0 : t.lens[row];
  const bool bad_len = bad_row || L < 0 || L > a.max_len ||
                       (long long)L > ((long long)t.max_blocks << t.bs_shift) ||
                       (long long)keep < (long long)a.first + a.last;
  const bool teller = g == 0 && rank == 0 && tid == 0;
  if (bad_len || L <= keep) {                  // the same for the whole cluster
    if (teller) a.new_lens[i] = L;
    if (bad_len && tid == 0) atomicOr(t.err, ERR_BAD_INDEX);
    return;
  }
  const int* table = t.table + (long long)row * t.max_blocks;
  float* weights = a.weights + ((long long)row * a.Hkv + g) * a.stride;
  const int seg = ((L + cs - 1) / cs + 31) & ~31;
  const int base = rank * seg, nw = seg / 32;
  // cells to choose from, and their part of this segment
  const int lo = a.first, hi = L - a.last, edge = keep - a.last;
  const int c0 = min(max(lo - base, 0), seg), c1 = min(max(hi - base, 0), seg);
  const int wanted = keep - a.first - a.last;

  // The sum of one int over the cluster's CTAs, and over those before this one.  All
  // loads are under way at once: a remote one takes about as long as one to L2.
  auto sum_of = [&](int* mine, int* before) -> int {
    int v[MAX_CLUSTER], all = 0, low = 0;
#pragma unroll
    for (int r = 0; r < MAX_CLUSTER; ++r) v[r] = r < cs ? *cl.map_shared_rank(mine, r) : 0;
#pragma unroll
    for (int r = 0; r < MAX_CLUSTER; ++r) {
      all += v[r];
      low += r < rank ? v[r] : 0;
    }
    if (before) *before = low;
    return all;
  };

  // ---- every block of the row names one of the pool that no other row holds
  if (tid == 0) s_bad = 0;
  hist[tid] = 0;
#pragma unroll
  for (int p = 0; p < 4; ++p) sums[p][tid] = 0;
  __syncthreads();
  const int blocks = (int)(((long long)L + (1 << t.bs_shift) - 1) >> t.bs_shift);
  for (int j = rank * ET + tid; j < blocks; j += cs * ET) {
    const int b = table[j];
    if (b < 0 || b >= t.num_blocks || (t.ref && t.ref[b] != 1)) s_bad = 1;
  }
  for (int p = c0 + tid; p < c1; p += ET) keys[p] = sortable(weights[base + p]);
  __syncthreads();

  // ---- the wanted-th largest weight, eight bits a pass
  uint32_t prefix = 0;
  int rest = wanted, ties = 0;
  sync_all();                                  // every CTA's sums stand at 0
  if (sum_of(&s_bad, nullptr) > 0) {           // the same for the whole cluster
    if (teller) {
      a.new_lens[i] = L;
      atomicOr(t.err, ERR_BAD_INDEX);
    }
    sync_all();                                // no CTA leaves while another reads its flag
    return;
  }
#pragma unroll 1
  for (int pass = 0; pass < 4; ++pass) {
    const int shift = 24 - 8 * pass;
    for (int p = c0 + tid; p < c1; p += ET) {
      const uint32_t key = keys[p];
      // 64 bits: a shift by 32 in the first pass
      if (((uint64_t)(key ^ prefix) >> (shift + 8)) == 0) atomicAdd(&hist[(key >> shift) & 255], 1);
    }
    __syncthreads();
    // Bins that are not empty go to every CTA's sums (few are: weights of a row lie
    // within some powers of two; reading all of eight histograms took twice as long)
    const int mine = hist[tid];
    hist[tid] = 0;
    if (mine > 0)
      for (int r = 0; r < cs; ++r) atomicAdd(cl.map_shared_rank(&sums[pass][tid], r), mine);
    sync_all();
    // Each warp finds the bin by itself, eight bins a lane, the highest first.
    int bin[8], n = 0;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      bin[u] = sums[pass][BINS - 1 - 8 * lane - u];
      n += bin[u];
    }
    int incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    int above = incl - n, found = 0, left = 0, there = 0;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (above < rest && rest <= above + bin[u]) {
        found = BINS - 1 - 8 * lane - u;
        left = rest - above;
        there = bin[u];
      }
      above += bin[u];
    }
    if (wanted > 0) {                          // one lane found it
      const int src = __ffs(__ballot_sync(0xffffffffu, there > 0)) - 1;
      prefix |= (uint32_t)__shfl_sync(0xffffffffu, found, src) << shift;
      rest = __shfl_sync(0xffffffffu, left, src);
      ties = __shfl_sync(0xffffffffu, there, src);
    }
  }

  // ---- which cells stay
  for (int w = warp; w < nw; w += EW) {
    const int p = 32 * w + lane;
    const bool in = wanted > 0 && p >= c0 && p < c1;
    const uint32_t key = in ? keys[p] : 0u;
    const unsigned gt = __ballot_sync(0xffffffffu, in && key > prefix);
    const unsigned eq = __ballot_sync(0xffffffffu, in && key == prefix);
    if (lane == 0) { s_gt[w] = gt; s_eq[w] = eq; }
  }
  __syncthreads();
  // ties: the lowest `rest` of them
  if (rest < ties) {                           // the same for the whole cluster
    int n = 0, all, at;
    for (int w = tid; w < nw; w += ET) n += __popc(s_eq[w]);
    (void)block_prefix(n, s_warp, &all);
    if (tid == 0) s_count[0] = all;
    sync_all();
    (void)sum_of(&s_count[0], &at);
    for (int w0 = 0; w0 < nw; w0 += ET) {
      const int w = w0 + tid;
      const uint32_t eq = w < nw ? s_eq[w] : 0u;
      int here;
      int left = rest - (at + block_prefix(__popc(eq), s_warp, &here));
      uint32_t take = 0, bits = eq;
      for (; bits && left > 0; --left) {
        take |= bits & -bits;
        bits &= bits - 1;
      }
      if (w < nw) s_eq[w] = take;
      at += here;
    }
    __syncthreads();
  }
  for (int w = tid; w < nw; w += ET) s_gt[w] |= s_eq[w];
  __syncthreads();
  auto places = [&](int w) { return range_bits(base + 32 * w, lo, edge) & ~s_gt[w]; };
  auto movers = [&](int w) { return range_bits(base + 32 * w, edge, hi) & s_gt[w]; };
  // free places and movers before each word, both in one number (places in the low half)
  int total = 0;
  for (int w0 = 0; w0 < nw; w0 += ET) {
    const int w = w0 + tid;
    int here;
    const int before =
        block_prefix(w < nw ? __popc(places(w)) | __popc(movers(w)) << 16 : 0, s_warp, &here);
    if (w < nw) s_eq[w] = (uint32_t)(total + before);
    total += here;
  }
  if (tid == 0) {
    s_count[1] = total & 0xffff;
    s_count[2] = (int)((unsigned)total >> 16);
  }
  sync_all();                                  // and every CTA is done with its weights
  int at_place, at_mover;
  const int moves = sum_of(&s_count[1], &at_place);
  (void)sum_of(&s_count[2], &at_mover);        // as many: both are wanted less the survivors
                                               // before the edge
  // the lists: entry x of the cluster's is entry x / cs of CTA x % cs, at most seg / 2
  const int half = seg / 2, cs_shift = __ffs(cs) - 1;
  for (int p = tid; p < seg; p += ET) {
    const int w = p >> 5;
    const uint32_t bit = 1u << (p & 31), mv = movers(w), pl = places(w);
    if ((mv | pl) & bit) {
      const bool moves_here = mv & bit;
      const uint32_t before = s_eq[w];
      const int x = moves_here ? at_mover + (int)(before >> 16) + __popc(mv & (bit - 1u))
                               : at_place + (int)(before & 0xffffu) + __popc(pl & (bit - 1u));
      cl.map_shared_rank(keys, x & (cs - 1))[(moves_here ? 0 : half) + (x >> cs_shift)] = base + p;
    }
  }
  sync_all();

  // ---- moves of this CTA's share: all sources lie behind the edge, all places before it
  const int mine = (moves - rank + cs - 1) >> cs_shift;    // moves >= 0, rank < cs
  uint32_t* src = keys;
  uint32_t* dst = keys + half;
  const int bmask = (1 << t.bs_shift) - 1;
  auto cell = [&](int p) {
    return ((uint32_t)table[p >> t.bs_shift] * (uint32_t)a.Hkv + (uint32_t)g << t.bs_shift) +
           (uint32_t)(p & bmask);
  };
  float wt = 0.f, ks = 0.f, vs = 0.f;          // of this thread's first move
  uint32_t to = 0;
  int wq = -1;
  for (int x = tid; x < mine; x += ET) {
    const int p = (int)src[x], q = (int)dst[x];
    const uint32_t f = cell(p), d = cell(q);
    src[x] = f;
    dst[x] = d;
    float k = 0.f, v = 0.f;
    const float w = weights[p];
    if (a.scale[0]) { k = a.scale[0][f]; v = a.scale[1][f]; }
    if (x == tid) {                            // written behind the codes' loads
      wt = w; ks = k; vs = v; to = d; wq = q;
    } else {
      weights[q] = w;
      if (a.scale[0]) { a.scale[0][d] = k; a.scale[1][d] = v; }
    }
  }
  __syncthreads();
  const int cshift = a.chunk_shift;            // 16-byte chunks of a cell in one buffer
  const int cmask = (1 << cshift) - 1;
  auto chunk_of = [&](int which, uint32_t c, int k) {
    return reinterpret_cast<uint4*>(a.code[which]) + ((long long)c << cshift) + k;
  };
  const int chunks = mine << (cshift + 1);     // below 2^21
  for (int e0 = tid; e0 < chunks; e0 += ET * MOVE_U) {
    uint4 c[MOVE_U];
#pragma unroll
    for (int u = 0; u < MOVE_U; ++u) {
      const int e = e0 + u * ET;
      if (e < chunks) c[u] = *chunk_of((e >> cshift) & 1, src[e >> (cshift + 1)], e & cmask);
    }
#pragma unroll
    for (int u = 0; u < MOVE_U; ++u) {
      const int e = e0 + u * ET;
      if (e < chunks) *chunk_of((e >> cshift) & 1, dst[e >> (cshift + 1)], e & cmask) = c[u];
    }
  }
  if (wq >= 0) {
    weights[wq] = wt;
    if (a.scale[0]) { a.scale[0][to] = ks; a.scale[1][to] = vs; }
  }

  // ---- the last cells, in order.  Where old and new places overlap one CTA takes
  // them, a round at a time: all of a round is read before any of it is written
  const int down = L - keep;
  const bool apart = down >= a.last;
  const int share = apart ? (a.last + cs - 1) / cs : (rank == 0 ? a.last : 0);
  const int r0 = apart ? min(a.last, rank * share) : 0, r1 = min(a.last, r0 + share);
  const int round = max(1, (ET * MOVE_U) >> (cshift + 1));   // cells, at most 2 ET
  for (int x0 = r0; x0 == r0 || x0 < r1; x0 += round) {
    const int cells = min(round, r1 - x0), nch = cells << (cshift + 1);   // <= 0: none here
    uint4 v[MOVE_U];
    float rw[2], rk[2], rv[2];
#pragma unroll
    for (int u = 0; u < MOVE_U; ++u) {
      const int e = tid + u * ET;
      if (e < nch) v[u] = *chunk_of((e >> cshift) & 1, cell(hi + x0 + (e >> (cshift + 1))), e & cmask);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int x = tid + u * ET;
      if (x < cells) {
        const uint32_t f = cell(hi + x0 + x);
        rw[u] = weights[hi + x0 + x];
        if (a.scale[0]) { rk[u] = a.scale[0][f]; rv[u] = a.scale[1][f]; }
      }
    }
    // the round has been read; before the first write, everything that moved above too
    if (x0 == r0) sync_all();
    else __syncthreads();
#pragma unroll
    for (int u = 0; u < MOVE_U; ++u) {
      const int e = tid + u * ET;
      if (e < nch) *chunk_of((e >> cshift) & 1, cell(edge + x0 + (e >> (cshift + 1))), e & cmask) = v[u];
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int x = tid + u * ET;
      if (x < cells) {
        const uint32_t d = cell(edge + x0 + x);
        weights[edge + x0 + x] = rw[u];
        if (a.scale[0]) { a.scale[0][d] = rk[u]; a.scale[1][d] = rv[u]; }
      }
    }
  }
  sync_all();                                  // the weights behind the new end have been read
  for (int p = keep + rank * ET + tid; p < L; p += cs * ET) weights[p] = 0.f;
  if (teller) a.new_lens[i] = keep;
}

}  // namespace

// CTAs per (row, KV head): as many as fill the SMs about twice, though no segment of 1,024
// cells or fewer is cut, and as many as hold the row's weights.  0: no cluster does.
int evict_cluster(int max_len, long long items) {
  int cs = 1;
  const long long sms = sm_count();
  while (cs < MAX_CLUSTER) {
    const long long seg = ((long long)max_len + cs - 1) / cs;
    if (seg <= MAX_SEGMENT / 2 && (items * cs >= 2 * sms || seg <= 1024)) break;
    cs *= 2;
  }
  return ((long long)max_len + cs - 1) / cs <= MAX_SEGMENT ? cs : 0;
}

cudaError_t launch_evict(EvictArgs a, int n, cudaStream_t st) {
  const int cs = evict_cluster(a.max_len, (long long)n * a.Hkv);
  if (cs <= 0) return cudaErrorInvalidValue;
  a.seg_max = ((a.max_len + cs - 1) / cs + 31) & ~31;
  const int smem = a.seg_max * 4 + 2 * (a.seg_max / 32) * 4;
  static bool attr_set[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               MAX_SEGMENT * 4 + 2 * (MAX_SEGMENT / 32) * 4);
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((long long)n * a.Hkv * cs));
  cfg.blockDim = dim3(ET);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cs;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, evict_kernel, a);
}

}  // namespace kvq
