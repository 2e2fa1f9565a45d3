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
// What bounds it.  The bytes (weights once, moved cells twice) take a few us; the
// rest is the chain of about nine cluster barriers with their scans.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kvq_internal.h"

namespace kvq {
namespace {

namespace cg = cooperative_groups;

constexpr int ET = 256;                        // threads per CTA, one per histogram bin
constexpr int EW = ET / 32;
constexpr int MAX_CLUSTER = 8;
constexpr int MAX_SEGMENT = 48 * 1024;         // cells of a CTA (their weights: 192 KB)
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

__global__ void __launch_bounds__(ET) evict_kernel(const EvictArgs a) {
  cg::cluster_group cl = cg::this_cluster();
  const int cs = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int item = blockIdx.x / cs;
  const int i = item / a.Hkv, g = item - i * a.Hkv;
  const PageTables& t = a.t;

  extern __shared__ uint32_t dyn[];
  uint32_t* keys = dyn;                        // [seg]; later the lists of moves
  uint32_t* s_gt = dyn + a.seg_max;            // [seg / 32] above the threshold, then: stays
  uint32_t* s_eq = s_gt + a.seg_max / 32;      // [seg / 32] at the threshold
  __shared__ int hist[2][ET];
  __shared__ int s_warp[EW];
  __shared__ int s_pick[3];                    // bin, weights of it still wanted, weights in it
  __shared__ int s_bad, s_count[3];            // what the other CTAs read: ties, places, survivors

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

  // ---- every block of the row names one of the pool that no other row holds
  if (tid == 0) s_bad = 0;
  hist[0][tid] = 0;
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
#pragma unroll 1
  for (int pass = 0; pass < 4; ++pass) {
    const int shift = 24 - 8 * pass;
    int* h = hist[pass & 1];
    for (int p0 = c0 + warp * 32; p0 < c1; p0 += ET) {
      const int p = p0 + lane;
      const uint32_t key = p < c1 ? keys[p] : 0u;
      // 64 bits: a shift by 32 in the first pass
      const bool in = p < c1 && ((uint64_t)(key ^ prefix) >> (shift + 8)) == 0;
      const unsigned active = __ballot_sync(0xffffffffu, in);
      if (in) {
        // neighbours of one bin count together
        const int bin = (key >> shift) & 255;
        const unsigned same = __match_any_sync(active, bin);
        if (lane == __ffs(same) - 1) atomicAdd(&h[bin], __popc(same));
      }
    }
    cl.sync();
    if (pass == 0) {
      int bad = 0;
      for (int r = 0; r < cs; ++r) bad |= *cl.map_shared_rank(&s_bad, r);
      if (bad) {                               // the same for the whole cluster
        if (teller) {
          a.new_lens[i] = L;
          atomicOr(t.err, ERR_BAD_INDEX);
        }
        cl.sync();                             // no CTA leaves while another reads its flag
        return;
      }
    }
    hist[(pass + 1) & 1][tid] = 0;             // read last before this barrier
    int n = 0;
    for (int r = 0; r < cs; ++r) n += cl.map_shared_rank(h, r)[255 - tid];
    // thread x holds bin 255 - x: the weights of higher bins are those of lower threads
    int all;
    const int above = block_prefix(n, s_warp, &all);
    if (above < rest && rest <= above + n) {
      s_pick[0] = 255 - tid;
      s_pick[1] = rest - above;
      s_pick[2] = n;
    }
    __syncthreads();
    if (wanted > 0) {
      prefix |= (uint32_t)s_pick[0] << shift;
      rest = s_pick[1];
      ties = s_pick[2];
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
  auto count = [&](auto bits_of) {             // bits over the CTA's words
    int n = 0;
    for (int w = tid; w < nw; w += ET) n += __popc(bits_of(w));
    int all;
    (void)block_prefix(n, s_warp, &all);
    return all;
  };
  auto before_me = [&](int which, int* total) {
    int n = 0, all = 0;
    for (int r = 0; r < cs; ++r) {
      const int x = *cl.map_shared_rank(&s_count[which], r);
      if (r < rank) n += x;
      all += x;
    }
    *total = all;
    return n;
  };
  if (rest < ties) {                           // the same for the whole cluster
    const int n = count([&](int w) { return s_eq[w]; });
    if (tid == 0) s_count[0] = n;
    cl.sync();
    int all, at = before_me(0, &all);
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
  {
    const int np = count(places), nm = count(movers);
    if (tid == 0) { s_count[1] = np; s_count[2] = nm; }
  }
  cl.sync();                                   // and every CTA is done with its weights
  int moves, same;
  int at_place = before_me(1, &moves), at_mover = before_me(2, &same);
  // as many survivors behind the edge as places before it: both are wanted less the
  // survivors before it
  const int per = (moves + cs - 1) / cs;       // at most seg / 2
  const int half = seg / 2;
  // the lists: entry x of the cluster's is entry x % per of CTA x / per
  auto scatter = [&](auto bits_of, int at, int off) {
    for (int w0 = 0; w0 < nw; w0 += ET) {
      const int w = w0 + tid;
      uint32_t bits = w < nw ? bits_of(w) : 0u;
      int here;
      int x = at + block_prefix(__popc(bits), s_warp, &here);
      for (; bits; bits &= bits - 1, ++x) {
        const int owner = x / per;
        cl.map_shared_rank(keys, owner)[off + x - owner * per] = base + 32 * w + __ffs(bits) - 1;
      }
      at += here;
    }
  };
  scatter(movers, at_mover, 0);
  scatter(places, at_place, half);
  cl.sync();

  // ---- moves of this CTA's share: all sources lie behind the edge, all places before it
  const int mine = max(0, min(per, moves - rank * per));
  uint32_t* src = keys;
  uint32_t* dst = keys + half;
  const int bmask = (1 << t.bs_shift) - 1;
  auto cell = [&](int p) {
    return ((uint32_t)table[p >> t.bs_shift] * (uint32_t)a.Hkv + (uint32_t)g << t.bs_shift) +
           (uint32_t)(p & bmask);
  };
  for (int x = tid; x < mine; x += ET) {
    const int p = (int)src[x], q = (int)dst[x];
    const uint32_t from = cell(p), to = cell(q);
    weights[q] = weights[p];
    if (a.scale[0]) {
      a.scale[0][to] = a.scale[0][from];
      a.scale[1][to] = a.scale[1][from];
    }
    src[x] = from;
    dst[x] = to;
  }
  __syncthreads();
  const int cshift = a.chunk_shift;            // 16-byte chunks of a cell in one buffer
  const int cmask = (1 << cshift) - 1;
  auto chunk_of = [&](int which, uint32_t c, int k) {
    return reinterpret_cast<uint4*>(a.code[which]) + ((long long)c << cshift) + k;
  };
  const long long chunks = (long long)mine << (cshift + 1);
  for (long long e0 = tid; e0 < chunks; e0 += ET * MOVE_U) {
    uint4 v[MOVE_U];
#pragma unroll
    for (int u = 0; u < MOVE_U; ++u) {
      const long long e = e0 + u * ET;
      if (e < chunks) v[u] = *chunk_of((int)(e >> cshift) & 1, src[e >> (cshift + 1)], (int)e & cmask);
    }
#pragma unroll
    for (int u = 0; u < MOVE_U; ++u) {
      const long long e = e0 + u * ET;
      if (e < chunks) *chunk_of((int)(e >> cshift) & 1, dst[e >> (cshift + 1)], (int)e & cmask) = v[u];
    }
  }
  cl.sync();                                   // what moved has been read

  // ---- the last cells, in order.  Where old and new places overlap one CTA takes
  // them, a round at a time: all of a round is read before any of it is written
  const int down = L - keep;
  const bool apart = down >= a.last;
  const int share = apart ? (a.last + cs - 1) / cs : (rank == 0 ? a.last : 0);
  const int r0 = apart ? min(a.last, rank * share) : 0, r1 = min(a.last, r0 + share);
  const int round = max(1, (ET * MOVE_U) >> (cshift + 1));   // cells, at most 2 ET
  for (int x0 = r0; x0 < r1; x0 += round) {
    const int cells = min(round, r1 - x0);
    const int nch = cells << (cshift + 1);
    uint4 v[MOVE_U];
    float wt[2], k[2], s[2];
#pragma unroll
    for (int u = 0; u < MOVE_U; ++u) {
      const int e = tid + u * ET;
      if (e < nch) v[u] = *chunk_of((e >> cshift) & 1, cell(hi + x0 + (e >> (cshift + 1))), e & cmask);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int x = tid + u * ET;
      if (x < cells) {
        const uint32_t from = cell(hi + x0 + x);
        wt[u] = weights[hi + x0 + x];
        if (a.scale[0]) { k[u] = a.scale[0][from]; s[u] = a.scale[1][from]; }
      }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < MOVE_U; ++u) {
      const int e = tid + u * ET;
      if (e < nch) *chunk_of((e >> cshift) & 1, cell(edge + x0 + (e >> (cshift + 1))), e & cmask) = v[u];
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int x = tid + u * ET;
      if (x < cells) {
        const uint32_t to = cell(edge + x0 + x);
        weights[edge + x0 + x] = wt[u];
        if (a.scale[0]) { a.scale[0][to] = k[u]; a.scale[1][to] = s[u]; }
      }
    }
    __syncthreads();
  }
  cl.sync();                                   // the weights behind the new end have been read
  for (int p = keep + rank * ET + tid; p < L; p += cs * ET) weights[p] = 0.f;
  if (teller) a.new_lens[i] = keep;
}

}  // namespace

// CTAs per (row, KV head): as many as fill the SMs about twice, with no fewer than
// 1,024 cells each, and as many as hold the row's weights.  0: no cluster does.
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
