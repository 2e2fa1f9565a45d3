// Pages of the cache: extending, forking, truncating (freeing) and compacting
// sequences' page tables, and the copy of pages that extending and compacting ask for.
//
// State, all in the caller's device memory: ref_count[block], the number of
// table entries that hold a block (0: free); block_table[row][j]; and
// context_lens[row].  There is no free list: a call that needs blocks takes the
// lowest-numbered free ones, in the order of its rows, so that the result does
// not depend on the order of atomics.
//
// What bounds them.  The table calls are bookkeeping: kilobytes, a chain of a few
// dependent loads, and the launch itself.  Each is one launch.  Forking and
// truncating take one CTA per row.  Extending and compacting have to know how
// many blocks below a given one are free, a prefix count over ref_count; they
// run as one cluster of eight CTAs whose counts are exchanged through
// distributed shared memory, so no CTA waits on one that may not be running.
// The copy of pages is an HBM stream, every byte read and written once.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <limits.h>
#include <stdint.h>

#include "kvq_internal.h"

namespace kvq {
namespace {

namespace cg = cooperative_groups;

constexpr int CLUSTER = 8;
constexpr int CT = 1024;                       // threads per CTA of the cluster
constexpr int CW = CT / 32;
constexpr int ROW_T = 512;                     // threads per row of fork and truncate

__device__ __forceinline__ int ceil_shift(int x, int shift) {
  return (int)(((long long)x + (1LL << shift) - 1) >> shift);
}

__device__ __forceinline__ bool len_ok(const PageTables& t, int L) {
  return L >= 0 && (long long)L <= ((long long)t.max_blocks << t.bs_shift);
}

// Whether `x` stands among the first n entries of list (all threads of the CTA
// take part and get the answer).
__device__ __forceinline__ bool listed(const int* list, int n, int x) {
  bool hit = false;
  for (int j = threadIdx.x; j < n; j += blockDim.x) hit |= list[j] == x;
  return __syncthreads_or(hit);
}

// ---------------------------------------------------------------- truncate
__global__ void __launch_bounds__(ROW_T)
    truncate_kernel(const PageTables t, const int* rows, const int* keep_lens) {
  const int i = blockIdx.x, row = rows[i];
  const bool seen = listed(rows, i, row);
  const int keep = keep_lens ? keep_lens[i] : 0;
  const bool bad_row = seen || row < 0 || row >= t.rows || keep < 0;
  const int L = bad_row ? -1 : t.lens[row];
  if (!len_ok(t, L)) {                         // the same for the whole CTA
    if (threadIdx.x == 0) atomicOr(t.err, ERR_BAD_INDEX);
    return;
  }
  const int left = min(L, keep);
  __syncthreads();                             // every thread has read the length
  if (threadIdx.x == 0) t.lens[row] = left;
  int* entry = t.table + (long long)row * t.max_blocks;
  const int j1 = ceil_shift(L, t.bs_shift);
  for (int j = ceil_shift(left, t.bs_shift) + threadIdx.x; j < j1; j += ROW_T) {
    const int b = entry[j];
    entry[j] = -1;
    bool ok = b >= 0 && b < t.num_blocks;
    if (ok && atomicSub(t.ref + b, 1) <= 0) {
      atomicAdd(t.ref + b, 1);                 // it was free already: leave it so
      ok = false;
    }
    if (!ok) atomicOr(t.err, ERR_BAD_INDEX);
  }
}

// ---------------------------------------------------------------- fork
__global__ void __launch_bounds__(ROW_T)
    fork_kernel(const PageTables t, const int* parents, const int* children, int n) {
  const int i = blockIdx.x, p = parents[i], c = children[i];
  // a child listed earlier, and a parent that this call fills, are refused: no
  // row is both read and written, whatever order the CTAs run in
  const bool seen = listed(children, i, c);
  const bool filled = listed(children, n, p);
  const bool bad = seen || filled || p < 0 || p >= t.rows || c < 0 || c >= t.rows;
  const int L = bad ? -1 : t.lens[p];
  const int Lc = bad ? 0 : t.lens[c];
  __syncthreads();
  if (!len_ok(t, L) || Lc != 0) {
    if (threadIdx.x == 0) atomicOr(t.err, ERR_BAD_INDEX);
    return;
  }
  if (threadIdx.x == 0) t.lens[c] = L;
  const int* from = t.table + (long long)p * t.max_blocks;
  int* to = t.table + (long long)c * t.max_blocks;
  const int j1 = ceil_shift(L, t.bs_shift);
  for (int j = threadIdx.x; j < j1; j += ROW_T) {
    const int b = from[j];
    to[j] = b;
    if (b >= 0 && b < t.num_blocks) atomicAdd(t.ref + b, 1);
    else atomicOr(t.err, ERR_BAD_INDEX);
  }
}

// ---------------------------------------------------------------- cluster helpers
// The blocks are cut into one contiguous run per warp of the cluster, in order
// of the warps: [run, run_end) is this warp's.
struct Run {
  long long first, last;
};

__device__ __forceinline__ Run my_run(long long num_blocks, int rank, int warp) {
  const long long per = (num_blocks + CLUSTER * CW - 1) / (CLUSTER * CW);
  const long long w = (long long)rank * CW + warp;
  Run r;
  r.first = min(num_blocks, w * per);
  r.last = min(num_blocks, (w + 1) * per);
  return r;
}

// Blocks of the run below `below` that are free (or, with USED, in use); every
// lane gets the count.
template <bool USED>
__device__ __forceinline__ int count_run(const int* ref, const Run r, long long below, int lane) {
  int n = 0;
  const long long last = min(r.last, below);
#pragma unroll 8
  for (long long b = r.first + lane; b < last; b += 32) n += (ref[b] > 0) == USED;
  return __reduce_add_sync(0xffffffffu, n);
}

// Exclusive prefix over the cluster's warps of one value per warp, and the
// total.  s_warp: CW ints, s_total: one int that the other CTAs read.
__device__ __forceinline__ int cluster_prefix(cg::cluster_group& cl, int value, int* s_warp,
                                              int* s_total, int* total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) s_warp[warp] = value;
  __syncthreads();
  if (warp == 0) {
    const int v = s_warp[lane];
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    s_warp[lane] = incl - v;
    if (lane == 31) *s_total = incl;
  }
  cl.sync();
  int before = 0, all = 0;
  const int rank = (int)cl.block_rank();
#pragma unroll
  for (int r = 0; r < CLUSTER; ++r) {
    const int x = *cl.map_shared_rank(s_total, r);
    if (r < rank) before += x;
    all += x;
  }
  *total = all;
  return before + s_warp[warp];
}

// First i in [0, n) with incl[i] > x (n if none); incl does not decrease.
__device__ __forceinline__ int upper(const int* incl, int n, int x) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (incl[mid] > x) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

// ---------------------------------------------------------------- extend
// Shared memory: six ints for each row of the call.
__global__ void __cluster_dims__(CLUSTER, 1, 1) __launch_bounds__(CT)
    extend_kernel(const PageTables t, const ExtendArgs x) {
  cg::cluster_group cl = cg::this_cluster();
  extern __shared__ int dyn[];
  const int n = x.n;
  int* s_row = dyn;                            // row, or -1 - row where refused
  int* s_old = s_row + n;                      // its length before the call
  int* s_first = s_old + n;                    // first table entry it gets; bit 31: a shared tail's
  int* s_need = s_first + n;                   // inclusive prefix of the blocks needed
  int* s_tok = s_need + n;                     // inclusive prefix of the tokens
  int* s_seen = s_tok + n;                     // nonzero: the row is named earlier too
  __shared__ int s_warp[CW], s_total, s_most;
  __shared__ long long s_scan[2][CW];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)cl.block_rank();
  const bool lead = rank == 0;

  // ---- free blocks of this warp's run (its loads overlap the rows' below)
  const Run run = my_run(t.num_blocks, rank, warp);
  const int my_free = count_run<false>(t.ref, run, t.num_blocks, lane);

  // ---- the rows, by every CTA alike: thread tid takes rows tid * per ...
  for (int i = tid; i < n; i += CT) {
    s_row[i] = x.rows[i];
    s_seen[i] = 0;
  }
  if (tid == 0) s_most = 0;
  __syncthreads();
  // rows named twice: each row against the earlier ones, 32 at a time, the pairs
  // spread over all threads (a loop over them by the row's own thread took 4 us for
  // 256 rows)
  for (unsigned w = tid; w < (unsigned)n * ((unsigned)(n + 31) / 32); w += CT) {
    const int i = (int)(w % (unsigned)n), j0 = (int)(w / (unsigned)n) * 32;
    if (j0 >= i) continue;
    const int row = s_row[i];
    bool hit = false;
#pragma unroll
    for (int j = 0; j < 32; ++j) hit |= j0 + j < i && s_row[min(j0 + j, i)] == row;
    if (hit) s_seen[i] = 1;
  }
  __syncthreads();
  const int per = (n + CT - 1) / CT;
  long long need_sum = 0, tok_sum = 0;
  bool bad_any = false;
  for (int k = 0; k < per; ++k) {
    const int i = tid * per + k;
    if (i >= n) break;
    const int row = s_row[i];
    const int add = x.new_tokens[i];
    bool bad = row < 0 || row >= t.rows || add < 0;
    bad = bad || s_seen[i] != 0;
    const int L = bad ? 0 : t.lens[row];
    bad = bad || !len_ok(t, L) || (long long)L + add > ((long long)t.max_blocks << t.bs_shift);
    int need = 0, first = 0;
    if (!bad) {
      const int have = ceil_shift(L, t.bs_shift);
      first = have;
      need = ceil_shift(L + add, t.bs_shift) - have;
      if (add > 0 && (L & (t.bs - 1))) {
        const int b = t.table[(long long)row * t.max_blocks + have - 1];
        if (b < 0 || b >= t.num_blocks) bad = true;
        else if (t.ref[b] > 1) {               // the tail block is shared: a copy of its own
          first = (have - 1) | INT_MIN;
          ++need;
        }
      }
    }
    if (bad) need = 0;
    bad_any |= bad;
    s_old[i] = bad ? -1 : L;
    s_first[i] = first;
    need_sum += need;
    tok_sum += max(add, 0);
    s_need[i] = need;
    s_tok[i] = max(add, 0);
  }
  if (lead && bad_any) atomicOr(t.err, ERR_BAD_INDEX);

  // ---- inclusive prefixes over the rows
  long long ni = need_sum, ti = tok_sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long a = __shfl_up_sync(0xffffffffu, ni, o), b = __shfl_up_sync(0xffffffffu, ti, o);
    if (lane >= o) { ni += a; ti += b; }
  }
  if (lane == 31) { s_scan[0][warp] = ni; s_scan[1][warp] = ti; }
  __syncthreads();
  long long nb = ni - need_sum, tb = ti - tok_sum;
  for (int w = 0; w < warp; ++w) { nb += s_scan[0][w]; tb += s_scan[1][w]; }
  for (int k = 0; k < per; ++k) {
    const int i = tid * per + k;
    if (i >= n) break;
    nb += s_need[i];
    tb += s_tok[i];
    s_need[i] = (int)min(nb, (long long)INT_MAX);
    s_tok[i] = (int)min(tb, (long long)INT_MAX);
  }

  // ---- free blocks before this warp's run, and in all
  int free_all;
  int rank_free = cluster_prefix(cl, my_free, s_warp, &s_total, &free_all);

  // ---- which rows get what they ask for: all of it or nothing.  Both prefixes
  // grow along the rows, so the rows that do hold the first ranks
  auto granted = [&](int i) -> bool {
    const int before = i ? s_need[i - 1] : 0;
    return s_old[i] >= 0 && s_tok[i] <= x.max_tokens &&
           (s_need[i] == before || s_need[i] <= free_all);
  };
  int most = 0;
  bool short_any = false, past_any = false;
  for (int i = tid; i < n; i += CT) {
    const bool g = granted(i);
    const int before = i ? s_need[i - 1] : 0;
    if (g && s_need[i] != before) most = max(most, s_need[i]);
    if (s_old[i] >= 0 && !g) {
      if (s_tok[i] > x.max_tokens) past_any = true;
      else short_any = true;
    }
    if (lead && !(g && s_first[i] < 0)) {
      x.copies[2 * i] = -1;
      x.copies[2 * i + 1] = -1;
    }
    if (lead) x.query_start[i + 1] = s_tok[i];
  }
  if (lead && tid == 0) x.query_start[0] = 0;
  most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 0 && most > 0) atomicMax(&s_most, most);
  if (lead && short_any) atomicOr(t.err, ERR_NO_BLOCKS);
  if (lead && past_any) atomicOr(t.err, ERR_BAD_INDEX);
  __syncthreads();
  most = s_most;

  // ---- the free block of rank r goes to the row whose prefix covers r
  for (long long b0 = run.first; b0 < run.last && rank_free < most; b0 += 32) {
    const long long b = b0 + lane;
    const bool fr = b < run.last && t.ref[b] <= 0;
    const unsigned m = __ballot_sync(0xffffffffu, fr);
    const int r = rank_free + __popc(m & ((1u << lane) - 1u));
    if (fr && r < most) {
      const int i = upper(s_need, n, r);
      const int k = r - (i ? s_need[i - 1] : 0);
      const int first = s_first[i];
      int* entry = t.table + (long long)s_row[i] * t.max_blocks + (first & INT_MAX) + k;
      if (first < 0 && k == 0) {
        x.copies[2 * i] = *entry;
        x.copies[2 * i + 1] = (int)b;
      }
      *entry = (int)b;
      t.ref[b] = 1;
    }
    rank_free += __popc(m);
  }
  cl.sync();                                   // tables and copies are visible to the cluster

  // ---- the shared tails lose a holder; lengths grow (no CTA reads them any more)
  if (lead)
    for (int i = tid; i < n; i += CT)
      if (granted(i)) {
        if (s_first[i] < 0) atomicSub(t.ref + x.copies[2 * i], 1);
        t.lens[s_row[i]] = s_old[i] + (s_tok[i] - (i ? s_tok[i - 1] : 0));
      }

  // ---- positions and slots of the new tokens
  const long long total = n ? s_tok[n - 1] : 0;
  for (long long k = (long long)rank * CT + tid; k < x.max_tokens; k += CLUSTER * CT) {
    long long pos = 0, slot = -1;
    if (k < total) {
      const int i = upper(s_tok, n, (int)k);
      if (s_old[i] >= 0) {
        pos = s_old[i] + (k - (i ? s_tok[i - 1] : 0));
        if (granted(i)) {
          const int b = t.table[(long long)s_row[i] * t.max_blocks + (pos >> t.bs_shift)];
          slot = ((long long)b << t.bs_shift) + (pos & (t.bs - 1));
        }
      }
    }
    x.positions[k] = pos;
    x.slots[k] = slot;
  }
}

// ---------------------------------------------------------------- compact
// Blocks in use at n_used and above move to the free blocks below it, both in
// ascending order.  While the tables are rewritten, ref_count of a block that
// moves holds -1 - its new id, so the map needs no memory of its own.
__global__ void __cluster_dims__(CLUSTER, 1, 1) __launch_bounds__(CT)
    compact_kernel(const PageTables t, int* moves, int* num_moves) {
  cg::cluster_group cl = cg::this_cluster();
  __shared__ int s_warp[2][CW], s_total[2];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)cl.block_rank();
  const Run run = my_run(t.num_blocks, rank, warp);
  int n_used, low;                             // blocks in use, and those of them below n_used
  int used = cluster_prefix(cl, count_run<true>(t.ref, run, t.num_blocks, lane), s_warp[0],
                            &s_total[0], &n_used);
  (void)cluster_prefix(cl, count_run<true>(t.ref, run, n_used, lane), s_warp[1], &s_total[1], &low);
  const int n = n_used - low;                  // holes below n_used = blocks that move
  for (long long b0 = run.first; b0 < run.last; b0 += 32) {
    const long long b = b0 + lane;
    const bool in = b < run.last;
    const bool u = in && t.ref[b] > 0;
    const unsigned m = __ballot_sync(0xffffffffu, u);
    const int before = used + __popc(m & ((1u << lane) - 1u));   // blocks in use below b
    if (u && b >= n_used) moves[2 * (long long)(before - low)] = (int)b;
    if (in && !u && b < n_used) moves[2 * (b - before) + 1] = (int)b;
    used += __popc(m);
  }
  if (rank == 0 && tid == 0) *num_moves = n;
  cl.sync();
  const int ct = rank * CT + tid;
  for (int i = ct; i < n; i += CLUSTER * CT) {
    const int s = moves[2 * (long long)i], d = moves[2 * (long long)i + 1];
    t.ref[d] = t.ref[s];
    t.ref[s] = -1 - d;
  }
  cl.sync();
  constexpr int SEG = 256;                     // table entries a warp takes at a time
  const int segs = (t.max_blocks + SEG - 1) / SEG;
  for (long long w = rank * CW + warp; w < (long long)t.rows * segs; w += CLUSTER * CW) {
    const int row = (int)(w / segs);
    const int j0 = (int)(w - (long long)row * segs) * SEG;
    const int L = t.lens[row];
    if (!len_ok(t, L)) {
      if (lane == 0 && j0 == 0) atomicOr(t.err, ERR_BAD_INDEX);
      continue;
    }
    const int j1 = min(j0 + SEG, ceil_shift(L, t.bs_shift));
    int* entry = t.table + (long long)row * t.max_blocks;
#pragma unroll 4
    for (int j = j0 + lane; j < j1; j += 32) {
      const int b = entry[j];
      const bool ok = b >= 0 && b < t.num_blocks;
      const int f = ok ? t.ref[b] : 0;
      if (f < 0) entry[j] = -1 - f;
      else if (f == 0) atomicOr(t.err, ERR_BAD_INDEX);   // no such block, or one that nothing holds
    }
  }
  cl.sync();
  for (int i = ct; i < n; i += CLUSTER * CT) t.ref[moves[2 * (long long)i]] = 0;
}

// ---------------------------------------------------------------- copy
constexpr int COPY_T = 256;
constexpr int COPY_U = 8;                      // 16-byte chunks a thread has in flight

// grid (x, layer).  A pair's bytes in a layer (K codes, V codes, K scales, V
// scales) are one run of `chunks` 16-byte chunks; the runs of all pairs are cut
// into equal shares of COPY_T * COPY_U chunks, whatever the page size.
__global__ void __launch_bounds__(COPY_T)
    copy_kernel(const __grid_constant__ CopyArgs a) {
  const CopyLayer& ly = a.layer[blockIdx.y];
  const unsigned code = ly.code_chunks, scale = ly.scale_chunks;
  const unsigned chunks = 2 * (code + scale);
  const int n = a.num_pairs ? max(0, min(*a.num_pairs, a.max_pairs)) : a.max_pairs;
  const long long total = (long long)n * chunks;
  const unsigned step_pair = COPY_T / chunks, step_rem = COPY_T % chunks;
  for (long long base = (long long)blockIdx.x * (COPY_T * COPY_U); base < total;
       base += (long long)gridDim.x * (COPY_T * COPY_U)) {
    const long long first = base + threadIdx.x;
    long long pair = first / chunks;
    unsigned rem = (unsigned)(first - pair * chunks);
    uint4 w[COPY_U];
    uint4* dst[COPY_U];
#pragma unroll
    for (int u = 0; u < COPY_U; ++u) {
      dst[u] = nullptr;
      if (first + u * COPY_T < total) {
        const int s = a.pairs[2 * pair], d = a.pairs[2 * pair + 1];
        if (s >= 0 && s < a.num_blocks && d >= 0 && d < a.num_blocks) {
          unsigned c = rem;
          const int part = c < code ? 0 : (c < 2 * code ? 1 : (c < 2 * code + scale ? 2 : 3));
          c -= part == 0 ? 0 : (part == 1 ? code : (part == 2 ? 2 * code : 2 * code + scale));
          const size_t len = part < 2 ? code : scale;
          uint4* buf = static_cast<uint4*>(ly.buf[part]);
          w[u] = buf[(size_t)s * len + c];
          dst[u] = buf + ((size_t)d * len + c);
        } else if (s >= 0 && rem == 0) {
          atomicOr(a.err, ERR_BAD_INDEX);
        }
      }
      pair += step_pair;
      rem += step_rem;
      if (rem >= chunks) { rem -= chunks; ++pair; }
    }
#pragma unroll
    for (int u = 0; u < COPY_U; ++u)
      if (dst[u]) *dst[u] = w[u];
  }
}

}  // namespace

cudaError_t launch_truncate(const PageTables& t, const int* rows, const int* keep, int n,
                            cudaStream_t st) {
  truncate_kernel<<<n, ROW_T, 0, st>>>(t, rows, keep);
  return cudaGetLastError();
}

cudaError_t launch_fork(const PageTables& t, const int* parents, const int* children, int n,
                        cudaStream_t st) {
  fork_kernel<<<n, ROW_T, 0, st>>>(t, parents, children, n);
  return cudaGetLastError();
}

cudaError_t launch_extend(const PageTables& t, const ExtendArgs& x, cudaStream_t st) {
  const int smem = 6 * x.n * (int)sizeof(int);
  if (smem > 40 * 1024) {                      // beside about 1 KB of static shared memory
    cudaError_t e = cudaFuncSetAttribute(extend_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         6 * EXTEND_MAX_ROWS * (int)sizeof(int));
    if (e != cudaSuccess) return e;
  }
  extend_kernel<<<CLUSTER, CT, smem, st>>>(t, x);
  return cudaGetLastError();
}

cudaError_t launch_compact(const PageTables& t, int* moves, int* num_moves, cudaStream_t st) {
  compact_kernel<<<CLUSTER, CT, 0, st>>>(t, moves, num_moves);
  return cudaGetLastError();
}

cudaError_t launch_copy_blocks(const CopyArgs& a, cudaStream_t st) {
  long long most = 0;
  for (int l = 0; l < a.layers; ++l) {
    const long long c = (long long)a.max_pairs * 2 * (a.layer[l].code_chunks + a.layer[l].scale_chunks);
    if (c > most) most = c;
  }
  long long gx = (most + COPY_T * COPY_U - 1) / (COPY_T * COPY_U);
  // about eight CTAs an SM are resident; several waves of them over the layers
  long long cap = ((long long)sm_count() * 32 + a.layers - 1) / a.layers;
  if (gx > cap) gx = cap;
  if (gx < 1) gx = 1;
  copy_kernel<<<dim3((unsigned)gx, (unsigned)a.layers), COPY_T, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace kvq
