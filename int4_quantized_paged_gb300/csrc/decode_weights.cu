// Decode attention that accumulates the softmax weight of every cell:
//   a[b][h][p] <- decay a[b][h][p] + sum over the query heads of KV head h of
//                 softmax_p(scale <q, K_hat[p]>)
// beside the attention's output: what an eviction goes by.
//
// The weight of a position needs the row's whole sum, which is known when its last
// tile has been read.  The decode kernel therefore leaves the scores, 4 G bytes for a
// position and KV head where K and V took 2 D and more, and a second pass turns them
// into weights with one exponent each: K is not read again.  Nothing is added by
// atomics; each sum has one thread, which adds the heads in their order.
//
// What bounds it: the decode's bytes, and 8 G + 8 more for each position and KV head
// (scores written and read, of which the L2 holds the read ones of small batches; a
// weight read and written).  64 rows of 1,500-4,200 positions, 32 heads of 128, FP8 per
// token and head: 79.5 us, 5.1 TB/s, where the decode without weights takes 68.5; 4 rows
// of 20,000-40,000, 64 heads of 64, BF16: 62.5 and 59.
#include <cuda.h>
#include <cuda_runtime.h>

#include "decode_kernel.cuh"
#include "join.cuh"

namespace kvq {
namespace {

constexpr int AT = 256;                        // threads
constexpr int AU = 4;                          // positions per thread, AT apart

template <int G>
__global__ void __launch_bounds__(AT)
    accumulate_kernel(const DecodeArgs a, float* weights, long long stride, float decay) {
  const int b = blockIdx.z, g = blockIdx.y;
  const int L = ctx_len(a, b);
  const int p0 = blockIdx.x * (AT * AU) + threadIdx.x;
  if ((int)blockIdx.x * (AT * AU) >= L) {
    // this grid does not end before the one it was launched behind, even if no row has a cell
    if (blockIdx.x == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  float* row = weights + ((long long)b * a.Hkv + g) * stride;
  float past[AU];
#pragma unroll
  for (int u = 0; u < AU; ++u) past[u] = p0 + u * AT < L ? row[p0 + u * AT] : 0.f;
  // launched as a programmatic dependent: the scores and sums are visible below
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float lse[G];
#pragma unroll
  for (int j = 0; j < G; ++j) lse[j] = a.lse[(long long)b * a.Hq + g * G + j];
  const float* scores = a.scores + ((long long)b * a.Hkv + g) * a.cap * G;
  float s[AU][G];
#pragma unroll
  for (int u = 0; u < AU; ++u) {
    const int p = p0 + u * AT;
    if (p >= L) continue;
    if constexpr (G >= 4) {
#pragma unroll
      for (int j = 0; j < G; j += 4) {
        const float4 v = *reinterpret_cast<const float4*>(scores + (long long)p * G + j);
        s[u][j] = v.x; s[u][j + 1] = v.y; s[u][j + 2] = v.z; s[u][j + 3] = v.w;
      }
    } else if constexpr (G == 2) {
      const float2 v = *reinterpret_cast<const float2*>(scores + (long long)p * 2);
      s[u][0] = v.x; s[u][1] = v.y;
    } else {
      s[u][0] = scores[p];
    }
  }
#pragma unroll
  for (int u = 0; u < AU; ++u) {
    const int p = p0 + u * AT;
    if (p >= L) continue;
    float w = 0.f;
#pragma unroll
    for (int j = 0; j < G; ++j)                // a row whose every block was refused has no sum
      w += lse[j] == -INFINITY ? 0.f : ex2(s[u][j] - lse[j]);
    row[p] = fmaf(decay, past[u], w);
  }
}

struct WeightsOp {
  const DecodeArgs& a;
  float* weights;
  long long stride;
  float decay;
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
    if (prepare<MODE, D, G, DECODE_WEIGHTS>(&smem) <= 0) return cudaErrorInvalidConfiguration;
    const int ctas = (a.workers + WARPS - 1) / WARPS;
    decode_kernel<MODE, D, G, DECODE_WEIGHTS><<<ctas, WARPS * 32, smem, st>>>(a, km, vm);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    e = launch_dependent(join_kernel<D, G, false>, dim3((unsigned)(a.B * a.Hkv)), JT, 0, st, a, SharedArgs{});
    if (e != cudaSuccess) return e;
    const unsigned parts = (unsigned)((a.cap + AT * AU - 1) / (AT * AU));
    if (parts == 0) return cudaSuccess;
    return launch_dependent(accumulate_kernel<G>, dim3(parts, (unsigned)a.Hkv, (unsigned)a.B), AT, 0, st, a,
                            weights, stride, decay);
  }
};

}  // namespace

cudaError_t launch_decode_weights(int mode, int D, int G, const DecodeArgs& a, float* weights,
                                  long long stride, float decay, cudaStream_t st) {
  return with_layer(mode, D, G, WeightsOp{a, weights, stride, decay, st});
}

}  // namespace kvq
