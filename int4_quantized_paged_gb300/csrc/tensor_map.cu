// TMA maps of a layer's code buffers, and the driver's encoder that makes them.
// Host code only.
#include <cuda.h>
#include <cuda_runtime.h>

#include "kvq_internal.h"

namespace kvq {
namespace {

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn look_up() {
  void* p = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                       &q) != cudaSuccess ||
      q != cudaDriverEntryPointSuccess)
    return nullptr;
  return reinterpret_cast<EncodeFn>(p);
}

// Looked up by the first call; threads whose first calls meet wait for it (a
// flag of its own let the second one through before the pointer was there).
EncodeFn encode_fn() {
  static const EncodeFn fn = look_up();
  return fn;
}

// Tiles of bytes with the 128-byte swizzle.
bool encode(CUtensorMap* m, cuuint32_t rank, const void* base, const cuuint64_t* dims,
            const cuuint64_t* strides, const cuuint32_t* box) {
  const cuuint32_t estr[3] = {1, 1, 1};
  const EncodeFn fn = encode_fn();
  return fn && fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, rank, const_cast<void*>(base), dims, strides,
                  box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

// The layer's code buffer as a 2-D uint8 tensor of 128-byte rows; one box is
// a 16-position tile of one (block, KV head) page.
bool make_tile_map(CUtensorMap* m, const void* base, long long total_bytes, int tile_bytes) {
  const cuuint64_t dims[2] = {128, (cuuint64_t)(total_bytes / 128)};
  const cuuint64_t strides[1] = {128};
  const cuuint32_t box[2] = {128, (cuuint32_t)(tile_bytes / 128)};
  return encode(m, 2, base, dims, strides, box);
}

// A BF16 layer's K buffer as a 3-D uint8 tensor [cell][64-d block][128 bytes]:
// one box is one 64-d block of 16 consecutive cells, which lands as 16 rows
// of the K operand (128-byte swizzle).
bool make_kblock_map(CUtensorMap* m, const void* base, long long total_bytes, int row_bytes) {
  const cuuint64_t dims[3] = {128, (cuuint64_t)(row_bytes / 128),
                              (cuuint64_t)(total_bytes / row_bytes)};
  const cuuint64_t strides[2] = {128, (cuuint64_t)row_bytes};
  const cuuint32_t box[3] = {128, 1, 16};
  return encode(m, 3, base, dims, strides, box);
}

}  // namespace kvq
