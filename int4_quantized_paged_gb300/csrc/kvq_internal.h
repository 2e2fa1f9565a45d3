// Internal interface between the C-ABI layer (api.cu) and the kernel
// translation units.  Not installed; not part of the ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace kvq {

enum Mode { BF16 = 0, FP8_PER_TENSOR = 1, FP8_PER_HEAD = 2, FP8_PER_TOKEN_HEAD = 3,
            INT4_PER_TOKEN_HEAD = 4 };

// Device error word bits.
enum : unsigned { ERR_BAD_INDEX = 1u, ERR_TIMEOUT = 2u, ERR_NO_BLOCKS = 4u };

struct WriteArgs {
  const uint16_t* k_new;       // bf16 bits
  const uint16_t* v_new;
  long long token_stride;      // elements between tokens
  const long long* slots;
  long long T;
  int Hkv;
  int bs;
  int bs_shift;                // log2(bs)
  long long num_blocks;
  const float* k_scale;        // static modes
  const float* v_scale;
  uint8_t* k_cache;
  uint8_t* v_cache;
  float* k_cs;                 // dynamic modes
  float* v_cs;
  unsigned* err;
};

struct DecodeArgs {
  const uint16_t* q;           // bf16 [B][Hq][D]
  const float* q_scale;        // FP8 query: [1] or [Hq] scales (nullptr: bf16 query)
  int q_scale_count;
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const float* k_scale;        // static modes: [1] or [Hkv]
  const float* v_scale;
  const float* k_cs;           // dynamic modes: [num_blocks][Hkv][bs]
  const float* v_cs;
  const int* block_table;      // [B][max_blocks]
  const int* context_lens;     // [B]
  float* out;                  // [B][Hq][D] fp32, or
  uint16_t* out_bf16;          // [B][Hq][D] bf16 (RN of the fp32 result) when non-null
  float* ws_o;                 // [B*Hkv + workers][G][D] unnormalised partial outputs
  float* ws_ml;                // [B*Hkv + workers][G][2] running max (log2 units) and sum
  long long* item_tiles;       // [B*Hkv + 1] first tile of each item in the tile list; T last
  unsigned* err;
  int B, Hq, Hkv, bs, bs_shift, max_blocks, window, workers;
  int stream_once;             // pages larger than L2: copy them evict-first
  long long num_blocks;
  float qk_scale;              // softmax_scale * log2(e)
};

enum RopeLayout { ROPE_HALF = 0, ROPE_INTERLEAVED = 1 };
constexpr int ROPE_MAX_PAIRS = 128;

// Frequencies of a rotation as fractions of a turn per position times 2^64.
struct RopeTable {
  unsigned long long phase[ROPE_MAX_PAIRS];
  float magnitude;
};

struct RopeArgs {
  WriteArgs w;                 // k, v, slots, caches (Hkv 0, slots nullptr: rotation only)
  const uint16_t* q;           // bf16, token stride q_stride (Hq 0: none)
  uint16_t* q_out;             // may be q
  long long q_stride, q_out_stride;
  const long long* positions;  // [T]
  int Hq;
  int rotary;                  // rotated elements of a head
  float sin_magnitude;         // magnitude, negative for the transpose
  int slices, per_slice;       // set by the launcher: slices of a token's vectors, vectors in each
};

// Page tables and reference counts of a pool of num_blocks blocks.
struct PageTables {
  int* ref;                    // [num_blocks]
  int* table;                  // [rows][max_blocks]
  int* lens;                   // [rows]
  long long num_blocks;
  int rows, max_blocks, bs, bs_shift;
  unsigned* err;
};

struct ExtendArgs {
  const int* rows;             // [n]
  const int* new_tokens;       // [n]
  int n;
  long long max_tokens;
  int* query_start;            // [n + 1]
  long long* positions;        // [max_tokens]
  long long* slots;            // [max_tokens]
  int* copies;                 // [n][2]
};
constexpr int EXTEND_MAX_ROWS = 4096;

struct CopyLayer {
  void* buf[4];                // K codes, V codes, K scales, V scales
  unsigned code_chunks, scale_chunks;   // 16-byte chunks of one block in a code / scale buffer
};
constexpr int COPY_MAX_LAYERS = 80;     // per launch (the kernel's parameters end at 4 KB)

struct CopyArgs {
  CopyLayer layer[COPY_MAX_LAYERS];
  const int* pairs;            // [max_pairs][2]
  const int* num_pairs;        // device count, or nullptr
  int max_pairs, layers;
  long long num_blocks;
  unsigned* err;
};

// Launchers (return cudaGetLastError() of the launch).
cudaError_t launch_cache_write(int mode, int D, const WriteArgs& a, cudaStream_t st);
cudaError_t launch_rope(int mode, int D, int layout, RopeArgs a, const RopeTable& tab,
                        cudaStream_t st);
cudaError_t launch_truncate(const PageTables& t, const int* rows, const int* keep_lens, int n,
                            cudaStream_t st);
cudaError_t launch_fork(const PageTables& t, const int* parents, const int* children, int n,
                        cudaStream_t st);
cudaError_t launch_extend(const PageTables& t, const ExtendArgs& x, cudaStream_t st);
cudaError_t launch_compact(const PageTables& t, int* moves, int* num_moves, cudaStream_t st);
cudaError_t launch_copy_blocks(const CopyArgs& a, cudaStream_t st);
cudaError_t launch_calibrate(const uint16_t* x, long long T, int Hkv, int D, float qmax,
                             float* out, cudaStream_t st);
cudaError_t launch_e4m3_encode(const float* in, uint8_t* out, long long n, cudaStream_t st);
// One warp whose bounded barrier wait runs out after limit_cycles (sets TIMEOUT).
cudaError_t launch_wait_check(long long limit_cycles, cudaStream_t st);
// Returns cudaErrorInvalidValue for an unsupported (mode, D, G) combination.
cudaError_t launch_decode(int mode, int D, int G, const DecodeArgs& a, cudaStream_t st);
bool decode_supported(int mode, int D, int G);
// Prefill: one CTA per (query tile, sequence, KV head); DecodeArgs supplies the
// caches, scales, block table, context lengths, q and out (no workspace).
cudaError_t launch_prefill(int mode, int D, int G, const DecodeArgs& a, const int* query_start,
                           int max_query_len, cudaStream_t st);
// Warp-specialised prefill for quantized layers of head_dim 64 or 128.
bool prefill_ws_supports(int mode, int D);
cudaError_t launch_prefill_ws(int mode, int D, int G, const DecodeArgs& a, const int* query_start,
                              int max_query_len, cudaStream_t st);
int prefill_rows_per_cta();
// Resident decode CTAs per SM on the current device (0 if unknown: no device).
int decode_ctas_per_sm(int mode, int D, int G);
int decode_warps_per_cta();

// 2-D TMA map of a layer's code buffer viewed as [total_bytes / 128] rows of
// 128 bytes, box of tile_bytes / 128 rows, 128B swizzle (false on failure).
bool make_tile_map(CUtensorMap* m, const void* base, long long total_bytes, int tile_bytes);

// A BF16 layer's K buffer as 64-d blocks of 16 cells (false on failure).
bool make_kblock_map(CUtensorMap* m, const void* base, long long total_bytes, int row_bytes);

// Cross attention of max_query_len queries a sequence at most: DecodeArgs as for
// the prefill, out_bf16, and for splits > 1 ws_o / ws_ml.
constexpr int CROSS_KEYS = 64;         // keys per tile; splits are whole tiles
int cross_query_tile(int D, int G);    // queries of one (sequence, KV head) a CTA takes
cudaError_t launch_cross(int mode, int D, int G, const DecodeArgs& a, const int* query_start,
                         int max_query_len, int splits, int split_tiles, cudaStream_t st);

// Device error word of the current device.
unsigned* error_word();

int sm_count();

}  // namespace kvq
