/*
 * kvq.h -- C ABI of libkvq, a quantized paged KV cache for one GB300 GPU.
 *
 * Two hot operations, both hand-written CUDA for sm_103a:
 *
 *   kvq_cache_write       new bf16 K/V vectors -> scale -> FP8 E4M3 / packed
 *                         INT4 / BF16 codes -> scatter into paged blocks.
 *   kvq_decode_attention  paged GQA decode over that cache, K scale folded
 *                         into the QK product, V scale into the PV sum.
 *
 * Around them: the work plan of the decode (kvq_decode_plan), its variants
 * (bf16 output, FP8 query, no caller workspace), prefill attention over the
 * same cache (kvq_prefill_attention), static per-head calibration, the
 * capacity accounting of the pages and the device codec on its own.
 *
 * The operations and their scale layouts follow three pages:
 *   [P1] "Per-tensor vs per-head FP8 KV cache scales"
 *   [P2] "Per-token-head KV cache scale overhead"
 *   [P3] "FP8 KV cache layer skipping vs per-head scales"
 *
 * Conventions for every call:
 *  - Pointers named *_cache, q, out, k_new, v_new, slot_mapping, block_table,
 *    context_lens, workspace and the scale arrays are DEVICE pointers owned by
 *    the caller; the library never allocates, frees or retains them.
 *  - Streams and pointers belong to the current device of the calling thread.
 *  - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *    stream).  Device work is enqueued asynchronously on it; a call returns
 *    once the work is enqueued.
 *  - Argument errors are detected on the host before anything is launched and
 *    reported as a kvq_status; nothing is launched in that case.  Index errors
 *    found on the device (a slot or block id outside the cache, a negative
 *    context length) skip the bad access and set a device error word that
 *    kvq_get_device_error() reads.  No call falls back to another path.
 *  - kvq_ctx is host-only configuration; it may be shared between threads
 *    for the read-only calls below.
 */
#ifndef KVQ_H_
#define KVQ_H_

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum kvq_status {
  KVQ_OK = 0,
  KVQ_ERR_INVALID_ARG = 1,  /* null pointer, bad size or layer index */
  KVQ_ERR_UNSUPPORTED = 2,  /* head_dim, block_size, mode or GQA ratio not built */
  KVQ_ERR_ALIGNMENT = 3,    /* a pointer or stride breaks the 16-byte rule */
  KVQ_ERR_WORKSPACE = 4,    /* workspace missing or smaller than kvq_decode_plan says */
  KVQ_ERR_CUDA = 5,         /* a CUDA launch or query failed */
  KVQ_ERR_BAD_INDEX = 6,    /* device saw a slot / block id outside the cache */
  KVQ_ERR_TIMEOUT = 7,      /* a bounded device wait gave up */
  KVQ_ERR_NO_BLOCKS = 8     /* device found fewer free blocks than a call asked for */
} kvq_status;

/* Cache dtype and scale layout of one layer ([P1] "Per-tensor vs per-head FP8
 * KV cache scales"; [P2] "INT4 makes the metadata fraction larger"; [P3] "FP8
 * KV cache layer skipping vs per-head scales"). */
typedef enum kvq_mode {
  KVQ_BF16 = 0,                /* skipped layer: native bf16, no scales */
  KVQ_FP8_PER_TENSOR = 1,      /* E4M3, one K and one V scale per layer */
  KVQ_FP8_PER_HEAD = 2,        /* E4M3, static scale per KV head */
  KVQ_FP8_PER_TOKEN_HEAD = 3,  /* E4M3, scale = amax/448 per token and head */
  KVQ_INT4_PER_TOKEN_HEAD = 4  /* packed symmetric INT4, scale = amax/7 */
} kvq_mode;

/* Model/cache description, the pages' statement of the problem: layers, Hq
 * query heads and Hkv KV heads ([P3] "Per-head scales have fixed overhead"),
 * head size and block size ([P2] "Per-token-head KV cache scale overhead",
 * "Convert bytes into block capacity"), the scale layout of each layer ([P1]
 * "Per-tensor vs per-head FP8 KV cache scales"), and the window and skipped
 * (KVQ_BF16) layers ([P3] "FP8 KV cache layer skipping vs per-head scales",
 * "Layer skipping follows retained-token footprint"). */
typedef struct kvq_config {
  int num_layers;
  int num_q_heads;          /* Hq; a multiple of num_kv_heads, Hq/Hkv <= 16 */
  int num_kv_heads;         /* Hkv */
  int head_dim;             /* D: 64, 128 or 256 */
  int block_size;           /* tokens per block: 16, 32, 64 or 128 */
  long long num_blocks;     /* blocks in each layer's cache */
  const int* layer_mode;    /* host [num_layers] of kvq_mode; copied by kvq_create */
  const int* layer_window;  /* host [num_layers]; 0 = full attention, W > 0 keeps
                               the last W positions; NULL = all full */
  float softmax_scale;      /* 0 => 1/sqrt(head_dim) */
} kvq_config;

typedef struct kvq_ctx kvq_ctx;

/* Validates and copies *cfg into a new context (the description above;
 * [P1] and [P3] as cited there).  Host only; no CUDA call.  Returns
 * KVQ_ERR_INVALID_ARG for a null pointer, a non-positive count, Hq not a
 * multiple of Hkv, a mode outside kvq_mode or a negative window, and
 * KVQ_ERR_UNSUPPORTED for a head size, block size or GQA ratio that is not
 * built or a cache too large for 32-bit cell indices.  *out is NULL on
 * error; the caller releases a context with kvq_destroy. */
kvq_status kvq_create(const kvq_config* cfg, kvq_ctx** out);
void kvq_destroy(kvq_ctx* ctx);

/* Bytes of one layer's K code buffer and K scale buffer (V is the same).
 * Codes: [num_blocks][Hkv][block_size][row] with row = 2D (BF16), D (FP8) or
 * D/2 (INT4) bytes ([P2] "The FP8 scale tax is 4 divided by head size": one
 * byte per FP8 element; "INT4 makes the metadata fraction larger": half a
 * byte per INT4 element).  Scales (dynamic modes only, else 0): [num_blocks]
 * [Hkv][block_size] fp32, one K and one V scale per token and KV head
 * (same section; the pages' padding of each scale is not stored).  Each
 * (block, head) page of codes and of scales is contiguous; a block of
 * block_size tokens holds block_size x the per-token bytes ([P2] "Convert
 * bytes into block capacity").  Host only; KVQ_ERR_INVALID_ARG for a bad
 * context or layer.  The caller allocates the buffers. */
kvq_status kvq_layer_buffer_sizes(const kvq_ctx* ctx, int layer, size_t* code_bytes,
                                  size_t* scale_bytes);

/* Capacity accounting for one sequence of `context_tokens` positions.
 * Payload 2 x Hkv x D x bytes/elem per layer and retained token, dynamic
 * scales 2 x Hkv x 4 bytes ([P2] "Per-token-head KV cache scale overhead"),
 * static scales 8 bytes per per-tensor layer and 8 x Hkv per per-head layer
 * ([P1] "Static per-head metadata is almost free"), window layers retain
 * min(context, W) positions ([P3] "Layer skipping follows retained-token
 * footprint"), block bytes = per-token bytes x block size ([P2] "Convert
 * bytes into block capacity").  Bytes are before allocator rounding. */
typedef struct kvq_capacity {
  double payload_bytes_per_token;   /* all layers, codes only */
  double scale_bytes_per_token;     /* all layers, dynamic scales only */
  double bytes_per_token;           /* payload + scales */
  double block_bytes;               /* bytes_per_token x block_size */
  long long retained_positions;     /* sum over layers of retained positions */
  long long static_scale_bytes;     /* per-tensor and per-head scale arrays */
  double cache_bytes;               /* retained codes + scales + static scales */
  double bf16_cache_bytes;          /* the same retention with every layer BF16 */
} kvq_capacity;
kvq_status kvq_cache_bytes(const kvq_ctx* ctx, long long context_tokens, kvq_capacity* out);

/* Fused quantize-and-scatter of num_tokens new K/V vectors into `layer`.
 *
 * k_new, v_new: bf16 [num_tokens][Hkv][D], token t starting at element
 *   t * kv_token_stride (0 => Hkv*D); 16-byte aligned, stride a multiple of 8.
 * slot_mapping: int64 [num_tokens]; token t goes to block slot/block_size,
 *   offset slot%block_size; slot < 0 skips the token (padding).
 * k_scale, v_scale: fp32, [1] for KVQ_FP8_PER_TENSOR, [Hkv] for
 *   KVQ_FP8_PER_HEAD, ignored (may be NULL) otherwise.
 * k_cache, v_cache: the layer's code buffers (16-byte aligned).
 * k_cache_scale, v_cache_scale: the layer's scale buffers for the dynamic
 *   modes, ignored (may be NULL) otherwise.
 * Per element: y = x / s rounded to fp32, then E4M3 round-to-nearest-even
 * with saturation to +-448, or INT4 q = clamp(rint(y), -7, 7) packed two per
 * byte (even element in the low nibble).  Dynamic scales: s = amax/448 (FP8)
 * or amax/7 (INT4) in fp32, s = 1 when amax = 0 ([P1] "Dynamic per-token-head
 * scales add 3.125 percent"; [P2] "INT4 makes the metadata fraction larger").
 * A slot past the cache skips the token and sets KVQ_ERR_BAD_INDEX on the
 * device word. */
kvq_status kvq_cache_write(const kvq_ctx* ctx, int layer, const void* k_new, const void* v_new,
                           long long kv_token_stride, const long long* slot_mapping,
                           long long num_tokens, const float* k_scale, const float* v_scale,
                           void* k_cache, void* v_cache, float* k_cache_scale,
                           float* v_cache_scale, void* stream);

/* Static per-head calibration: scale_out[h] = amax over a bf16 sample
 * x [num_tokens][Hkv][D] of head h, divided by qmax (448 for E4M3) in fp32;
 * 1.0 for an all-zero head ([P1] "Calibration changes which scale layout
 * exists": an online maximum stands in for warm-up calibration).
 * scale_out: device fp32 [Hkv], overwritten. */
kvq_status kvq_calibrate_per_head(const kvq_ctx* ctx, const void* x, long long num_tokens,
                                  float qmax, float* scale_out, void* stream);

/* ------------------------------------------------------------- rotary positions
 * Pair i (0 <= i < rotary_dim / 2) of a head vector x at position p becomes
 *   x'[a] = m (x[a] cos(p f_i) - x[b] sin(p f_i))
 *   x'[b] = m (x[a] sin(p f_i) + x[b] cos(p f_i))
 * with (a, b) = (i, i + rotary_dim/2) (KVQ_ROPE_HALF) or (2i, 2i + 1)
 * (KVQ_ROPE_INTERLEAVED), and elements from rotary_dim on pass through.  The
 * pages have no counterpart; q and k reach kvq_cache_write and the attention
 * calls rotated, and these calls are how they get there. */
typedef enum kvq_rope_layout { KVQ_ROPE_HALF = 0, KVQ_ROPE_INTERLEAVED = 1 } kvq_rope_layout;

/* How the frequencies f_i = base^(-2i / rotary_dim) are scaled for contexts
 * longer than the model was trained on, s = factor:
 *  KVQ_ROPE_PLAIN   not at all
 *  KVQ_ROPE_LINEAR  f_i / s (positions interpolated)
 *  KVQ_ROPE_BASE    base replaced by base s^(r / (r - 2)), r = rotary_dim
 *  KVQ_ROPE_PARTS   by the turns n_i = original_context f_i / (2 pi) that pair
 *                   i makes over the original context: kept above
 *                   high_rotations, f_i / s below low_rotations, and
 *                   g f_i + (1 - g) f_i / s with g = (n_i - low) / (high - low)
 *                   between. */
typedef enum kvq_rope_scaling {
  KVQ_ROPE_PLAIN = 0,
  KVQ_ROPE_LINEAR = 1,
  KVQ_ROPE_BASE = 2,
  KVQ_ROPE_PARTS = 3
} kvq_rope_scaling;

typedef struct kvq_rope_config {
  int head_dim;               /* 64, 128 or 256 */
  int rotary_dim;             /* a multiple of 16, 16..head_dim */
  int layout;                 /* kvq_rope_layout */
  int scaling;                /* kvq_rope_scaling */
  double base;                /* > 0 */
  double factor;              /* > 0; read by the scaled kinds only */
  double original_context;    /* > 0; KVQ_ROPE_PARTS only */
  double low_rotations;       /* KVQ_ROPE_PARTS only, 0 <= low < high */
  double high_rotations;
  float magnitude;            /* m above, 1/16..16; 0 => 1 */
  const double* frequencies;  /* host [rotary_dim / 2], copied: the f_i themselves (scaling must
                                 be KVQ_ROPE_PLAIN, base is not read); NULL = from base */
} kvq_rope_config;

typedef struct kvq_rope kvq_rope;

/* Validates *cfg and computes the frequencies into a new handle.  Host only;
 * no CUDA call and no device memory.  KVQ_ERR_INVALID_ARG for a null pointer, a
 * value outside the ranges above or not finite, KVQ_ERR_UNSUPPORTED for a
 * head_dim or rotary_dim that is not built.  *out is NULL on error; the caller
 * releases a handle with kvq_rope_destroy.  A handle may be shared by threads. */
kvq_status kvq_rope_create(const kvq_rope_config* cfg, kvq_rope** out);
void kvq_rope_destroy(kvq_rope* rope);

/* The frequencies f_i after scaling (host double [rotary_dim / 2]) and m. */
kvq_status kvq_rope_frequencies(const kvq_rope* rope, double* frequencies, float* magnitude);

/* Rotation alone: out[t][h] = the rotation of x[t][h] at positions[t].
 * x, out: bf16 [num_tokens][num_heads][head_dim], token t starting at element
 *   t * its stride (0 => num_heads * head_dim); 16-byte aligned, strides
 *   multiples of 8 and at least num_heads * head_dim.  out may be x (with the
 *   same stride); otherwise they must not overlap.
 * positions: int64 [num_tokens], any value (negative ones included).
 * inverse: nonzero turns by -p f_i, still times m.  That is the transpose of the
 *   map, hence its gradient with respect to x, and for m = 1 its inverse.
 * Angles are taken modulo one turn in 64-bit fixed point from frequencies that
 * are doubles: an angle is off by |p| f_i 2^-52 radians at most (2e-10 at position
 * 10^6 and f = 1), and by 2^-24 of its distance from the nearest quarter turn.  The
 * rotation is computed in fp32 and rounded to bf16 once. */
kvq_status kvq_rope_apply(const kvq_rope* rope, const void* x, long long x_token_stride,
                          const long long* positions, long long num_tokens, int num_heads,
                          void* out, long long out_token_stride, int inverse, void* stream);

/* kvq_cache_write of rotated keys, with the queries rotated in the same launch.
 *
 * q, q_out: bf16 [num_tokens][Hq][D] with token strides as for kvq_rope_apply
 *   (0 => Hq*D); q_out gets the rotated queries of EVERY token (bf16, what the
 *   attention calls take) and may be q.  Both NULL: no queries.
 * k_new, v_new, kv_token_stride, slot_mapping, scales and caches as for
 *   kvq_cache_write.  k is rotated at positions[t] in fp32 and quantized from
 *   there, without the rounding to bf16 that a rotation followed by
 *   kvq_cache_write has in between (a BF16 layer rounds once, to the same bits);
 *   v is stored as kvq_cache_write stores it.  q, k and v may be parts of one
 *   fused buffer.  A token with slot < 0 has its q rotated and stores nothing.
 * Slots are distinct, as for kvq_cache_write (a slot given twice holds bytes of
 * both tokens). */
kvq_status kvq_rope_cache_write(const kvq_ctx* ctx, const kvq_rope* rope, int layer, const void* q,
                                long long q_token_stride, void* q_out,
                                long long q_out_token_stride, const void* k_new,
                                const void* v_new, long long kv_token_stride,
                                const long long* positions, const long long* slot_mapping,
                                long long num_tokens, const float* k_scale, const float* v_scale,
                                void* k_cache, void* v_cache, float* k_cache_scale,
                                float* v_cache_scale, void* stream);

/* ------------------------------------------------------------- pages of the pool
 * One pool of num_blocks blocks serves every layer of a context: a block id
 * names the same block in each layer's cache.  Its state is three device arrays
 * of the caller, which every call below reads and updates on the stream:
 *   ref_count     int32 [num_blocks]   table entries that hold the block; 0 = free
 *   block_table   int32 [table_rows][max_blocks_per_seq]   as the attention calls take it
 *   context_lens  int32 [table_rows]   positions of the row; ceil(len / block_size)
 *                                      entries of its table row are in use
 * An empty pool is ref_count 0, context_lens 0 and any table.  The calls keep
 *   ref_count[b] = the number of used table entries that hold b.
 * They need no workspace, allocate nothing, never synchronise and can be
 * captured into a graph; calls on one pool must be ordered by the caller (one
 * stream, or events).  Rows whose entries repeat a block (rings of window
 * layers) are not for these calls.
 *
 * A row index outside the table, a row that a call may name once and names
 * again, a length that is negative or past the row's entries, and a block id
 * outside the pool set KVQ_ERR_BAD_INDEX on the device word; that row (that
 * entry, for a block id) is left as it is and the others proceed.  num_rows or
 * num_forks = 0 is KVQ_OK and writes nothing. */

/* Takes num_rows rows and new_tokens[i] >= 0 further positions for row rows[i]
 * (distinct rows): hands out the blocks they need, lowest free ids first in the
 * order of the rows, and gives what the write and the prefill take.
 *   query_start   int32 [num_rows + 1]  prefix sums of new_tokens
 *   positions     int64 [max_tokens]    position of each new token
 *   slot_mapping  int64 [max_tokens]    its slot; -1 for a token of a refused row
 *   copies        int32 [num_rows][2]   see below
 * Entries from query_start[num_rows] to max_tokens are filled with position 0
 * and slot -1 (a padded batch).
 * A row whose last block is partly filled and held by another entry too gets a
 * block of its own for it: copies[i] = (shared block, new block), else (-1, -1).
 * That goes by the holders before the call: where all of them grow in one call,
 * each takes a block, and the shared one is free with its page still to be read.
 * kvq_copy_blocks(copies) therefore comes before anything is written AND before
 * the next call that changes the pool, which may hand out or rename these blocks.
 * A row gets all that it asks for or nothing.  When the rows up to and including
 * row i need more blocks than are free, row i is refused if it needs any
 * (KVQ_ERR_NO_BLOCKS on the device word); when they have more than max_tokens
 * tokens it is refused too (KVQ_ERR_BAD_INDEX).  A refused row keeps its length
 * and table, but its tokens are counted: query_start runs past max_tokens where
 * the tokens do, and an attention call with it then reads and writes rows that q
 * and out have only if they are made for the sum of new_tokens.
 * num_rows <= 4096; max_tokens < 2^31 - 1. */
kvq_status kvq_extend_sequences(const kvq_ctx* ctx, const int* rows, const int* new_tokens,
                                int num_rows, int* ref_count, int* block_table, int table_rows,
                                int max_blocks_per_seq, int* context_lens, long long max_tokens,
                                int* query_start, long long* positions, long long* slot_mapping,
                                int* copies, void* stream);

/* Row children[i] becomes a copy of row parents[i] that shares all its blocks
 * (no page is copied until one of them grows; see kvq_extend_sequences).
 * Children are distinct, empty rows (length 0); a parent may be named often, but
 * not as a child of the same call. */
kvq_status kvq_fork_sequences(const kvq_ctx* ctx, const int* parents, const int* children,
                              int num_forks, int* ref_count, int* block_table, int table_rows,
                              int max_blocks_per_seq, int* context_lens, void* stream);

/* Cuts row rows[i] (distinct rows) to its first min(length, keep_lens[i])
 * positions, or to none with keep_lens NULL: blocks past them lose a holder (and
 * are free when it was the last), their table entries become -1 (one that names
 * no block of the pool, too). */
kvq_status kvq_truncate_sequences(const kvq_ctx* ctx, const int* rows, const int* keep_lens,
                                  int num_rows, int* ref_count, int* block_table, int table_rows,
                                  int max_blocks_per_seq, int* context_lens, void* stream);

/* Renames blocks so that those in use become 0 .. n-1, n their number: block
 * ids >= n in use go to the free ids below n, both in ascending order.  Tables
 * and reference counts are rewritten.
 *   moves      int32 [num_blocks / 2][2]  (old, new) id of each block that moved
 *   num_moves  int32 [1]                  their number; later entries are not written
 * kvq_copy_blocks(moves, num_blocks / 2, num_moves) then moves the pages of
 * every layer, before they are read or written and before the next call that
 * changes the pool.  Copies that kvq_extend_sequences asked for come first. */
kvq_status kvq_compact_blocks(const kvq_ctx* ctx, int* ref_count, int* block_table,
                              int table_rows, int max_blocks_per_seq, int* context_lens,
                              int* moves, int* num_moves, void* stream);

/* Copies block pairs[i][0] to block pairs[i][1] in the caches of num_layers
 * layers from first_layer on: K and V codes and, for dynamic modes, scales.
 *   pairs      device int32 [max_pairs][2]; a negative source is skipped, an id
 *              outside the pool is skipped and sets KVQ_ERR_BAD_INDEX
 *   num_pairs  device int32 [1]: the first min(*num_pairs, max_pairs) pairs are
 *              copied; NULL = max_pairs
 *   k_caches, v_caches, k_cache_scales, v_cache_scales: HOST arrays [num_layers]
 *              of the layers' device buffers (16-byte aligned; read during the
 *              call); the scale arrays may be NULL when no layer is dynamic, and
 *              entries of other layers are not read
 * The pairs are copied at once: destinations are distinct and none is another
 * pair's source (the pairs that the calls above give are so). */
kvq_status kvq_copy_blocks(const kvq_ctx* ctx, int first_layer, int num_layers, const int* pairs,
                           int max_pairs, const int* num_pairs, void* const* k_caches,
                           void* const* v_caches, float* const* k_cache_scales,
                           float* const* v_cache_scales, void* stream);

/* Work plan for a decode call.  The retained positions of all (sequence, KV
 * head) items are cut into 16-position tiles and divided evenly among
 * `num_workers` worker warps (split-K over the context, balanced whatever the
 * context lengths); an item shared by several workers is merged by
 * log-sum-exp.  The pages fix no decode schedule; split-K with a
 * log-sum-exp merge is this library's way of spreading the retained
 * positions of few, long sequences ([P3] "Performance can favor the larger
 * cache": latency grows with every context token) over every SM.  On input *num_workers > 0 requests a count, 0 asks for the
 * plan's choice (fill every SM, from the batch, KV heads, the longest
 * context and the device); on output it holds the count and
 * *workspace_bytes what a call with that count needs (0 for one worker). */
kvq_status kvq_decode_plan(const kvq_ctx* ctx, int layer, int batch, int max_context,
                           int* num_workers, size_t* workspace_bytes);

/* Workspace bytes of a decode call with num_workers = 0 (the plan's choice):
 * kvq_decode_plan's *workspace_bytes for that count.  0 when one worker
 * suffices, and also when an argument is invalid (kvq_decode_plan reports
 * which). */
size_t kvq_decode_workspace_size(const kvq_ctx* ctx, int layer, int batch, int max_context);

/* Paged decode attention, one query token per sequence.
 *
 * Scales are folded, never applied element by element: the K scale (per
 * tensor, per KV head or per token and KV head, [P1] "Per-tensor vs per-head
 * FP8 KV cache scales", "Range sharing explains the accuracy trade")
 * multiplies the dot product of q with the raw codes, and the V scale the
 * softmax weight that meets the raw V codes.  Window layers read only their
 * last W positions, and KVQ_BF16 layers their native bf16 values ([P3] "FP8
 * KV cache layer skipping vs per-head scales", "Layer skipping follows
 * retained-token footprint").  Packed INT4 layers as [P2] "INT4 makes the
 * metadata fraction larger".
 *
 * q: bf16 [batch][Hq][D], 16-byte aligned.  Query head hq reads KV head
 *   hq / (Hq/Hkv).
 * block_table: int32 [batch][max_blocks_per_seq]; entries for positions that
 *   are not read may hold anything (e.g. -1).  Row b must cover context_lens[b]
 *   positions (context_lens[b] <= max_blocks_per_seq x block_size): a longer
 *   context is an index error -- only the covered positions are read and
 *   KVQ_ERR_BAD_INDEX is set on the device word.  Only positions [lo, L) are
 *   read, so a window layer may reuse its freed blocks as a ring: with
 *   R = ceil(W / block_size) + 1 physical blocks per sequence, logical block j
 *   may map to ring slot j mod R (the block a new position overwrites holds
 *   only positions outside the window).
 * context_lens: int32 [batch]; L counts the current token, whose K/V were
 *   written first.  The query attends to positions [lo, L), lo = max(0, L-W)
 *   for a window W, else 0.  L = 0 gives a zero output row.
 * out: fp32 [batch][Hq][D] = sum_p softmax(softmax_scale <q, K_hat[p]>) V_hat[p]
 *   with K_hat = code x K scale, V_hat = code x V scale.
 * max_context: an upper bound of context_lens, used only by the plan; more
 *   than max_blocks_per_seq x block_size returns KVQ_ERR_INVALID_ARG.
 * num_workers: worker warps (see kvq_decode_plan); 0 = the plan's choice.
 *   With more than one worker, partials go to `workspace` (16-byte aligned,
 *   kvq_decode_plan gives its size); its contents need no initialisation.
 * Scale pointers as for kvq_cache_write; dynamic scale buffers are 16-byte
 * aligned (they are fetched by bulk copies). */
kvq_status kvq_decode_attention(const kvq_ctx* ctx, int layer, const void* q,
                                const void* k_cache, const void* v_cache, const float* k_scale,
                                const float* v_scale, const float* k_cache_scale,
                                const float* v_cache_scale, const int* block_table,
                                int max_blocks_per_seq, const int* context_lens, int batch,
                                int max_context, float* out, int num_workers, void* workspace,
                                size_t workspace_bytes, void* stream);

/* kvq_decode_attention with an FP8 query.  Each query element x becomes the
 * E4M3 code of RN32(x / q_scale) (round to nearest even, saturating to
 * +-448, as kvq_cache_write encodes), and the scores use its value times
 * q_scale: out = sum_p softmax(softmax_scale <q_hat, K_hat[p]>) V_hat[p] with
 * q_hat = E4M3(q / q_scale) x q_scale.  This is the per-tensor FP8 path with
 * one scale each for Q, K and V, and the per-attention-head path with one Q
 * scale per query head ([P3] "FP8 KV cache layer skipping vs per-head
 * scales", opening section).
 * q_scale: device fp32, q_scale_count = 1 (one scale) or Hq (one per query
 *   head), each finite and > 0.  Other arguments, errors and workspace as for
 *   kvq_decode_attention; the output is fp32. */
kvq_status kvq_decode_attention_fp8_query(const kvq_ctx* ctx, int layer, const void* q,
                                          const float* q_scale, int q_scale_count,
                                          const void* k_cache, const void* v_cache,
                                          const float* k_scale, const float* v_scale,
                                          const float* k_cache_scale,
                                          const float* v_cache_scale, const int* block_table,
                                          int max_blocks_per_seq, const int* context_lens,
                                          int batch, int max_context, float* out,
                                          int num_workers, void* workspace,
                                          size_t workspace_bytes, void* stream);

/* kvq_decode_attention with a bf16 output: out is bf16 [batch][Hq][D]
 * (16-byte aligned), each element the round-to-nearest-even bf16 of the fp32
 * value kvq_decode_attention returns for the same arguments and num_workers.
 * The pages leave the attention output's dtype open; this variant returns
 * the model's native bf16 (the dtype [P3] "FP8 KV cache layer skipping vs
 * per-head scales" keeps for unquantized layers) and halves the output
 * traffic.  The arithmetic up to the final rounding is
 * kvq_decode_attention's.  Arguments, errors and workspace as for
 * kvq_decode_attention. */
kvq_status kvq_decode_attention_bf16(const kvq_ctx* ctx, int layer, const void* q,
                                     const void* k_cache, const void* v_cache,
                                     const float* k_scale, const float* v_scale,
                                     const float* k_cache_scale, const float* v_cache_scale,
                                     const int* block_table, int max_blocks_per_seq,
                                     const int* context_lens, int batch, int max_context,
                                     void* out, int num_workers, void* workspace,
                                     size_t workspace_bytes, void* stream);

/* Prefill (chunked multi-query) attention over the quantized paged cache:
 * the new tokens of each sequence attend causally to the cache, as at the
 * prefill stage whose time to first token the pages record ([P3] "FP8 KV
 * cache layer skipping vs per-head scales", section "Run a four-way
 * ablation").
 *
 * Sequence b has n_b = query_start[b+1] - query_start[b] new tokens at
 * positions [L_b - n_b, L_b), L_b = context_lens[b] >= n_b; their K/V were
 * written first (kvq_cache_write).  Query row query_start[b] + i of q (bf16
 * [T][Hq][D], T = query_start[batch], 16-byte aligned) sits at position
 * p = L_b - n_b + i and attends to positions [lo(p), p], lo(p) =
 * max(0, p + 1 - W) for a window W, else 0; out (fp32 [T][Hq][D]) is the
 * softmax(softmax_scale <q, K_hat>) weighted sum of V_hat over them, exactly
 * what kvq_decode_attention returns for that query with context p + 1.
 * query_start: int32 [batch + 1], query_start[0] = 0, non-decreasing.
 * max_query_len: an upper bound of every n_b (sizes the grid; rows past n_b
 *   do no work).
 * Scale pointers and block table as for kvq_decode_attention.  No workspace;
 * n_b > L_b, or L_b beyond the positions the sequence's block-table row
 * covers (max_blocks_per_seq x block_size), sets the BAD_INDEX bit of the
 * device error word and skips that sequence; a block id outside
 * [0, num_blocks) sets the same bit, nothing is read for that page, and its
 * positions are left out of the softmax (the output stays finite). */
kvq_status kvq_prefill_attention(const kvq_ctx* ctx, int layer, const void* q,
                                 const void* k_cache, const void* v_cache, const float* k_scale,
                                 const float* v_scale, const float* k_cache_scale,
                                 const float* v_cache_scale, const int* block_table,
                                 int max_blocks_per_seq, const int* query_start,
                                 const int* context_lens, int batch, int max_query_len,
                                 float* out, void* stream);

/* Cross attention: the queries of each sequence attend to ALL positions of an
 * encoder's states, which are in the paged cache (written by kvq_cache_write; a
 * cache of this kind is usually a context of its own, filled once per request
 * and shared by its beams through their table rows).  Without a mask and
 * without rotated positions, of another length than the queries:
 *   out[t] = sum_p softmax(softmax_scale <q[t], K_hat[p]>) V_hat[p],
 *   p in [0, encoder_lens[b]).
 * The pages have no counterpart; K_hat, V_hat and the scale layouts are those
 * of kvq_decode_attention.
 *
 * q: bf16 [T][Hq][D]; out: bf16 [T][Hq][D], both 16-byte aligned.
 * query_start: int32 [batch + 1] as for kvq_prefill_attention: sequence b has
 *   rows [query_start[b], query_start[b + 1]), none included.  NULL: one query
 *   per sequence, row b (a decoding step); max_query_len is then 0 or 1.
 * encoder_lens: int32 [batch].  0 gives zero rows.
 * max_query_len: an upper bound of the queries of a sequence; rows past it set
 *   KVQ_ERR_BAD_INDEX on the device word and are not computed.
 * max_encoder_len: an upper bound of encoder_lens, used by the plan only; more
 *   than the table rows cover is KVQ_ERR_INVALID_ARG.
 * num_splits, workspace: from kvq_cross_plan with the same sizes; num_splits 0
 *   = the plan's choice.  With query_start NULL and max_query_len 1 the call takes
 *   the worker warps that the plan of 0 chooses, and num_splits of them only where
 *   the workspace is smaller than theirs.  The workspace (16-byte aligned) needs no
 *   initialisation; overlapping calls need one each.
 * Softmax and sums are fp32.  What meets a V code is the softmax weight (relative
 * to the row's largest) times the V scale, rounded to f16: off by 2^-11 of itself, an
 * eighth of the output's own rounding, while it is above 2^-20 of the largest V
 * scale that the sequence has for the KV head, and by 2^-31 of that scale below
 * (a BF16 layer's scale: the power of two of a V row's largest value over 2^14).  A layer with a window is
 * KVQ_ERR_UNSUPPORTED.  A length that is negative or past the table row sets
 * KVQ_ERR_BAD_INDEX and leaves that sequence's rows as they were (with
 * query_start NULL: as kvq_decode_attention treats it); a block id outside the
 * cache sets it and leaves the page's positions out.  Scale pointers as for
 * kvq_decode_attention; dynamic scale buffers are 16-byte aligned. */
kvq_status kvq_cross_attention(const kvq_ctx* ctx, int layer, const void* q, const void* k_cache,
                               const void* v_cache, const float* k_scale, const float* v_scale,
                               const float* k_cache_scale, const float* v_cache_scale,
                               const int* block_table, int max_blocks_per_seq,
                               const int* query_start, const int* encoder_lens, int batch,
                               int max_query_len, int max_encoder_len, void* out, int num_splits,
                               void* workspace, size_t workspace_bytes, void* stream);

/* Splits of the keys and workspace bytes of a kvq_cross_attention call: on input
 * *num_splits > 0 (at most 1024) requests a count, 0 asks for the plan's choice
 * (one split when the queries fill the SMs; for few queries, as many as do).
 * max_query_len 0 plans the form with query_start NULL (*num_splits then counts
 * worker warps, as in kvq_decode_plan).  The workspace of max_query_len 1 serves
 * the call with query_start and the one without. */
kvq_status kvq_cross_plan(const kvq_ctx* ctx, int layer, int batch, int max_query_len,
                          int max_encoder_len, int* num_splits, size_t* workspace_bytes);

/* Decode attention that allocates nothing and needs no workspace from the
 * caller.  The pages have no counterpart to this call; it exists for callers
 * that cannot provide device scratch: code running where no device allocator
 * may be used (a serving loop that forbids allocations after start-up, a
 * plugin inside a host process that owns every device buffer) or bindings
 * that cannot manage device memory at all.
 *
 * Arguments and results are those of kvq_decode_attention without
 * `workspace`/`workspace_bytes`.  The split-K partials live instead in one
 * static device array of KVQ_FIXED_SCRATCH_BYTES (16 MiB) per GPU, held by
 * every GPU that loads the library until the process exits.  With
 * num_workers = 0 the plan's worker count is cut to the most workers whose
 * partials fit (at worst one worker, which needs no scratch).  An explicit
 * num_workers whose plan (kvq_decode_plan for the same batch, max_context
 * and num_workers) needs more than the array returns KVQ_ERR_WORKSPACE and
 * launches nothing; pass a smaller num_workers to fit.
 *
 * The first call on a device looks the array's address up on that device
 * (make that device current first; make the first call before any stream
 * capture).  Every call on a device shares the one array: calls whose GPU
 * work overlaps (different streams, concurrent host threads) race on it and
 * must be serialised by the caller.  The array keeps the last call's
 * contents; no call reads anything it did not write itself. */
#define KVQ_FIXED_SCRATCH_BYTES (16u * 1024u * 1024u)
kvq_status kvq_decode_attention_fixed_scratch(const kvq_ctx* ctx, int layer, const void* q,
                                              const void* k_cache, const void* v_cache,
                                              const float* k_scale, const float* v_scale,
                                              const float* k_cache_scale,
                                              const float* v_cache_scale, const int* block_table,
                                              int max_blocks_per_seq, const int* context_lens,
                                              int batch, int max_context, float* out,
                                              int num_workers, void* stream);

/* The device codec on its own: out[i] = E4M3 code of in[i] (RNE, saturating
 * to +-448), exactly as kvq_cache_write encodes y.  in: device fp32 [n],
 * out: device uint8 [n]. */
kvq_status kvq_e4m3_encode(const float* in, unsigned char* out, long long n, void* stream);

/* Synchronizes `stream`, returns the device error word of the current device
 * as a status (KVQ_OK, KVQ_ERR_BAD_INDEX, KVQ_ERR_TIMEOUT or
 * KVQ_ERR_NO_BLOCKS) and clears it. */
kvq_status kvq_get_device_error(void* stream);

/* Check of the timeout path (no counterpart on the pages).  Every wait of the
 * decode, prefill, cross and staged cache-write kernels on a shared-memory barrier
 * is bounded (about 2 s); a wait that runs out sets the TIMEOUT bit of the
 * device error word and the kernel stops instead of hanging the GPU.  This
 * call enqueues one warp that waits in the same way on a barrier that expects
 * bytes no copy ever delivers (no copy is issued, so nothing is in flight
 * when it gives up), with a limit of `limit_cycles` SM clock cycles
 * (0 < limit_cycles <= 2^31; 2,000,000 is about 1 ms).  Afterwards
 * kvq_get_device_error() returns KVQ_ERR_TIMEOUT and the context stays
 * usable.  Returns KVQ_ERR_INVALID_ARG for a limit outside the range. */
kvq_status kvq_check_bounded_wait(long long limit_cycles, void* stream);

const char* kvq_status_string(kvq_status s);

#ifdef __cplusplus
}
#endif
#endif /* KVQ_H_ */
