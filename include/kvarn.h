/*
 * kvarn.h -- C ABI of the GB300 (sm_103a) KVarN 2-bit KV-cache library
 * (3- and 4-bit codes as options of the same format).
 *
 * KVarN stores the K and V caches at 2 bits per element without calibration
 * data: each block of tokens is rotated by a randomised Hadamard matrix over
 * head_dim, normalised along the token axis and the channel axis in turn
 * until both have unit variance, and quantised in 32-channel groups; the
 * scales are kept and applied again when the cache is read. Decode attention
 * reads the packed cache directly, with the query rotated by the same matrix
 * and the inverse rotation applied once to the output.
 *
 * Sources (page title, section):
 *   "KVarN: cuantizacion de KV-Cache normalizada por varianza mitiga la
 *    acumulacion de errores en tareas de razonamiento" -- English abstract:
 *    Hadamard rotation then dual-scaling variance normalisation over both
 *    axes of K and V, calibration-free, 2-bit.
 *   "KVarN：方差归一化让 2-bit KV 缓存扛住长链推理" -- section 三, 3.1
 *    (randomised Hadamard on K and V; q multiplied by the same matrix so
 *    Q K^T is unchanged) and 3.2 (token-axis then channel-axis variance to 1,
 *    repeated 2-3 times; grouped scales kept for dequantisation; statistics
 *    computed at decode time and fusable into the KV write kernel).
 *
 * Conventions for every entry point
 *   - Pointers marked "device" must be device memory of the current CUDA
 *     device; "host" pointers are host memory. Nothing is allocated, freed or
 *     synchronised by the library except where stated (kvarn_read_error).
 *   - stream is a cudaStream_t passed as void* (NULL = legacy default
 *     stream). All device work is enqueued on it, in order.
 *   - The caller owns every buffer. Buffers written by a call must not be
 *     read or written by other work until that call's stream work completes.
 *   - Return value: KVARN_OK, or a negative kvarn_status when the arguments
 *     are rejected on the host (nothing enqueued) or a launch fails.
 *     Data-dependent faults found on the device (a block id outside the
 *     pool, a position beyond the block table, non-finite input, a wait that
 *     ran out of time) never trap: the kernel skips the affected unit and
 *     ORs a KVARN_DEVERR_* flag into the workspace error word, which
 *     kvarn_read_error returns. Outputs of a call that raised a flag are
 *     unspecified.
 *
 * Data layouts (little-endian; fp16/bf16 are IEEE binary16 / bfloat16)
 *   Head-block: one (physical block, kv head, K or V): B tokens x 128
 *   channels with `bits` (2, 3 or 4) bits per code, packed as (X = 16*bits*B)
 *     [0, X)             codes, in 8*bits-byte records (order below)
 *     [X, X+8B)          s: fp16 [4][B]   per (group, token) step
 *     [X+8B, X+16B)      z: fp16 [4][B]   per (group, token) zero (lowest level)
 *     [X+16B, X+18B)     R: fp16 [B]      per-token factor
 *     [X+18B, X+18B+256) C: fp16 [128]    per-channel factor
 *   = 1856 / 3456 bytes for 2 bits at B = 32 / 64, 2368 / 4480 for 3 bits,
 *   2880 / 5504 for 4 bits.
 *   The value of element (t, c) in the rotated space is
 *   (code * s[g][t] + z[g][t]) * R[t] * C[c] with g = c / 32 and code in
 *   0 .. 2^bits - 1. Code records: record r = 32*sb + 4a + b (sb = t / 32)
 *   holds 2*bits little-endian 32-bit words; a code sits at bit position p
 *   of word w of its record:
 *     kind K: a = (t%32)/4, i = t%4, g = c/32, b = (c%32)/8, e = c%8;
 *             2 bits: w = 2i + g/2, p = 2*(4*(g%2) + e/2) + 16*(e%2)
 *             4 bits: w = 4i + g,   p = 4*(e/2) + 16*(e%2)
 *     kind V: b = (t%32)/8, d = t%8, g = c/32, a = (c%32)/4, f = c%4;
 *             2 bits: w = 2g + f/2, p = 2*(4*(d/4) + 2*((d%4)/2) + f%2) + 16*(d%2)
 *             4 bits: w = 4g + f,   p = 4*(d/2) + 16*(d%2)
 *   3 bits: words 0..7 of a 12-word record hold each code's low two bits
 *           at its 2-bit (w, p); words 8..11 hold its high bit at word
 *           8 + w/2, bit 8*(w%2) + j + 16*h, where p = 2j + 16h
 *   (each lane of the attention kernel's warp reads exactly one record per
 *   32 tokens and turns it into tensor-core operands with one mask and one
 *   fp16 multiply per pair of codes).
 *   Pool: physical block p holds its head-blocks at
 *     pool + p*kvarn_block_bytes + (2*h + kind)*kvarn_head_block_bytes,
 *   kind 0 = K, 1 = V. pool must be 16-byte aligned.
 *   Staging (the incomplete tail block, raw unrotated values):
 *     bf16 [max_seqs][n_kv][2][B][128]; token t of sequence b is row t % B.
 *   Block table: int32 [batch][max_blocks_per_seq], logical -> physical.
 */
#ifndef KVARN_H_
#define KVARN_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    KVARN_OK = 0,
    KVARN_ERR_INVALID_ARG = -1,   /* null/misaligned pointer, bad size or config field */
    KVARN_ERR_UNSUPPORTED = -2,   /* a valid config this build does not implement */
    KVARN_ERR_CUDA = -3,          /* a CUDA runtime call or launch failed */
    KVARN_ERR_WORKSPACE = -4      /* workspace_bytes below kvarn_workspace_bytes */
} kvarn_status;

/* device error word flags (sticky, OR-ed) */
#define KVARN_DEVERR_BLOCK_ID 0x1u      /* physical block id < 0 or >= n_pool_blocks */
#define KVARN_DEVERR_POSITION 0x2u      /* pos / seq_len outside [0, max_blocks*B] */
#define KVARN_DEVERR_NONFINITE 0x4u     /* NaN or Inf in a block being quantised */
#define KVARN_DEVERR_WAIT_TIMEOUT 0x8u  /* a shared-memory copy wait hit its limit */

typedef enum { KVARN_BF16 = 0, KVARN_FP32 = 1 } kvarn_dtype;
typedef enum { KVARN_KIND_K = 0, KVARN_KIND_V = 1 } kvarn_kind;

typedef struct kvarn_config {
    int32_t head_dim;       /* must be 128 */
    int32_t block_size;     /* tokens per block B: 32 or 64 */
    int32_t group_size;     /* channels per quantisation group: must be 32 */
    int32_t bits;           /* bits per code: 2 (the method), 3 or 4 */
    int32_t varn_iters;     /* VarN iterations (token pass then channel pass): 0..8 */
    int32_t n_q_heads;      /* query heads */
    int32_t n_kv_heads;     /* kv heads; n_q_heads / n_kv_heads in 1..4 */
    float sm_scale;         /* softmax scale; 0 means 1/sqrt(head_dim) */
    uint32_t sign_bits[4];  /* rotation signs: bit c set => channel c negated */
    uint32_t flags;         /* 0 for the method; KVARN_FLAG_* bits select an ablation */
} kvarn_config;

/*
 * Ablation switches (section 五 of the method page, its ablation list: the
 * full method against Hadamard only, VarN only, and VarN along one axis).
 * They change what is stored, so a cache must be read with the flags it was
 * written with. Hadamard only = flags 0 with varn_iters 0.
 *   KVARN_FLAG_NO_ROTATION      no Hadamard rotation (R = I): keys, values and
 *                               queries stay in the original space and the
 *                               output is not rotated back
 *   KVARN_FLAG_NO_TOKEN_PASS    VarN without its token-axis pass (R_t = 1)
 *   KVARN_FLAG_NO_CHANNEL_PASS  VarN without its channel-axis pass (C_c = 1)
 */
#define KVARN_FLAG_NO_ROTATION 0x1u
#define KVARN_FLAG_NO_TOKEN_PASS 0x2u
#define KVARN_FLAG_NO_CHANNEL_PASS 0x4u
/*
 * Test switch (no counterpart in the paper): with it, every warp of
 * kvarn_decode_attn's split kernel, which kvarn_decode_attn_weights shares, and of the one that
 * kvarn_tree_attn has for few query rows gives up its first shared-memory copy wait
 * at once (and the tensor-core kernels of kvarn_prefix_attn, kvarn_tree_attn and
 * their bf16 forms act as if their first had), so the wait-timeout path runs without
 * anything hanging:
 * KVARN_DEVERR_WAIT_TIMEOUT is raised, the copies already in flight are
 * waited for, the warp stops, the call's outputs are unspecified and the
 * workspace stays usable (clear the error word and call again). Ignored by
 * the other entry points; never set it outside tests.
 */
#define KVARN_FLAG_TEST_WAIT_TIMEOUT 0x100u

/* Library version string, e.g. "kvarn 0.1 sm_103a". */
const char* kvarn_version(void);

/* Human-readable text for a kvarn_status value. */
const char* kvarn_status_string(int status);

/* Bytes of one packed head-block: (16*bits + 18)*B + 256 (50*B + 256 at 2
 * bits). 0 for an invalid config. */
size_t kvarn_head_block_bytes(const kvarn_config* cfg);

/* Bytes of one physical block: n_kv_heads * 2 * kvarn_head_block_bytes. */
size_t kvarn_block_bytes(const kvarn_config* cfg);

/* Bytes of the bf16 staging buffer for max_seqs sequences:
 * max_seqs * n_kv * 2 * B * 128 * 2. */
size_t kvarn_staging_bytes(const kvarn_config* cfg, int32_t max_seqs);

/* Minimum workspace for kvarn_decode_attn / kvarn_decode_attn_bf16 with this
 * batch on the CURRENT device (the split-K partial results depend on its SM
 * count): 256 header bytes (the error word is the first uint32), one
 * partial (max, sum, 128 accumulators per query head) per (sequence, kv
 * head) and per resident warp, then 8 bytes per (sequence, kv head) in
 * which the split kernel records the first and last warp of each for the
 * merge. batch = 0 gives the 256 bytes that kvarn_quantize_block and
 * kvarn_append need. 0 on a bad config. */
size_t kvarn_workspace_bytes(const kvarn_config* cfg, int32_t batch, int32_t max_blocks_per_seq);

/* Workspace with which kvarn_prefill_attn runs at full speed for this batch
 * and chunk on the CURRENT device: at least kvarn_workspace_bytes(cfg,
 * batch * chunk, ...), and room for several partials per row when there are
 * too few (sequence, kv head, row tile) units to fill the GPU (2-bit caches;
 * the block split adapts to the workspace actually passed). 0 on a bad
 * config. */
size_t kvarn_prefill_workspace_bytes(const kvarn_config* cfg, int32_t batch, int32_t chunk,
                                     int32_t max_blocks_per_seq);

/*
 * kvarn_quantize_block -- bulk quantise-on-write of complete head-blocks
 * (prefill). Passage: abstract (rotation then dual-axis normalisation, 2-bit);
 * section 三 3.1-3.2 of the method page.
 *
 * For each n in [0, n_head_blocks): reads the B x 128 block
 *   src[n*src_block_stride + t*src_token_stride + c]  (elements, dtype
 *   src_dtype: KVARN_BF16 or KVARN_FP32; device)
 * rotates each token by H diag(sigma)/sqrt(128), runs varn_iters passes of
 * token-axis then channel-axis variance normalisation, rounds the factors to
 * fp16, quantises each (token, 32-channel group) to `bits` bits
 * (2^bits - 1 steps) with an fp16 step and zero, and writes one packed head-block of `kind` layout to
 *   dst_base + dst_offsets[n]   (bytes; device int64 array, NULL means
 *                               n * kvarn_head_block_bytes)
 * dst_base + offset must be 16-byte aligned. workspace: >= 256 bytes of
 * device memory whose first uint32 is the error word (KVARN_DEVERR_NONFINITE).
 */
int kvarn_quantize_block(const kvarn_config* cfg, int32_t kind, const void* src, int32_t src_dtype,
                         int64_t n_head_blocks, int64_t src_block_stride,
                         int64_t src_token_stride, void* dst_base, const int64_t* dst_offsets,
                         void* workspace, void* stream);

/*
 * kvarn_append -- one decode step's KV write (quantise-on-append). Passage:
 * section 三 3.2 of the method page (scales computed at decode time from the
 * data itself, fused into the KV write kernel).
 *
 * For each sequence b < batch and kv head h, the new token's K and V
 * (k_new, v_new: device bf16 [batch][n_kv][128]) are written to staging row
 * pos[b] % B (pos: device int32 [batch], the index of the new token, i.e.
 * the length before this step). When that row completes the block
 * (pos[b] % B == B - 1), the whole block is quantised exactly as
 * kvarn_quantize_block does and written to physical block
 * block_table[b][pos[b] / B] of the pool (n_pool_blocks blocks); the staging
 * rows are left as they are. Nothing is re-quantised later. Device faults:
 * KVARN_DEVERR_POSITION (pos < 0 or pos >= max_blocks_per_seq * B),
 * KVARN_DEVERR_BLOCK_ID, KVARN_DEVERR_NONFINITE.
 */
int kvarn_append(const kvarn_config* cfg, void* pool, int64_t n_pool_blocks, void* staging,
                 const int32_t* block_table, int32_t max_blocks_per_seq, const int32_t* pos,
                 const void* k_new, const void* v_new, int32_t batch, void* workspace,
                 void* stream);

/*
 * Rotary positions for kvarn_append_rope and kvarn_append_rope_bf16 (library
 * conveniences, like the head norms: the method's pages start from keys that
 * a model has rotated already). Filled by kvarn_rope_init; plain host data.
 *   KVARN_ROPE_HALF         channels i and i + rotary_dim / 2 are pair i
 *   KVARN_ROPE_INTERLEAVED  channels 2i and 2i + 1 are pair i
 */
typedef enum { KVARN_ROPE_HALF = 0, KVARN_ROPE_INTERLEAVED = 1 } kvarn_rope_layout;

typedef struct kvarn_rope {
    int32_t rotary_dim;   /* channels rotated, from channel 0: a multiple of 16, 0..128; the others pass */
    int32_t layout;       /* kvarn_rope_layout */
    float scale;          /* multiplies cos and sin (attention factor of some long-context scalings), else 1 */
    float eps;            /* epsilon of the head norms */
    uint64_t turns[64];   /* pair i's turns per position, fraction of one, in units of 2^-64 */
} kvarn_rope;

/* Fills *rope (host) from the angular rates inv_freq[rotary_dim / 2] (host,
 * radians per position, |rate| <= 2^20; however scaled for long contexts).
 * KVARN_ERR_UNSUPPORTED for a rotary_dim that is no multiple of 16. */
int kvarn_rope_init(kvarn_rope* rope, int32_t rotary_dim, int32_t layout, const double* inv_freq, float scale,
                    float eps);

/*
 * kvarn_append_rope -- keys and values of one step appended to the packed
 * cache with head norms and rotary positions on the way, and the step's
 * queries normed and rotated in the same launch: one token per sequence
 * (decode) or a ragged run of tokens per sequence (prompts).
 *
 * Token rows: q [n_tokens][n_q][128], k and v [n_tokens][n_kv][128], device
 * bf16, rows of one token contiguous, q_stride / k_stride / v_stride elements
 * (multiples of 8) from one token to the next, so columns of one projection's
 * output serve as they are. With cu_tokens (device int32 [batch + 1],
 * ascending from 0 or more) rows cu_tokens[b] .. cu_tokens[b+1] - 1 are
 * sequence b's; a sequence may have none, and rows outside every sequence are
 * left alone, with their q_out. Without it (NULL) n_tokens is batch and row b
 * is sequence b's one token.
 *
 * Row i of sequence b is its token pos[b] + i (pos: device int32 [batch],
 * tokens cached before), turned by the angles of position
 * (rope_pos ? rope_pos[b] : pos[b]) + i (rope_pos: device int32 [batch], for a
 * cache that does not start at position 0, such as the own tokens behind a
 * shared prefix):
 *   q_out = rope(norm(q)), key = rope(norm(k)), value = v,
 *   norm(x) = x w / sqrt(mean(x^2) + eps) with q_weight / k_weight (device
 *   bf16 [128]; NULL: no norm).
 * q_out: [n_tokens][n_q][128], q_out_dtype KVARN_BF16 or KVARN_FP32; it may
 * be q itself where q's rows are laid out like it. q and q_out may both be
 * NULL. The key is rounded to bf16.
 *
 * Tokens of complete blocks are quantised as kvarn_quantize_block does, from
 * the staging rows of earlier tokens and the new rows, and written to the
 * pool; tokens of the incomplete block go to their staging rows (other staging
 * rows are left as they are): the pool then holds the bytes that kvarn_append
 * would have written token by token. Device faults: KVARN_DEVERR_POSITION
 * (pos < 0, a token beyond the block table, cu_tokens not ascending or beyond
 * n_tokens: nothing of that sequence is written, its q_out rows neither),
 * KVARN_DEVERR_BLOCK_ID, KVARN_DEVERR_NONFINITE.
 */
int kvarn_append_rope(const kvarn_config* cfg, const kvarn_rope* rope, void* pool, int64_t n_pool_blocks,
                      void* staging, const int32_t* block_table, int32_t max_blocks_per_seq, const int32_t* pos,
                      const int32_t* rope_pos, const int32_t* cu_tokens, int64_t n_tokens, int32_t batch,
                      const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride,
                      int64_t v_stride, const void* q_weight, const void* k_weight, void* q_out,
                      int32_t q_out_dtype, void* workspace, void* stream);

/*
 * kvarn_append_rope_bf16 -- the same into the plain bf16 pages of
 * kvarn_decode_attn_bf16 (kv_pool: bf16 [n_pool_blocks][n_kv][2][B][128]):
 * every token goes to its row of its page. Device faults as there, without
 * KVARN_DEVERR_NONFINITE. workspace: >= 256 bytes, for the error word.
 */
int kvarn_append_rope_bf16(const kvarn_config* cfg, const kvarn_rope* rope, void* kv_pool, int64_t n_pool_blocks,
                           const int32_t* block_table, int32_t max_blocks_per_seq, const int32_t* pos,
                           const int32_t* rope_pos, const int32_t* cu_tokens, int64_t n_tokens, int32_t batch,
                           const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride,
                           int64_t v_stride, const void* q_weight, const void* k_weight, void* q_out,
                           int32_t q_out_dtype, void* workspace, void* stream);

/*
 * kvarn_decode_attn -- decode attention over the packed cache. Passage:
 * section 三 3.1 of the method page (the query is multiplied by the same
 * Hadamard matrix, so q.k is unchanged).
 *
 * q: device [batch][n_q][128], dtype q_dtype (KVARN_BF16 or KVARN_FP32).
 * seq_lens: device int32 [batch], tokens per sequence including the newest.
 * For query head j of sequence b (kv head h = j / (n_q / n_kv)):
 *   out[b][j][:] = sum_t softmax_t(sm_scale * q.k_t) v_t
 * over the first floor(L/B)*B tokens from the pool (dequantised on the fly)
 * and the remaining L % B tokens from staging (raw bf16). out: device fp32
 * [batch][n_q][128]. L = 0 gives zeros. workspace: device, at least
 * kvarn_workspace_bytes(cfg, batch, max_blocks_per_seq) bytes, 16-byte
 * aligned, passed as workspace_bytes. The work is split evenly over the
 * GPU's resident warps (split-K over each sequence's blocks) and merged by a
 * second kernel on the same stream. n_pool_blocks must be below 2^31
 * (KVARN_ERR_INVALID_ARG otherwise). Device faults: KVARN_DEVERR_BLOCK_ID,
 * KVARN_DEVERR_POSITION, KVARN_DEVERR_WAIT_TIMEOUT.
 */
int kvarn_decode_attn(const kvarn_config* cfg, const void* q, int32_t q_dtype, const void* pool,
                      int64_t n_pool_blocks, const void* staging, const int32_t* block_table,
                      int32_t max_blocks_per_seq, const int32_t* seq_lens, int32_t batch,
                      float* out, void* workspace, size_t workspace_bytes, void* stream);

/*
 * kvarn_prefill_attn -- chunked prefill attention over the same packed cache
 * (the pages describe only the decode step; this is its causal extension,
 * with the query multiplied by the same Hadamard matrix, section 三 3.1).
 *
 * The last `chunk` tokens of every sequence have already been appended
 * (kvarn_append / kvarn_quantize_block); q: device [batch][chunk][n_q][128]
 * (q_dtype KVARN_BF16 or KVARN_FP32) holds their queries. Query row r of
 * sequence b sits at position p = seq_lens[b] - chunk + r and, for query
 * head j (kv head j / (n_q / n_kv)),
 *   out[b][r][j][:] = sum_{t <= p} softmax_t(sm_scale * q.k_t) v_t
 * with every token read from the cache as it stands: tokens below
 * floor(L/B)*B dequantised from the pool, the rest raw bf16 from staging. A
 * row with p < 0 (seq_lens[b] < chunk) gives zeros. out: device fp32
 * [batch][chunk][n_q][128]. chunk >= 1; chunk = 1 is kvarn_decode_attn.
 * workspace: at least kvarn_workspace_bytes(cfg, batch * chunk,
 * max_blocks_per_seq) bytes; kvarn_prefill_workspace_bytes gives the size
 * with which short chunks split each sequence's blocks over enough warps.
 * One warp scores 8 query vectors (8 / G rows x G heads) against each
 * block, building each code's tensor-core operand once for all 8. Device
 * faults as kvarn_decode_attn.
 */
int kvarn_prefill_attn(const kvarn_config* cfg, const void* q, int32_t q_dtype, const void* pool,
                       int64_t n_pool_blocks, const void* staging, const int32_t* block_table,
                       int32_t max_blocks_per_seq, const int32_t* seq_lens, int32_t batch, int32_t chunk,
                       float* out, void* workspace, size_t workspace_bytes, void* stream);

/*
 * kvarn_dequantize -- packed head-blocks back to fp32 values. Passage:
 * section 三 3.2 of the method page (the kept scales restore the data).
 * Reads n_head_blocks head-blocks of `kind` layout at src_base +
 * src_offsets[n] (device int64 bytes; NULL = contiguous) and writes out
 * (device fp32 [n][B][128]): rotated != 0 gives the rotated-space values
 * (code*s + z)*R*C; rotated == 0 also applies the inverse rotation.
 */
int kvarn_dequantize(const kvarn_config* cfg, int32_t kind, const void* src_base,
                     const int64_t* src_offsets, int64_t n_head_blocks, int32_t rotated,
                     float* out, void* stream);

/*
 * kvarn_error_decomposition -- the magnitude / direction split of each
 * token's quantisation error. Passage: section 二 of the method page: with
 * x^ = x + eps, eps = E_M + E_D, E_M = (|x^| - |x|) x/|x| (length error) and
 * E_D = |x^| (x^/|x^| - x/|x|) (direction error).
 * src: the values before quantisation, laid out as for kvarn_quantize_block
 * (n_head_blocks blocks of B rows, strides in elements, dtype src_dtype);
 * packed_base + packed_offsets[n] (device int64 bytes; NULL = contiguous):
 * the head-blocks of `kind` layout written from them with the same cfg.
 * out: device fp32 [n][B][4] = (|x|, |x^|, |E_M|, |E_D|) per token. A zero
 * token (direction undefined) reports all of its error as |E_M|. Read-only
 * on its inputs; no error word.
 */
int kvarn_error_decomposition(const kvarn_config* cfg, int32_t kind, const void* src, int32_t src_dtype,
                              int64_t n_head_blocks, int64_t src_block_stride, int64_t src_token_stride,
                              const void* packed_base, const int64_t* packed_offsets, float* out,
                              void* stream);

/*
 * kvarn_decode_attn_bf16 -- the same decode attention over a plain bf16
 * paged cache (the comparison point for the 2-bit path; no rotation, no
 * staging). kv_pool: device bf16 [n_pool_blocks][n_kv][2][B][128]; every
 * token of a sequence, the last block partly filled, is in the pool.
 * Other arguments as kvarn_decode_attn.
 */
int kvarn_decode_attn_bf16(const kvarn_config* cfg, const void* q, int32_t q_dtype,
                           const void* kv_pool, int64_t n_pool_blocks,
                           const int32_t* block_table, int32_t max_blocks_per_seq,
                           const int32_t* seq_lens, int32_t batch, float* out, void* workspace,
                           size_t workspace_bytes, void* stream);

/* Workspace bytes for kvarn_prefix_attn / kvarn_prefix_attn_bf16 with this
 * batch and prefix_blocks on the CURRENT device: the decode workspace for the
 * own tokens, then one partial per (token range of the prefix, sequence,
 * query head). It serves shorter prefixes of the same batch too. 0 on a bad
 * config. */
size_t kvarn_prefix_workspace_bytes(const kvarn_config* cfg, int32_t batch, int32_t prefix_blocks);

/*
 * kvarn_prefix_attn -- decode attention over the packed cache for a batch
 * whose sequences share a prefix (a system prompt, one document, several
 * samples of one prompt), read once for all of them. (A serving convenience;
 * the query is multiplied by the same Hadamard matrix, section 三 3.1.)
 *
 * The prefix's blocks are prefix_table (device int32 [prefix_blocks], at most
 * 2^30 tokens), every one complete in the pool; sequence b sees its first prefix_lens[b] tokens
 * (device int32 [batch], 0 .. prefix_blocks * B: any count, the same for all
 * or not). Its own tokens follow: block_table, seq_lens and staging as for
 * kvarn_decode_attn, their indices starting at 0.
 *   out[b][j][:] = sum_t softmax_t(sm_scale * q.k_t) v_t
 * over the prefix's tokens and the own ones together; no token at all gives
 * zeros, and a query that is not finite NaN (the other rows keep theirs). out: device [batch][n_q][128], out_dtype KVARN_BF16 or KVARN_FP32.
 * workspace: at least kvarn_prefix_workspace_bytes(cfg, batch, prefix_blocks)
 * bytes, 16-byte aligned; calls that may overlap need one each. A prefix block
 * quantised from values that were not finite (flagged when it was written)
 * makes the outputs of every sequence with a prefix undefined.
 * Device faults: KVARN_DEVERR_BLOCK_ID, KVARN_DEVERR_POSITION (a length outside
 * its range), KVARN_DEVERR_WAIT_TIMEOUT.
 */
int kvarn_prefix_attn(const kvarn_config* cfg, const void* q, int32_t q_dtype, const void* pool,
                      int64_t n_pool_blocks, const void* staging, const int32_t* prefix_table,
                      int32_t prefix_blocks, const int32_t* prefix_lens, const int32_t* block_table,
                      int32_t max_blocks_per_seq, const int32_t* seq_lens, int32_t batch, void* out,
                      int32_t out_dtype, void* workspace, size_t workspace_bytes, void* stream);

/*
 * kvarn_prefix_attn_bf16 -- the same over the bf16 pages of
 * kvarn_decode_attn_bf16; the last page of the prefix may be partly filled,
 * and its rows behind the longest prefix_lens may hold anything. The values
 * before that must be finite even for sequences that do not see them (their
 * weight of 0 takes part in the product). Softmax weights and an fp32 query
 * enter the products as two bf16 halves, within 2^-16, as in
 * kvarn_decode_attn_bf16. In kvarn_prefix_attn queries, keys, weights and values
 * of blocks enter them as two fp16 halves, within 2^-22 (the prefix's keys and
 * values below 2^-18 of the largest of their 64 tokens: within 2^-39 of that one; its
 * weights below 2^-10 of the row's largest: within 2^-32 of that one), and weights and
 * fp32 queries of the raw rows as two bf16 halves.
 */
int kvarn_prefix_attn_bf16(const kvarn_config* cfg, const void* q, int32_t q_dtype, const void* kv_pool,
                           int64_t n_pool_blocks, const int32_t* prefix_table, int32_t prefix_blocks,
                           const int32_t* prefix_lens, const int32_t* block_table, int32_t max_blocks_per_seq,
                           const int32_t* seq_lens, int32_t batch, void* out, int32_t out_dtype, void* workspace,
                           size_t workspace_bytes, void* stream);

/* Workspace bytes for kvarn_tree_attn / kvarn_tree_attn_bf16 with this batch,
 * number of drafts and table width on the CURRENT device. It grows with each of the
 * three: a workspace for the largest call serves them all. 0 on a bad config or size. */
size_t kvarn_tree_workspace_bytes(const kvarn_config* cfg, int32_t batch, int32_t drafts,
                                  int32_t max_blocks_per_seq);

/*
 * kvarn_tree_attn -- attention for a tree of drafted tokens over the packed
 * cache (verification of several guessed continuations in one pass). (A serving
 * convenience; the query is multiplied by the same Hadamard matrix, section 三 3.1.)
 *
 * Every sequence has `drafts` rows (1 .. KVARN_MAX_DRAFTS): q [batch][drafts]
 * [n_q][128] (q_dtype KVARN_BF16 or KVARN_FP32), and k, v [batch][drafts][n_kv]
 * [128] (bf16, the heads of a token contiguous, k_stride / v_stride elements, a
 * multiple of 8, from one token to the next, the sequences one after the
 * other: columns of one projection's output serve as they are). The drafted
 * tokens are not in the cache; those that are accepted can be appended later.
 * draft_lens (device int32 [batch], 0 .. drafts; NULL: all of them): the rows
 * from draft_lens[b] on are padding, whose inputs are not looked at and whose
 * outputs are left as they were.
 *
 * Row r of sequence b sees every cached token (seq_lens[b], as for
 * kvarn_decode_attn) and the drafted tokens i < draft_lens[b] for which bit i % 32
 * of mask[b][r][i / 32] is set (device uint32 [batch][drafts][(drafts + 31) / 32]):
 * its ancestors in the tree and itself, or any other set.
 *   out[b][r][j] = sum_t softmax_t(sm_scale * q.k_t) v_t
 * over those; a row that sees nothing gives zeros, one with a score that is not a
 * number NaN. out: device [batch][drafts][n_q][128], out_dtype KVARN_BF16 or
 * KVARN_FP32. A drafted value that is not finite makes the rows that see it NaN,
 * and no other row. fp32 queries (of bf16 pages and raw rows) and softmax weights
 * enter the products as two 16-bit halves, within 2^-16; over the packed cache
 * rotated queries and weights within 2^-22. With more than a few query rows weights
 * there are, below 2^-14 of the row's largest, within 2^-36 of that one, and keys and
 * values within 2^-18 (4 bits) to 2^-20 (2 bits) of the largest level of their token's
 * 32 channels or, where that is more, 2^-29 of the largest level of their 64 tokens.
 * Sums over tokens are the tensor core's, which cuts the fp32 sum at each step and drops
 * what is below 2^-25 of it: beside a large weight whose value is not small, weights
 * below 2^-25 of it may be missing from out.
 * workspace: at least kvarn_tree_workspace_bytes(cfg, batch, drafts, max_blocks_per_seq)
 * bytes, 16-byte aligned; calls that may overlap need one each. Device faults:
 * KVARN_DEVERR_BLOCK_ID, KVARN_DEVERR_POSITION (a length outside its range: NaN rows),
 * KVARN_DEVERR_WAIT_TIMEOUT.
 */
#define KVARN_MAX_DRAFTS 128
int kvarn_tree_attn(const kvarn_config* cfg, const void* q, int32_t q_dtype, const void* pool,
                    int64_t n_pool_blocks, const void* staging, const int32_t* block_table,
                    int32_t max_blocks_per_seq, const int32_t* seq_lens, const void* k, const void* v,
                    int64_t k_stride, int64_t v_stride, const uint32_t* mask, const int32_t* draft_lens,
                    int32_t batch, int32_t drafts, void* out, int32_t out_dtype, void* workspace,
                    size_t workspace_bytes, void* stream);

/* kvarn_tree_attn_bf16 -- the same over the bf16 pages of kvarn_decode_attn_bf16. */
int kvarn_tree_attn_bf16(const kvarn_config* cfg, const void* q, int32_t q_dtype, const void* kv_pool,
                         int64_t n_pool_blocks, const int32_t* block_table, int32_t max_blocks_per_seq,
                         const int32_t* seq_lens, const void* k, const void* v, int64_t k_stride,
                         int64_t v_stride, const uint32_t* mask, const int32_t* draft_lens, int32_t batch,
                         int32_t drafts, void* out, int32_t out_dtype, void* workspace,
                         size_t workspace_bytes, void* stream);

/* Workspace bytes for kvarn_decode_attn_weights / kvarn_decode_attn_weights_bf16
 * on the CURRENT device: kvarn_workspace_bytes, a maximum and a sum per query
 * head and the scores of a full block table. 0 on a bad config or size. */
size_t kvarn_weights_workspace_bytes(const kvarn_config* cfg, int32_t batch, int32_t max_blocks_per_seq);

/*
 * kvarn_decode_attn_weights -- kvarn_decode_attn that also keeps how much
 * attention each cached token gets. (A library convenience: what eviction
 * from a cache goes by.)
 *
 * Beside out (device [batch][n_q][128], out_dtype KVARN_BF16 or KVARN_FP32; the fp32
 * values are those of kvarn_decode_attn), for every token t < seq_lens[b] and kv head h,
 *   weights_out[b][h][t] = decay * weights_in[b][h][t]
 *                          + sum over the query heads j of h of softmax_t(sm_scale * q_j.k_t)
 * weights_in, weights_out: device fp32 [batch][n_kv][weights_stride], 16-byte
 * aligned, weights_stride a multiple of 4 and at least max_blocks_per_seq * B;
 * weights_out behind a sequence's end is left as it was. They may be the same
 * buffer (weights kept from step to step) or two that do not overlap.
 * weights_in NULL or decay 0: this step's weights alone. decay in 0 .. 1.
 * workspace: at least kvarn_weights_workspace_bytes bytes, 16-byte aligned.
 * Device faults as kvarn_decode_attn; a sequence with one has its weights unspecified, and so
 * has a kv head with a score that is not finite (its out is NaN, or counts finite scores alone).
 */
int kvarn_decode_attn_weights(const kvarn_config* cfg, const void* q, int32_t q_dtype, const void* pool,
                              int64_t n_pool_blocks, const void* staging, const int32_t* block_table,
                              int32_t max_blocks_per_seq, const int32_t* seq_lens, int32_t batch, void* out,
                              int32_t out_dtype, const float* weights_in, float* weights_out,
                              int64_t weights_stride, float decay, void* workspace, size_t workspace_bytes,
                              void* stream);

/* kvarn_decode_attn_weights_bf16 -- the same over the bf16 pages of kvarn_decode_attn_bf16. */
int kvarn_decode_attn_weights_bf16(const kvarn_config* cfg, const void* q, int32_t q_dtype, const void* kv_pool,
                                   int64_t n_pool_blocks, const int32_t* block_table,
                                   int32_t max_blocks_per_seq, const int32_t* seq_lens, int32_t batch, void* out,
                                   int32_t out_dtype, const float* weights_in, float* weights_out,
                                   int64_t weights_stride, float decay, void* workspace, size_t workspace_bytes,
                                   void* stream);

/*
 * kvarn_evict_bf16 -- cuts the sequences of a bf16 paged cache down to a budget
 * of tokens, by the weights that kvarn_decode_attn_weights_bf16 keeps. (A library
 * convenience; keys are rotated already, so that attention does not ask for a
 * token's place.)
 *
 * For every (sequence b, kv head h) with L = seq_lens[b] tokens (device int32 [batch]):
 * L <= budget keeps all; otherwise the last `recent` tokens stay (0 .. budget), and of
 * the others the budget - recent with the greatest weights[b][h][t] (device fp32
 * [batch][n_kv][weights_stride], 16-byte aligned, the stride a multiple of 4; not
 * negative; what is not a number counts as 0; ties go to the lowest t). Each kv head keeps its own. What is kept goes, in
 * order, to the pages new_table (device int32 [batch][new_max_blocks]), which must not be
 * among those that the call reads; old pages are only read, so that they may be shared
 * with other sequences, and are free afterwards.
 *   new_lens[b]           min(L, budget)  (device int32 [batch], not seq_lens itself)
 *   kept[b][h][i]         the token now at place i, -1 from the new length on
 *                         (device int32 [batch][n_kv][budget])
 *   new_weights[b][h][i]  its weight, 0 from the new length on (device fp32 [batch][n_kv]
 *                         [new_weights_stride], the first new_max_blocks * B columns
 *                         written; must not overlap weights)
 * Rows of the new pages behind the new length are left as they were.
 * After an eviction a token's place in the cache is no longer its position in the
 * text: the caller keeps the positions, and appends with pos = new_lens and
 * rope_pos = the position of the first new token (kvarn_append_rope_bf16, kvarn_append_rope;
 * without rope_pos new keys and queries would be turned as if they stood before kept
 * ones). Drafted keys and queries are turned by the caller likewise.
 * budget >= 1, new_max_blocks * B >= budget. workspace: >= 256 bytes, for the error
 * word. Device faults: KVARN_DEVERR_BLOCK_ID (the row or block is not moved),
 * KVARN_DEVERR_POSITION (a length beyond the block table: new length 0, nothing moved).
 */
int kvarn_evict_bf16(const kvarn_config* cfg, void* kv_pool, int64_t n_pool_blocks, const int32_t* block_table,
                     int32_t max_blocks_per_seq, const int32_t* seq_lens, const float* weights,
                     int64_t weights_stride, int32_t budget, int32_t recent, const int32_t* new_table,
                     int32_t new_max_blocks, int32_t* new_lens, float* new_weights, int64_t new_weights_stride,
                     int32_t* kept, int32_t batch, void* workspace, void* stream);

/*
 * kvarn_evict -- the same over the packed cache, by whole blocks, whose codes
 * share their factors: budget and recent are multiples of B, a block's weight is
 * the sum of its tokens' (in 64 bits, rounded to fp32), and kept [batch][n_kv][budget / B] names
 * blocks. The L % B tokens of the incomplete block stay where they are in staging, behind
 * the kept blocks: new_lens[b] = min(L - L % B, budget) + L % B, their weights
 * move along, and new_max_blocks * B > budget. rope_pos as there.
 */
int kvarn_evict(const kvarn_config* cfg, void* pool, int64_t n_pool_blocks, const int32_t* block_table,
                int32_t max_blocks_per_seq, const int32_t* seq_lens, const float* weights, int64_t weights_stride,
                int32_t budget, int32_t recent, const int32_t* new_table, int32_t new_max_blocks,
                int32_t* new_lens, float* new_weights, int64_t new_weights_stride, int32_t* kept, int32_t batch,
                void* workspace, void* stream);

/*
 * kvarn_decode_attn_noalloc -- kvarn_decode_attn for callers that cannot
 * allocate device memory. (The paper has no counterpart; this is a library
 * convenience.) Some callers can only hand over their inputs and outputs: a
 * plug-in interface with no workspace argument, a runtime whose memory
 * planner owns all device memory, or a loop that must not call cudaMalloc
 * because allocation can synchronise the device. This entry point allocates
 * nothing: its split-K scratch is a 16 MiB array compiled into the library
 * (held on every GPU that loads the library until the process exits).
 *
 * Arguments and results are those of kvarn_decode_attn, without the
 * workspace. error_word (device uint32, may be NULL) receives this call's
 * KVARN_DEVERR_* flags (0 when none). The scratch must hold
 * kvarn_workspace_bytes(cfg, batch, max_blocks_per_seq) bytes (256 + (batch *
 * n_kv + resident warps) * G * 528 + batch * n_kv * 8); larger problems are refused with
 * KVARN_ERR_WORKSPACE before anything is enqueued.
 *
 * The first call on each device looks up the array's device address (with
 * that device current) and caches it; make that first call before any stream
 * capture. Every call shares the one array: calls whose GPU work overlaps
 * (other streams, other host threads) race on it and must be serialised by
 * the caller. Each call clears the error word it uses before its kernels run.
 */
int kvarn_decode_attn_noalloc(const kvarn_config* cfg, const void* q, int32_t q_dtype,
                              const void* pool, int64_t n_pool_blocks, const void* staging,
                              const int32_t* block_table, int32_t max_blocks_per_seq,
                              const int32_t* seq_lens, int32_t batch, float* out,
                              uint32_t* error_word, void* stream);

/* Copies the workspace error word to *code (host) after synchronising
 * stream. Returns KVARN_OK or KVARN_ERR_CUDA. */
int kvarn_read_error(const void* workspace, uint32_t* code, void* stream);

/* Zeroes the workspace error word (enqueued on stream). */
int kvarn_clear_error(void* workspace, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* KVARN_H_ */
