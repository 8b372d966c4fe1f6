// tree.cu -- attention for a tree of drafted tokens: T rows a sequence, each
// over all cached tokens and over the drafted ones that its mask shows.
//
// Calls as graph nodes (8 kv heads, 4 query heads each): 1 x 8 drafts over 1000 bf16 tokens 13.6 to 14.4 us, 64 x 16
// over up to 8192 260 to 267, 32 x 33 191 to 200; 3 x 12 over 1500 2-bit tokens 27, 48 x 16 over up to 8192 4-bit
// tokens 400, 64 x 8 2-bit 490 (bf16 253).
#include "host_checks.h"
#include "tree_join.cuh"

namespace kvarn {

cudaError_t launch_tree_bf16(const TreeArgs& a, bool wide, cudaStream_t st);
cudaError_t launch_prefill_all(const kvarn_config& cfg, const void* q, int q_dtype, const void* pool, int64_t n_pool_blocks,
                               int64_t block_bytes, const int32_t* block_table, int max_blocks, const int32_t* seq_lens, int batch,
                               int chunk, float* partials, uint32_t* err, int splits, cudaStream_t st);
int64_t prefill_splits(const kvarn_config& cfg, int64_t batch, int64_t chunk, int device);
int prefill_grid_warps(int block_size, int bits, int device);
cudaError_t launch_tree_packed(const kvarn_config& c, const TreeArgs& a, bool wide, cudaStream_t st);

namespace {

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// How a call is cut: CTAs that share a unit's query rows (128 each, or 256 where
// there are more: `wide`), and ranges of cached tokens, as many as fill the GPU with them.
struct TreePlan {
    bool wide, extra;
    int row_tiles, rows_pad, ranges;
};
// Up to 8 rows beyond 128, of bf16 pages and queries, go beside one row tile (`extra`, two CTAs an SM)
// where the tables have room for 16 tiles of 64 tokens a range, else as a second row tile: 32 x 33 drafts
// over 8192 tokens, 8 kv heads, 192 against 218 us, 8 x 34 over 4096 (13 tiles) 47.3 against 46.5,
// 2 x 33 over 1000 20.7 against 18.2.
constexpr int kExtraTiles = 16;
TreePlan tree_plan(const kvarn_config& c, int drafts, bool packed, int q_dtype, int64_t tiles) {
    const int R = drafts * (c.n_q_heads / c.n_kv_heads), sms = (int)current_device_sms();
    const bool many = R > kPRows && (packed || q_dtype == KVARN_BF16);
    const bool extra = many && !packed && R <= kPRows + kExtraRows && tiles >= (int64_t)kExtraTiles * 2 * sms;
    TreePlan p{many && !extra, extra, 1, (R + 31) / 32 * 32, 0};
    const int rows = p.wide ? 2 * kPRows : kPRows;
    if (!extra) p.row_tiles = (R + rows - 1) / rows;
    const int ctas = packed || p.wide || q_dtype == KVARN_FP32 ? 1 : 2;   // an SM
    p.ranges = ctas * sms / p.row_tiles;
    return p;
}

// Whether the prefill kernel takes the packed cache's tokens: up to three of its warps a unit, 8 / G
// drafts each, every warp expanding the codes for itself on mma.sync, so that
// its time grows by the warp, where a 128-row tile of tcgen05 costs the same for
// one row as for all. 64 sequences x 8192 2-bit tokens, 8 kv heads, prefill kernel
// against tree_packed_kernel: a warp 181 / 510 us, two 293 / 519, three 411 / 532,
// four 553 / 460; 2 x 2000 tokens 20.7 / 24.2, 22.7 / 26.8, 24.6 / 26.9, 25.0 / 26.8.
constexpr int kFewWarps = 3;
bool few_rows(const kvarn_config& c, int drafts) {
    const int per = 8 / (c.n_q_heads / c.n_kv_heads);
    return (drafts + per - 1) / per <= kFewWarps;
}

// Warps that share a unit's blocks there: as many as fill the GPU, two blocks each at least, 32 at
// most (1 x 2 drafts over 16384 tokens: 16 35.1 us, 32 28.3, 64 27.7, 128 35.6; 1 x 6 37.1, 36.8,
// 38.6, 40.4; 4 x 2 42.9, 39.3, 41.5, 42.1: the join reads a partial of each).
constexpr int kFewSplits = 32;
int few_splits(const kvarn_config& c, int64_t batch, int drafts, int max_blocks) {
    const int device = current_device(), per = 8 / (c.n_q_heads / c.n_kv_heads);
    const int64_t units = batch * c.n_kv_heads * ((drafts + per - 1) / per), warps = prefill_grid_warps(c.block_size, c.bits, device);
    int64_t n = prefill_splits(c, batch, drafts, device);
    if (units > 0 && 2 * units <= warps) n = warps / units;
    n = n < max_blocks / 2 ? n : max_blocks / 2;
    return (int)(n < 1 ? 1 : n < kFewSplits ? n : kFewSplits);
}

// The workspace: header, unit map, rotated queries and their scales, partials. Its size grows with the batch, the
// drafts and the table, so that one made for the largest call serves them all: what either cache and query type
// and any length needs is bounded by terms that do not shrink.
//   ranges: at most 2 an SM of up to 128 rows, or with `extra` 160 of partials; one of 256 rows (half as
//   many ranges of 512) takes less than that
//   few_splits: units splits <= warps with half a wave of units, <= 2.5 warps + units / 2 with more
//   (prefill_splits), and a unit is up to 8 rows; one split is always taken
struct TreeSpace {
    size_t turned, scales, partials, bytes;
};
TreeSpace tree_space(const kvarn_config& c, int32_t batch, int32_t drafts, int32_t max_blocks) {
    TreeSpace t = {0, 0, 0, kWsHeader};
    if (batch == 0) return t;
    const int64_t sms = current_device_sms(), G = c.n_q_heads / c.n_kv_heads;
    const int64_t units = (int64_t)batch * c.n_kv_heads, pad = (drafts * G + 31) / 32 * 32;
    t.turned = align256(kWsHeader + units * 2 * sizeof(int32_t));
    t.scales = t.turned + units * pad * 2 * kD * sizeof(uint16_t);
    t.partials = align256(t.scales + units * pad * sizeof(float));
    constexpr int64_t kExtraPad = kPRows + 32;
    const int64_t ranges = units * pad + 2 * sms * (pad < kExtraPad ? pad : kExtraPad);   // partial rows
    const int64_t warps = prefill_grid_warps(c.block_size, c.bits, current_device()), per = 8 / G;
    const int64_t d = drafts < kFewWarps * per ? drafts : kFewWarps * per, rows = batch * d * c.n_q_heads;
    const int64_t cap = max_blocks / 2 < 1 ? 1 : max_blocks / 2 < kFewSplits ? max_blocks / 2 : kFewSplits;
    const int64_t most = 20 * warps + 4 * units * ((d + per - 1) / per);
    int64_t few = cap * rows < most ? cap * rows : most;
    few = few > rows ? few : rows;
    const size_t a = ranges * 33 * sizeof(float4), b = few * kPartialStride * sizeof(float);
    t.bytes = sms > 0 && warps > 0 ? t.partials + (a > b ? a : b) : 0;
    return t;
}

template <bool PACKED>
int tree_attn(const kvarn_config* cfg, const void* q, int32_t q_dtype, const void* pool, int64_t n_pool_blocks,
              const void* staging, const int32_t* block_table, int32_t max_blocks, const int32_t* seq_lens, const void* k,
              const void* v, int64_t k_stride, int64_t v_stride, const uint32_t* mask, const int32_t* draft_lens,
              int32_t batch, int32_t drafts, void* out, int32_t out_dtype, void* workspace, size_t workspace_bytes,
              void* stream) {
    kvarn_config c;
    int r = check_config(cfg, &c);
    if (r != KVARN_OK) return r;
    if (out_dtype != KVARN_BF16 && out_dtype != KVARN_FP32) return KVARN_ERR_INVALID_ARG;
    if (drafts < 1 || drafts > KVARN_MAX_DRAFTS) return KVARN_ERR_INVALID_ARG;
    if (max_blocks == 0) block_table = seq_lens;         // a table without columns is never read
    r = check_packed_attn_args(c, q, q_dtype, pool, n_pool_blocks, PACKED ? staging : pool, block_table, max_blocks,
                               seq_lens, batch, drafts, (const float*)out);
    if (r != KVARN_OK || batch == 0) return r;
    if (!k || !v || !mask || !workspace || !aligned(k, 16) || !aligned(v, 16) || !aligned(mask, 4) ||
        !aligned(draft_lens, 4) || !aligned(workspace, 16))
        return KVARN_ERR_INVALID_ARG;
    if (k_stride % 8 || v_stride % 8 || k_stride < (int64_t)c.n_kv_heads * kD || v_stride < (int64_t)c.n_kv_heads * kD)
        return KVARN_ERR_INVALID_ARG;
    if (batch > 65535 || c.n_kv_heads > 65535) return KVARN_ERR_INVALID_ARG;
    if (!PACKED && n_pool_blocks > 0x7fffffff / ((int64_t)c.n_kv_heads * 2 * c.block_size)) return KVARN_ERR_INVALID_ARG;
    const TreeSpace space = tree_space(c, batch, drafts, max_blocks);
    if (space.bytes == 0) return KVARN_ERR_CUDA;
    if (workspace_bytes < space.bytes) return KVARN_ERR_WORKSPACE;
    const cudaStream_t st = (cudaStream_t)stream;

    TreeArgs a = {};
    a.q = q;
    a.pool = (const uint8_t*)pool;
    a.staging = (const uint16_t*)staging;
    a.table = block_table;
    a.lens = seq_lens;
    a.k = (const uint16_t*)k;
    a.v = (const uint16_t*)v;
    a.mask = mask;
    a.draft_lens = draft_lens;
    a.out = out;
    a.err = (uint32_t*)workspace;
    a.n_pool_blocks = n_pool_blocks;
    a.block_bytes = PACKED ? block_bytes_of(c) : (int64_t)c.n_kv_heads * 2 * c.block_size * kD * 2;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.q_dtype = q_dtype;
    a.out_bf16 = out_dtype == KVARN_BF16;
    a.max_blocks = max_blocks;
    a.batch = batch;
    a.drafts = drafts;
    a.words = (drafts + 31) / 32;
    a.n_q = c.n_q_heads;
    a.n_kv = c.n_kv_heads;
    a.G = c.n_q_heads / c.n_kv_heads;
    a.sm_scale = c.sm_scale;
    a.flags = c.flags;
    for (int i = 0; i < 4; ++i) a.sb[i] = c.sign_bits[i];
    const TreePlan plan = tree_plan(c, drafts, PACKED, q_dtype, (int64_t)batch * c.n_kv_heads * max_blocks * c.block_size / 64);
    uint8_t* ws = (uint8_t*)workspace;
    a.B = c.block_size;
    a.unit_map = (int32_t*)(ws + kWsHeader);
    a.turned = (uint16_t*)(ws + space.turned);
    a.turned_scale = (float*)(ws + space.scales);
    a.partials = (float4*)(ws + space.partials);
    a.row_tiles = plan.row_tiles;
    a.rows_pad = plan.rows_pad;
    a.ranges = plan.ranges;
    a.extra = plan.extra;
    a.late = max_blocks > 0;
    cudaError_t e = cudaSuccess;
    if (max_blocks > 0) {
        if (!PACKED) {
            e = launch_tree_bf16(a, plan.wide, st);
        } else if (few_rows(c, drafts)) {
            a.few = few_splits(c, batch, drafts, max_blocks);
            e = launch_prefill_all(c, q, q_dtype, pool, n_pool_blocks, a.block_bytes, block_table, max_blocks, seq_lens, batch, drafts,
                                   (float*)a.partials, a.err, a.few, st);
        } else {
            e = launch_tree_packed(c, a, plan.wide, st);
        }
    }
    if (e == cudaSuccess) e = launch_tree_join<PACKED>(a, st);
    return e == cudaSuccess ? KVARN_OK : KVARN_ERR_CUDA;
}

}  // namespace
}  // namespace kvarn

using namespace kvarn;

extern "C" {

size_t kvarn_tree_workspace_bytes(const kvarn_config* cfg, int32_t batch, int32_t drafts, int32_t max_blocks_per_seq) {
    kvarn_config c;
    if (check_config(cfg, &c) != KVARN_OK || batch < 0 || drafts < 1 || drafts > KVARN_MAX_DRAFTS || max_blocks_per_seq < 0 ||
        (int64_t)batch * drafts > 0x7fffffff / c.n_q_heads || (int64_t)max_blocks_per_seq * c.block_size > 0x7fffffff)
        return 0;
    return tree_space(c, batch, drafts, max_blocks_per_seq).bytes;
}

int kvarn_tree_attn(const kvarn_config* cfg, const void* q, int32_t q_dtype, const void* pool, int64_t n_pool_blocks,
                    const void* staging, const int32_t* block_table, int32_t max_blocks_per_seq, const int32_t* seq_lens,
                    const void* k, const void* v, int64_t k_stride, int64_t v_stride, const uint32_t* mask,
                    const int32_t* draft_lens, int32_t batch, int32_t drafts, void* out, int32_t out_dtype,
                    void* workspace, size_t workspace_bytes, void* stream) {
    return tree_attn<true>(cfg, q, q_dtype, pool, n_pool_blocks, staging, block_table, max_blocks_per_seq, seq_lens, k, v,
                           k_stride, v_stride, mask, draft_lens, batch, drafts, out, out_dtype, workspace, workspace_bytes,
                           stream);
}

int kvarn_tree_attn_bf16(const kvarn_config* cfg, const void* q, int32_t q_dtype, const void* kv_pool, int64_t n_pool_blocks,
                         const int32_t* block_table, int32_t max_blocks_per_seq, const int32_t* seq_lens, const void* k,
                         const void* v, int64_t k_stride, int64_t v_stride, const uint32_t* mask, const int32_t* draft_lens,
                         int32_t batch, int32_t drafts, void* out, int32_t out_dtype, void* workspace,
                         size_t workspace_bytes, void* stream) {
    return tree_attn<false>(cfg, q, q_dtype, kv_pool, n_pool_blocks, nullptr, block_table, max_blocks_per_seq, seq_lens, k, v,
                            k_stride, v_stride, mask, draft_lens, batch, drafts, out, out_dtype, workspace, workspace_bytes,
                            stream);
}

}  // extern "C"
