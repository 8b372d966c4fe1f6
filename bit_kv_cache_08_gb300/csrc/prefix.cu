// prefix.cu -- decode attention for a batch whose sequences share a prefix:
// out = softmax(sm_scale q.k) v over the first prefix_lens[b] tokens of the
// shared prefix, then sequence b's own tokens.
//
// The prefix is read once for the whole batch: with R = batch * G query rows
// per kv head, S = Q K^T and O = P V are matrix products of R rows, which a
// decode that walks each sequence's own block table reads R times over. Three
// launches: the prefix kernel (partials of token ranges), the split kernel of
// the plain decode attention over the own tokens, and a merge of both kinds
// of partial in the log-sum-exp sense,
//   m = max m_i,  l = sum l_i 2^(m_i - m),  acc = sum acc_i 2^(m_i - m),
// which also rotates back and adds the raw tail rows (packed cache). Where own
// tables are short, the last two are one: prefix_join_kernel over bf16 pages,
// prefix_join_packed_kernel (attention.cu) over the packed cache.
#include "host_checks.h"
#include "prefix_merge.cuh"

namespace kvarn {

AttnArgs decode_split_args(const kvarn_config& cfg, const void* q, int q_dtype, const void* pool, int64_t n_pool_blocks,
                           int64_t block_bytes, const void* staging, const int32_t* block_table, int max_blocks,
                           const int32_t* seq_lens, int batch, float* out, void* workspace, int nw);
cudaError_t launch_decode_split(const kvarn_config& cfg, const AttnArgs& a, bool late, cudaStream_t st);
cudaError_t launch_prefix_join_packed(const kvarn_config& cfg, const AttnArgs& a, const PrefixMerge& pm, cudaStream_t st);
cudaError_t launch_decode_split_bf16(const kvarn_config& cfg, const void* q, int q_dtype, const void* kv_pool,
                                     int64_t n_pool_blocks, const int32_t* block_table, int max_blocks,
                                     const int32_t* seq_lens, int batch, float* out, void* workspace, int nw,
                                     bool late, AttnArgs* args, cudaStream_t st);

cudaError_t launch_prefix_bf16(const PrefixArgs& p, int block_size, cudaStream_t st);
cudaError_t launch_prefix_packed(const kvarn_config& c, const PrefixArgs& p, cudaStream_t st);

// ---------------------------------------------------------------- merge
// One CTA of 4 warps per (sequence, kv head): the raw tail rows (ROT), which
// wait for nothing, then, when the split kernel is through, 4 / G warps to
// each of the G query heads with a share of the row's partials; the row's first
// warp combines the shares and finishes the row. On the tensor cores a tail row
// costs a quarter of the instructions that it costs scored by a lane, which
// took 6 and 5 us off calls of 64 x 8192 at 2 bits and 128 x 32 768 at 4 (55 and
// 210 us now; the kernel alone and cold 14 and 19).
constexpr int kMergeWarps = 4;
template <int B, bool ROT>
__global__ void __launch_bounds__(32 * kMergeWarps, 4) prefix_merge_kernel(AttnArgs a, PrefixMerge pm) {
    const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
    const int b = blockIdx.x, h = blockIdx.y;
    const int parts = merge_parts(a.G, kMergeWarps), g = wp / parts, part = wp % parts;
    __shared__ __align__(16) float slices[kMergeWarps][kPartialStride];
    __shared__ __align__(16) float tails[ROT ? 4 : 1][4][kPartialStride];
    __shared__ uint2 qf[8][32];
    const int L = a.seq_lens[b], PL = pm.lens[b];
    if (!lengths_ok<B>(a, pm, L, PL)) {
        wait_prior_grids();
        refuse_row(a, pm, b, h);
        return;
    }
    const int ntail = ROT ? L % B : 0;
    if (ROT && ntail > 0) tail_slice16<B, kMergeWarps>(a, b, h, ntail, wp, lane, qf, tails);
    wait_prior_grids();
    if (g < a.G) {
        // the own partials: those of the warps that the split kernel's unit map
        // names (a range outside the grid, left by a warp that gave up, is none)
        const int64_t u = (int64_t)b * a.n_kv + h;
        const int2 wm = __ldcg(reinterpret_cast<const int2*>(a.unit_map) + u);
        const int np = (ROT ? L >= B : L > 0) && wm.x >= 0 && wm.y >= wm.x && wm.y < a.nw ? wm.y - wm.x + 1 : 0;
        const float* p0 = a.partials + ((u + max(wm.x, 0)) * a.G + g) * kPartialStride;
        float m = -INFINITY, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
        const int n = np + (PL > 0 ? pm.splits : 0);
        const int64_t R = (int64_t)a.batch * a.G;
        lse_list<16>(p0, np, (int64_t)a.G * kPartialStride, pm.partials + partial_row(0, a.n_kv, h, R, (int64_t)b * a.G + g),
                     partial_row(1, a.n_kv, 0, R, 0), n * part / parts, n * (part + 1) / parts, lane, m, l, acc);
        put_slice(slices[wp], lane, m, l, acc);
    }
    __syncthreads();
    if (g >= a.G || part != 0) return;
    float m = -INFINITY, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
    combine_slices(&slices[wp][0], parts, lane, m, l, acc);
    finish_row<ROT>(a, pm, (int64_t)b * a.n_q + h * a.G + g, L > 0 || PL > 0, ntail > 0 ? &tails[g][0][0] : nullptr, lane, m, l, acc);
}

// ---------------------------------------------------------------- own tokens and merge in one (bf16 pages)
constexpr int kJoinTokens = 2048;   // of an own table's columns, at most

// The 16-token chunks wp, wp + W, ... of a unit's own pages, for bf16_slice.
template <int B, int W>
struct OwnChunks {
    const AttnArgs& a;
    int L, wp, held;
    __device__ __forceinline__ OwnChunks(const AttnArgs& a, int b, int L, int wp, int lane) : a(a), L(L), wp(wp) {
        // lane i holds the block of chunk i (without a look at L, which is on its way too); -1: a bad one
        static_assert(kJoinTokens <= 32 * W * kChunk, "a lane for each chunk of a warp");
        const int c = (wp + W * lane) / (B / kChunk);
        held = c < a.max_blocks ? a.block_table[(int64_t)b * a.max_blocks + c] : 0;
        if (held < 0 || held >= a.n_pool_blocks) held = -1;
        if (held < 0 && lane < count()) raise_error(a.err, KVARN_DEVERR_BLOCK_ID);
    }
    __device__ __forceinline__ int count() const {
        const int chunks = (L + kChunk - 1) / kChunk;
        return chunks > wp ? (chunks - wp + W - 1) / W : 0;
    }
    __device__ __forceinline__ ChunkRows operator()(int i) const {
        const int phys = __shfl_sync(kFull, held, i);
        return {max(phys, 0) * a.block_bytes + (wp + W * i) % (B / kChunk) * (kChunk * kD * 2),
                phys >= 0 ? L - (wp + W * i) * kChunk : 0};
    }
};

// One CTA of W warps per (sequence, kv head): its own tokens, then, when the
// prefix kernel is through, the merge with the prefix's partials. Against the
// split kernel and a merge this saves a launch and the own tokens' partials,
// but a unit has only its CTA. Memory bounds it (512 bytes a token and kv
// head) where the units fill the GPU, the chain of dependent loads where they
// do not. A call of 64 sequences with 192 own tokens of 8 kv heads behind 8192
// of a prefix takes 32.6 us as a graph node with CTAs of 4 at 16 warps per SM and
// 40.7 with the split kernel and a merge, 128 with 384 behind 32 768 take 118.0
// and 127.2. (8 or 12 warps per SM with the next chunk's loads in flight during a
// chunk's products took 12 and 4 us more for the first, 21 more and 1 less for the
// second.)
template <int B, int W>
__global__ void __launch_bounds__(32 * W, 16 / W) prefix_join_kernel(AttnArgs a, PrefixMerge pm) {
    const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
    const int b = blockIdx.x, h = blockIdx.y;
    const int parts = merge_parts(a.G, W), g = wp / parts, part = wp % parts;
    const int64_t gw = (int64_t)b * a.n_q + h * a.G + g;
    __shared__ __align__(16) float own[4][W][kPartialStride];
    __shared__ __align__(16) float slices[W][kPartialStride];
    __shared__ uint2 qf[8][32];
    const int L = a.seq_lens[b], PL = pm.lens[b];
    if (!lengths_ok<B>(a, pm, L, PL)) {
        wait_prior_grids();
        refuse_row(a, pm, b, h);
        return;
    }
    const OwnChunks<B, W> chunks(a, b, L, wp, lane);
    bf16_slice<B, W, W>(a, b, h, chunks.count(), a.pool + (int64_t)h * 2 * B * kD * 2, chunks, wp, lane, qf, own);
    wait_prior_grids();   // the prefix kernel, beside which this one may have started
    if (g < a.G) prefix_slice(a, pm, b, h, g, part, parts, PL, lane, slices[wp]);
    __syncthreads();
    if (g >= a.G || part != 0) return;
    float m = -INFINITY, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
    combine_slices(&slices[wp][0], parts, lane, m, l, acc);
    float mo = -INFINITY, lo = 0.f, ao[4] = {0.f, 0.f, 0.f, 0.f};
    combine_slices(&own[g][0][0], W, lane, mo, lo, ao);
    add_slice(m, l, acc, mo, lo, ao);
    finish_row<false>(a, pm, gw, L > 0 || PL > 0, nullptr, lane, m, l, acc);
}

// ---------------------------------------------------------------- host side
namespace {

constexpr int64_t kMaxPrefix = 1 << 30;   // tokens

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// How the prefix kernel is cut: query rows of a CTA, token ranges (splits) and
// partials per range (2 for one row tile over bf16 pages, where the even and
// the odd K/V tiles of a range are summed apart).
struct PrefixPlan {
    int rows, streams, splits;
    int most;   // ranges that a shorter prefix may take: the workspace holds them, so that it serves that one too
};

PrefixPlan prefix_plan(const kvarn_config& c, int64_t batch, int64_t prefix_blocks, bool packed, int q_dtype) {
    const int64_t sms = current_device_sms(), R = batch * (c.n_q_heads / c.n_kv_heads);
    PrefixPlan p{kPRows, 1, 0, 0};
    if (sms <= 0) return p;
    if (R > kPRows && (packed || q_dtype == KVARN_BF16)) p.rows = 2 * kPRows;
    else if (!packed) p.streams = 2;
    // The token ranges that make waves of CTAs times a CTA's tiles least: 3 tiles
    // stand for a CTA's start and end; of the ranges with the same tiles for a CTA
    // the fewest, for there are as many partials. More than one wave only where one
    // would leave many SMs idle. Calls with a few own tokens as graph nodes, 32
    // query heads on 8 kv heads, us by ranges (* the plan's):
    //   64 behind 8192     bf16  10: 28.6  13: 25.1  16*: 23.9  19: 24.8
    //                      2-bit 13: 47.8  16: 43.5  19*: 41.5
    //   128 behind 32 768  bf16   7: 97.1   8: 87.9   9*: 81.4  19: 92.9
    //                      4-bit  7: 212    8: 188    9*: 171   19: 184
    //   300 behind 8192    bf16   2: 94.0   3*: 73.4  4: 101    5: 90.3   8: 96.3
    //                      2-bit  2: 195    3*: 145   4: 207    5: 177    8: 182
    //   1300 behind 8000   bf16   1: 367    2: 314    3*: 306   4: 307
    //                      2-bit  1: 742    2: 606    3*: 575   4: 568
    // Packed CTAs of one tile lost 3 us to twice the partials.
    const int64_t units = c.n_kv_heads * ((R + p.rows - 1) / p.rows);
    const int64_t tile = packed ? 64 : 128, tiles = (prefix_blocks * c.block_size + tile - 1) / tile;
    const int64_t ranges = packed ? (tiles + 1) / 2 : tiles;
    const int max_waves = 4 * units > sms ? 4 : 1;
    auto within = [&](int64_t s) { return s > ranges ? (ranges > 1 ? ranges : 1) : s > 1 ? s : 1; };
    int64_t least = 0;
    for (int waves = 1; waves <= max_waves; ++waves) {
        const int64_t s = within(waves * sms / units), per = (tiles + s - 1) / s;
        const int64_t few = per > 0 ? (tiles + per - 1) / per : 1;
        const int64_t cost = (units * few + sms - 1) / sms * (per + 3);
        if (waves > 1 && cost >= least) continue;
        least = cost;
        p.splits = (int)few;
    }
    p.most = (int)within(max_waves * sms / units);
    return p;
}

size_t prefix_ws_bytes(const kvarn_config& c, int32_t batch, int64_t prefix_blocks) {
    if (batch == 0) return kWsHeader;
    const size_t own = decode_ws_bytes(c, batch);
    int slots = 0;   // the most that either cache and query type needs
    for (int k = 0; k < 3; ++k) {
        const PrefixPlan p = prefix_plan(c, batch, prefix_blocks, k == 0, k == 1 ? KVARN_BF16 : KVARN_FP32);
        if (p.splits == 0) return 0;
        slots = p.most * p.streams > slots ? p.most * p.streams : slots;
    }
    if (own == 0) return 0;
    return align256(own) + (size_t)slots * batch * c.n_q_heads * kPartialStride * sizeof(float);
}

template <bool PACKED>
int prefix_attn(const kvarn_config* cfg, const void* q, int32_t q_dtype, const void* pool, int64_t n_pool_blocks,
                const void* staging, const int32_t* prefix_table, int32_t prefix_blocks, const int32_t* prefix_lens,
                const int32_t* block_table, int32_t max_blocks, const int32_t* seq_lens, int32_t batch, void* out,
                int32_t out_dtype, void* workspace, size_t workspace_bytes, void* stream) {
    kvarn_config c;
    int r = check_config(cfg, &c);
    if (r != KVARN_OK) return r;
    if (out_dtype != KVARN_BF16 && out_dtype != KVARN_FP32) return KVARN_ERR_INVALID_ARG;
    if (prefix_blocks < 0 || (int64_t)prefix_blocks * c.block_size > kMaxPrefix) return KVARN_ERR_INVALID_ARG;
    if (max_blocks == 0) block_table = seq_lens;         // tables without columns are never read
    if (prefix_blocks == 0) prefix_table = prefix_lens;
    r = check_packed_attn_args(c, q, q_dtype, pool, n_pool_blocks, PACKED ? staging : pool, block_table, max_blocks,
                               seq_lens, batch, 1, (const float*)out);
    if (r != KVARN_OK || batch == 0) return r;
    if (!prefix_table || !prefix_lens || !workspace || !aligned(prefix_table, 4) || !aligned(prefix_lens, 4) ||
        !aligned(workspace, 16))
        return KVARN_ERR_INVALID_ARG;
    const int G = c.n_q_heads / c.n_kv_heads;
    if (!PACKED && n_pool_blocks > 0x7fffffff / ((int64_t)c.n_kv_heads * 2 * c.block_size)) return KVARN_ERR_INVALID_ARG;
    if (((int64_t)batch * G + kPRows - 1) / kPRows > 65535 || c.n_kv_heads > 65535) return KVARN_ERR_INVALID_ARG;
    const size_t need = prefix_ws_bytes(c, batch, prefix_blocks);
    if (need == 0) return KVARN_ERR_CUDA;
    if (workspace_bytes < need) return KVARN_ERR_WORKSPACE;
    const int d = current_device();
    const int nw = PACKED ? attn_grid_warps(c.block_size, c.bits, d) : attn_bf16_grid_warps(c.block_size, d);
    if (nw <= 0) return KVARN_ERR_CUDA;
    const cudaStream_t st = (cudaStream_t)stream;

    PrefixArgs p = {};
    p.q = q;
    p.pool = (const uint8_t*)pool;
    p.table = prefix_table;
    p.lens = prefix_lens;
    p.partials = (float*)((uint8_t*)workspace + align256(decode_ws_bytes(c, batch)));
    p.err = (uint32_t*)workspace;
    p.n_pool_blocks = n_pool_blocks;
    p.block_bytes = PACKED ? block_bytes_of(c) : (int64_t)c.n_kv_heads * 2 * c.block_size * kD * 2;
    p.q_dtype = q_dtype;
    p.n_blocks = prefix_blocks;
    p.batch = batch;
    p.n_q = c.n_q_heads;
    p.n_kv = c.n_kv_heads;
    p.G = G;
    const PrefixPlan plan = prefix_plan(c, batch, prefix_blocks, PACKED, q_dtype);
    p.splits = plan.splits;
    p.sm_scale = c.sm_scale;
    p.flags = c.flags;
    for (int i = 0; i < 4; ++i) p.sb[i] = c.sign_bits[i];
    cudaError_t e;
    AttnArgs a = {};
    // An own table of more columns may hold sequences that are long for one CTA:
    // 4 sequences of up to 2048 / 4096 own tokens in bf16 pages, 8 kv heads, take
    // 28 / 38 us against 29 / 32 by the split kernel and a merge, 128 sequences
    // 169 / 310 against 181 / 325. Packed blocks need an SM's shared memory for a
    // unit: with a CTA per SM 16 sequences behind 4096 tokens take 21 .. 34 us
    // against 24 .. 39 (up to 64 .. 2048 own tokens), 4 sequences 20 .. 33 against
    // 22 .. 34, though 25 .. 28 against 22 .. 23 with 256 to 1024.
    const bool join = (int64_t)max_blocks * c.block_size <= kJoinTokens &&
                      (!PACKED || (int64_t)batch * c.n_kv_heads <= current_device_sms());
    if constexpr (PACKED) {
        a = decode_split_args(c, q, q_dtype, pool, n_pool_blocks, p.block_bytes, staging, block_table, max_blocks, seq_lens,
                              batch, nullptr, workspace, nw);
        e = launch_prefix_packed(c, p, st);
        if (e == cudaSuccess && !join) e = launch_decode_split(c, a, true, st);
    } else {
        e = launch_prefix_bf16(p, c.block_size, st);
        if (e == cudaSuccess && !join)
            e = launch_decode_split_bf16(c, q, q_dtype, pool, n_pool_blocks, block_table, max_blocks, seq_lens, batch,
                                         nullptr, workspace, nw, true, &a, st);
    }
    if (e != cudaSuccess) return KVARN_ERR_CUDA;
    const PrefixMerge pm{p.partials, prefix_lens, prefix_blocks * c.block_size, plan.splits * plan.streams, out, out_dtype == KVARN_BF16};
    const dim3 units(batch, c.n_kv_heads);
    const int threads = 32 * kMergeWarps;
    if constexpr (PACKED) {
        if (join)
            e = launch_prefix_join_packed(c, a, pm, st);
        else
            e = c.block_size == 32 ? launch_pdl(prefix_merge_kernel<32, true>, units, threads, 0, st, a, pm)
                                   : launch_pdl(prefix_merge_kernel<64, true>, units, threads, 0, st, a, pm);
    } else if (!join)
        e = launch_pdl(prefix_merge_kernel<kChunk, false>, units, threads, 0, st, a, pm);
    else {
        a.q = q;
        a.pool = p.pool;
        a.block_table = block_table;
        a.seq_lens = seq_lens;
        a.err = p.err;
        a.n_pool_blocks = n_pool_blocks;
        a.block_bytes = p.block_bytes;
        a.q_dtype = q_dtype;
        a.max_blocks = max_blocks;
        a.batch = batch;
        a.n_q = p.n_q;
        a.n_kv = p.n_kv;
        a.G = G;
        a.sm_scale = c.sm_scale;
        const auto start = [&](auto w) {
            constexpr int W = decltype(w)::value;
            return c.block_size == 32 ? launch_pdl(prefix_join_kernel<32, W>, units, 32 * W, 0, st, a, pm)
                                      : launch_pdl(prefix_join_kernel<64, W>, units, 32 * W, 0, st, a, pm);
        };
        // 16 warps per SM, and as many of them to a unit as let all units run at
        // once: 16 sequences of up to 64 / 1024 own tokens, 8 kv heads, take 14.0 /
        // 22.6 us with 16 to a unit and 15.5 / 30.5 with 8, 28 sequences 17.0 / 36.2
        // with 8 and 19.6 / 50.4 with 4. Beyond that 4, but 8 for long tables: 64
        // sequences 21.1 / 64.5 with 4, 23.2 / 63.2 with 8, 40 of 1024 57 and 49.
        const int64_t n = (int64_t)batch * c.n_kv_heads, sms = current_device_sms();
        const bool wide = n <= 2 * sms || (int64_t)max_blocks * c.block_size > kJoinTokens / 4;
        e = n <= sms ? start(std::integral_constant<int, 16>{})
                     : wide ? start(std::integral_constant<int, 8>{}) : start(std::integral_constant<int, 4>{});
    }
    return e == cudaSuccess ? KVARN_OK : KVARN_ERR_CUDA;
}

}  // namespace
}  // namespace kvarn

using namespace kvarn;

extern "C" {

size_t kvarn_prefix_workspace_bytes(const kvarn_config* cfg, int32_t batch, int32_t prefix_blocks) {
    kvarn_config c;
    if (check_config(cfg, &c) != KVARN_OK || batch < 0 || prefix_blocks < 0 ||
        (int64_t)prefix_blocks * c.block_size > kMaxPrefix || batch > 0x7fffffff / c.n_q_heads)
        return 0;
    return prefix_ws_bytes(c, batch, prefix_blocks);
}

int kvarn_prefix_attn(const kvarn_config* cfg, const void* q, int32_t q_dtype, const void* pool, int64_t n_pool_blocks,
                      const void* staging, const int32_t* prefix_table, int32_t prefix_blocks,
                      const int32_t* prefix_lens, const int32_t* block_table, int32_t max_blocks_per_seq,
                      const int32_t* seq_lens, int32_t batch, void* out, int32_t out_dtype, void* workspace,
                      size_t workspace_bytes, void* stream) {
    return prefix_attn<true>(cfg, q, q_dtype, pool, n_pool_blocks, staging, prefix_table, prefix_blocks, prefix_lens,
                             block_table, max_blocks_per_seq, seq_lens, batch, out, out_dtype, workspace,
                             workspace_bytes, stream);
}

int kvarn_prefix_attn_bf16(const kvarn_config* cfg, const void* q, int32_t q_dtype, const void* kv_pool,
                           int64_t n_pool_blocks, const int32_t* prefix_table, int32_t prefix_blocks,
                           const int32_t* prefix_lens, const int32_t* block_table, int32_t max_blocks_per_seq,
                           const int32_t* seq_lens, int32_t batch, void* out, int32_t out_dtype, void* workspace,
                           size_t workspace_bytes, void* stream) {
    return prefix_attn<false>(cfg, q, q_dtype, kv_pool, n_pool_blocks, nullptr, prefix_table, prefix_blocks, prefix_lens,
                              block_table, max_blocks_per_seq, seq_lens, batch, out, out_dtype, workspace,
                              workspace_bytes, stream);
}

}  // extern "C"
