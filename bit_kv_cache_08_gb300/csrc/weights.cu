// weights.cu -- decode attention that also keeps the attention each cached
// token gets: beside out = sum_t p_t v_t,
//   weights_out[b][h][t] = decay weights_in[b][h][t] + sum_{j in h} p_j(t).
//
// p_j(t) = 2^(s_j(t) - m_j) / l_j needs the row's final maximum m and sum l,
// which are known only when every block has been read. The decode attention's
// split kernel (attention.cu, attention_bf16.cu) leaves its scores s (log2
// domain, fp32) in the workspace, its merge m and 1 / l, and weigh_kernel reads
// them once: 4 G bytes a token and kv head written and read, against the keys
// read and multiplied a second time. That traffic is what the weights cost. 8 kv heads, 4 query
// heads each, lengths 0.75 of these on average: 32 sequences x 8192 bf16 tokens 154 us without them and 168
// with (63 MB, 9 us at the rate of a copy), 64 x 8192 2-bit tokens 114 and 131 (126 MB, partly in L2; blocks of
// 32 132 and 152), 2 x 1000 8.3 and 9.7.
#include "attn_common.cuh"
#include "host_checks.h"

#include <type_traits>

namespace kvarn {

AttnArgs decode_split_args(const kvarn_config& cfg, const void* q, int q_dtype, const void* pool, int64_t n_pool_blocks,
                           int64_t block_bytes, const void* staging, const int32_t* block_table, int max_blocks,
                           const int32_t* seq_lens, int batch, float* out, void* workspace, int nw);
AttnArgs decode_split_args_bf16(const kvarn_config& cfg, const void* q, int q_dtype, const void* kv_pool, int64_t n_pool_blocks,
                                const int32_t* block_table, int max_blocks, const int32_t* seq_lens, int batch, float* out,
                                void* workspace, int nw);
cudaError_t launch_decode_scores(const kvarn_config& cfg, const AttnArgs& a, cudaStream_t st);
cudaError_t launch_decode_scores_bf16(const kvarn_config& cfg, const AttnArgs& a, cudaStream_t st);

struct WeighArgs {
    const float* scores;     // [batch][n_q][score_stride]
    const float2* stats;     // [batch][n_q] (maximum, 1 / sum)
    const int32_t* seq_lens;
    const float* in;         // nullptr: no earlier weights
    float* out;
    int64_t score_stride, stride;
    int64_t units;           // (sequence, kv head) pairs
    int n_kv;
    float decay;
};

// A thread takes 4 tokens of one (sequence, kv head). The kernel starts beside the
// merge, and a thread of the first wave has its loads of scores and of `in` on their way
// before it waits for the merge's (m, 1 / l). The merge's own scores, of the
// packed cache's raw tail rows, are read behind the wait.
constexpr int kWeighThreads = 256, kWeighTokens = 4 * kWeighThreads;
template <int G, int TAIL>
__global__ void __launch_bounds__(kWeighThreads) weigh_kernel(WeighArgs a) {
    const int t = blockIdx.x * kWeighTokens + 4 * threadIdx.x;
    bool waited = false;
    for (int64_t u = blockIdx.y; u < a.units; u += gridDim.y) {
        const int L = a.seq_lens[u / a.n_kv];
        const bool mine = t < L && L <= a.score_stride;   // (a length out of range: flagged by the merge)
        if (!waited && (!mine || (TAIL > 0 && t >= L - L % max(TAIL, 1)))) wait_prior_grids(), waited = true;
        if (!mine) continue;
        float w[4] = {0.f, 0.f, 0.f, 0.f};
        if (a.in != nullptr) {
            const float4 x = __ldcg(reinterpret_cast<const float4*>(a.in + u * a.stride + t));
            w[0] = a.decay * x.x;
            w[1] = a.decay * x.y;
            w[2] = a.decay * x.z;
            w[3] = a.decay * x.w;
        }
        float4 s[G];
#pragma unroll
        for (int j = 0; j < G; ++j) s[j] = __ldcg(reinterpret_cast<const float4*>(a.scores + (u * G + j) * a.score_stride + t));
        if (!waited) wait_prior_grids(), waited = true;
#pragma unroll
        for (int j = 0; j < G; ++j) {
            const float2 st = __ldcg(a.stats + u * G + j);
            w[0] = fmaf(exp2f(s[j].x - st.x), st.y, w[0]);
            w[1] = fmaf(exp2f(s[j].y - st.x), st.y, w[1]);
            w[2] = fmaf(exp2f(s[j].z - st.x), st.y, w[2]);
            w[3] = fmaf(exp2f(s[j].w - st.x), st.y, w[3]);
        }
        float* dst = a.out + u * a.stride + t;
        if (t + 4 <= L) {
            *reinterpret_cast<float4*>(dst) = make_float4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
            for (int k = 0; k < 3; ++k)
                if (t + k < L) dst[k] = w[k];
        }
    }
    if (!waited) wait_prior_grids();
}

namespace {

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// Columns of the scores: a full block table's tokens.
int64_t score_columns(const kvarn_config& c, int64_t max_blocks) { return max_blocks * c.block_size; }

size_t weights_ws_bytes(const kvarn_config& c, int32_t batch, int32_t max_blocks) {
    const size_t own = decode_ws_bytes(c, batch);
    if (own == 0 || batch == 0) return own;
    const size_t rows = (size_t)batch * c.n_q_heads;
    return align256(own) + align256(rows * sizeof(float2)) + rows * score_columns(c, max_blocks) * sizeof(float);
}

template <bool PACKED>
int attn_weights(const kvarn_config* cfg, const void* q, int32_t q_dtype, const void* pool, int64_t n_pool_blocks,
                 const void* staging, const int32_t* block_table, int32_t max_blocks, const int32_t* seq_lens,
                 int32_t batch, void* out, int32_t out_dtype, const float* weights_in, float* weights_out,
                 int64_t weights_stride, float decay, void* workspace, size_t workspace_bytes, void* stream) {
    kvarn_config c;
    int r = check_config(cfg, &c);
    if (r != KVARN_OK) return r;
    if (out_dtype != KVARN_BF16 && out_dtype != KVARN_FP32) return KVARN_ERR_INVALID_ARG;
    if (!(decay >= 0.f && decay <= 1.f)) return KVARN_ERR_INVALID_ARG;
    r = check_packed_attn_args(c, q, q_dtype, pool, n_pool_blocks, PACKED ? staging : pool, block_table, max_blocks,
                               seq_lens, batch, 1, (const float*)out);
    if (r != KVARN_OK || batch == 0) return r;
    if (!weights_out || !workspace || !aligned(weights_out, 16) || !aligned(weights_in, 16) || !aligned(workspace, 16))
        return KVARN_ERR_INVALID_ARG;
    const int64_t columns = score_columns(c, max_blocks), units = (int64_t)batch * c.n_kv_heads;
    if (weights_stride % 4 || weights_stride < columns) return KVARN_ERR_INVALID_ARG;
    const size_t need = weights_ws_bytes(c, batch, max_blocks);
    if (need == 0) return KVARN_ERR_CUDA;
    if (workspace_bytes < need) return KVARN_ERR_WORKSPACE;
    const int d = current_device();
    const int nw = PACKED ? attn_grid_warps(c.block_size, c.bits, d) : attn_bf16_grid_warps(c.block_size, d);
    if (nw <= 0) return KVARN_ERR_CUDA;
    const cudaStream_t st = (cudaStream_t)stream;

    AttnArgs a = PACKED ? decode_split_args(c, q, q_dtype, pool, n_pool_blocks, block_bytes_of(c), staging, block_table,
                                            max_blocks, seq_lens, batch, (float*)out, workspace, nw)
                        : decode_split_args_bf16(c, q, q_dtype, pool, n_pool_blocks, block_table, max_blocks, seq_lens, batch,
                                                 (float*)out, workspace, nw);
    uint8_t* ws = (uint8_t*)workspace + align256(decode_ws_bytes(c, batch));
    a.stats = (float2*)ws;
    a.scores = (float*)(ws + align256((size_t)batch * c.n_q_heads * sizeof(float2)));
    a.score_stride = columns;
    a.out_bf16 = out_dtype == KVARN_BF16;
    cudaError_t e = PACKED ? launch_decode_scores(c, a, st) : launch_decode_scores_bf16(c, a, st);
    if (e != cudaSuccess) return KVARN_ERR_CUDA;
    if (columns == 0) return KVARN_OK;

    WeighArgs w = {};
    w.scores = a.scores;
    w.stats = a.stats;
    w.seq_lens = seq_lens;
    w.in = decay > 0.f ? weights_in : nullptr;
    w.out = weights_out;
    w.score_stride = columns;
    w.stride = weights_stride;
    w.units = units;
    w.n_kv = c.n_kv_heads;
    w.decay = decay;
    const dim3 grid((unsigned)((columns + kWeighTokens - 1) / kWeighTokens), (unsigned)(units < 65535 ? units : 65535));
    auto weigh = [&](auto tail) {
        constexpr int TAIL = decltype(tail)::value;
        return a.G == 1 ? weigh_kernel<1, TAIL> : a.G == 2 ? weigh_kernel<2, TAIL> : a.G == 3 ? weigh_kernel<3, TAIL> : weigh_kernel<4, TAIL>;
    };
    using std::integral_constant;
    const auto fn = !PACKED ? weigh(integral_constant<int, 0>()) : c.block_size == 32 ? weigh(integral_constant<int, 32>()) : weigh(integral_constant<int, 64>());
    e = launch_pdl(fn, grid, kWeighThreads, 0, st, w);
    return e == cudaSuccess ? KVARN_OK : KVARN_ERR_CUDA;
}

}  // namespace
}  // namespace kvarn

using namespace kvarn;

extern "C" {

size_t kvarn_weights_workspace_bytes(const kvarn_config* cfg, int32_t batch, int32_t max_blocks_per_seq) {
    kvarn_config c;
    if (check_config(cfg, &c) != KVARN_OK || batch < 0 || max_blocks_per_seq < 0 || batch > 0x7fffffff / c.n_q_heads ||
        (int64_t)max_blocks_per_seq * c.block_size > 0x7fffffff)
        return 0;
    return weights_ws_bytes(c, batch, max_blocks_per_seq);
}

int kvarn_decode_attn_weights(const kvarn_config* cfg, const void* q, int32_t q_dtype, const void* pool,
                              int64_t n_pool_blocks, const void* staging, const int32_t* block_table,
                              int32_t max_blocks_per_seq, const int32_t* seq_lens, int32_t batch, void* out,
                              int32_t out_dtype, const float* weights_in, float* weights_out, int64_t weights_stride,
                              float decay, void* workspace, size_t workspace_bytes, void* stream) {
    return attn_weights<true>(cfg, q, q_dtype, pool, n_pool_blocks, staging, block_table, max_blocks_per_seq, seq_lens,
                              batch, out, out_dtype, weights_in, weights_out, weights_stride, decay, workspace,
                              workspace_bytes, stream);
}

int kvarn_decode_attn_weights_bf16(const kvarn_config* cfg, const void* q, int32_t q_dtype, const void* kv_pool,
                                   int64_t n_pool_blocks, const int32_t* block_table, int32_t max_blocks_per_seq,
                                   const int32_t* seq_lens, int32_t batch, void* out, int32_t out_dtype,
                                   const float* weights_in, float* weights_out, int64_t weights_stride, float decay,
                                   void* workspace, size_t workspace_bytes, void* stream) {
    return attn_weights<false>(cfg, q, q_dtype, kv_pool, n_pool_blocks, nullptr, block_table, max_blocks_per_seq, seq_lens,
                               batch, out, out_dtype, weights_in, weights_out, weights_stride, decay, workspace,
                               workspace_bytes, stream);
}

}  // extern "C"
