// tree.cu -- attention for a tree of drafted tokens: T rows a sequence, each
// over all cached tokens and over the drafted ones that its mask shows.
#include "host_checks.h"
#include "quantize.cuh"
#include "tree_join.cuh"

namespace kvarn {

cudaError_t launch_tree_bf16(const TreeArgs& a, bool wide, cudaStream_t st);

constexpr int kSimpleRows = 16;   // query rows of a CTA: 4 a warp

// The code of (token t, channel c) of a head-block's code section.
template <int BITS>
__device__ __forceinline__ int code_at(const uint8_t* hb, int kind, int t, int c) {
    int ra, rb, w, p;
    const int g = c / 32;
    if (kind == 0) {
        const int i = t % 4, e = c % 8;
        ra = t % 32 / 4, rb = c % 32 / 8;
        w = BITS == 4 ? 4 * i + g : 2 * i + g / 2;
        p = BITS == 4 ? 4 * (e / 2) + 16 * (e % 2) : 2 * (4 * (g % 2) + e / 2) + 16 * (e % 2);
    } else {
        const int d = t % 8, f = c % 4;
        rb = t % 32 / 8, ra = c % 32 / 4;
        w = BITS == 4 ? 4 * g + f : 2 * g + f / 2;
        p = BITS == 4 ? 4 * (d / 2) + 16 * (d % 2) : 2 * (4 * (d / 4) + 2 * (d % 4 / 2) + f % 2) + 16 * (d % 2);
    }
    const uint32_t* rec = reinterpret_cast<const uint32_t*>(hb) + (32 * (t / 32) + 4 * ra + rb) * 4 * BITS;
    if (BITS == 4) return rec[w] >> p & 15;
    int code = rec[w] >> p & 3;
    if (BITS == 3) code |= (rec[8 + w / 2] >> (8 * (w % 2) + p % 16 / 2 + 16 * (p / 16)) & 1) << 2;
    return code;
}

__device__ __forceinline__ void visit(float s, const float (&v)[4], float& m, float& l, float (&acc)[4]) {
    const float mn = fmaxf(m, s);
    const float f = m == -INFINITY ? 0.f : exp2f(m - mn), p = exp2f(s - mn);
    l = l * f + p;
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[k] = fmaf(acc[k], f, p * v[k]);
    m = mn;
}

// One CTA per 16 query rows of a (sequence, kv head), 4 rows a warp, one token
// after the other.
template <int B, int BITS, bool PACKED>
__global__ void __launch_bounds__(128) tree_simple_kernel(TreeArgs a) {
    wait_prior_grids();
    __shared__ __align__(16) float ks[32][kD], vs[32][kD];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int h = blockIdx.y, b = blockIdx.z;
    const int L = a.lens[b], T = tree_rows(a, b);
    const bool bad = L < 0 || (int64_t)L > (int64_t)a.max_blocks * B || T < 0;
    if (bad && tid == 0) raise_error(a.err, KVARN_DEVERR_POSITION);
    const int R = a.drafts * a.G;
    float q[4][4], qr[4][4], m[4], l[4], acc[4][4];
    const float qs = a.sm_scale * kLog2e;
    const bool rotate = PACKED && !(a.flags & KVARN_FLAG_NO_ROTATION);
    float sg[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) sg[k] = sign_of4(a.sb[0], a.sb[1], a.sb[2], a.sb[3], 4 * lane + k);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = blockIdx.x * kSimpleRows + 4 * warp + i;
        m[i] = -INFINITY;
        l[i] = acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
        q[i][0] = q[i][1] = q[i][2] = q[i][3] = 0.f;
        if (row < R) load_q4(a.q, a.q_dtype, ((int64_t)b * a.drafts + row / a.G) * a.n_q + h * a.G + row % a.G, lane, q[i]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            q[i][k] *= qs;
            qr[i][k] = rotate ? q[i][k] * sg[k] : q[i][k];
        }
        if (rotate) {
            fwht128(qr[i], lane);
#pragma unroll
            for (int k = 0; k < 4; ++k) qr[i][k] *= kInvSqrtD;
        }
    }
    const int inside = bad ? 0 : PACKED ? L / B * B : L;
    for (int t0 = 0; t0 < inside; t0 += 32) {
        const int64_t page = a.table[(int64_t)b * a.max_blocks + t0 / B];
        const bool ok = page >= 0 && page < a.n_pool_blocks;
        if (!ok && tid == 0) raise_error(a.err, KVARN_DEVERR_BLOCK_ID);
        __syncthreads();
        for (int x = tid; x < 2 * 32 * kD; x += 128) {
            const int kind = x / (32 * kD), t = x / kD % 32, c = x % kD;
            float val = 0.f;
            if (ok && t0 + t < inside) {
                const uint8_t* block = a.pool + page * a.block_bytes;
                const int bt = t0 % B + t;
                if (PACKED) {
                    const uint8_t* hb = block + (2 * h + kind) * head_block_bytes(B, BITS);
                    auto half_at = [&](int off, int i) { return h2f(reinterpret_cast<const uint16_t*>(hb + off)[i]); };
                    val = fmaf((float)code_at<BITS>(hb, kind, bt, c), half_at(off_s(B, BITS), c / 32 * B + bt),
                               half_at(off_z(B, BITS), c / 32 * B + bt)) *
                          half_at(off_R(B, BITS), bt) * half_at(off_C(B, BITS), c);
                } else {
                    val = bf2f(reinterpret_cast<const uint16_t*>(block)[((2 * h + kind) * B + bt) * kD + c]);
                }
            }
            (kind ? vs : ks)[t][c] = val;
        }
        __syncthreads();
        if (!ok) continue;
        for (int t = 0; t < min(32, inside - t0); ++t) {
            const float4 k4 = reinterpret_cast<const float4*>(ks[t])[lane], v4 = reinterpret_cast<const float4*>(vs[t])[lane];
            const float vv[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float s = warp_sum(qr[i][0] * k4.x + qr[i][1] * k4.y + qr[i][2] * k4.z + qr[i][3] * k4.w);
                visit(s, vv, m[i], l[i], acc[i]);
            }
        }
    }
    if (rotate)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            fwht128(acc[i], lane);
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[i][k] *= kInvSqrtD * sg[k];
        }
    auto row4 = [&](const uint16_t* p, float (&x)[4]) {
        const uint2 u = reinterpret_cast<const uint2*>(p)[lane];
        x[0] = __uint_as_float(u.x << 16);
        x[1] = __uint_as_float(u.x & 0xffff0000u);
        x[2] = __uint_as_float(u.y << 16);
        x[3] = __uint_as_float(u.y & 0xffff0000u);
    };
    const int tail = bad ? 0 : L - inside;
    for (int t = 0; t < tail; ++t) {
        float kk[4], vv[4];
        const uint16_t* st = a.staging + (((int64_t)b * a.n_kv + h) * 2 * B + t) * kD;
        row4(st, kk);
        row4(st + B * kD, vv);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            visit(warp_sum(q[i][0] * kk[0] + q[i][1] * kk[1] + q[i][2] * kk[2] + q[i][3] * kk[3]), vv, m[i], l[i], acc[i]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = blockIdx.x * kSimpleRows + 4 * warp + i;
        const int r = row / a.G;
        if (row >= R || (!bad && r >= T)) continue;
        bool any = !bad && L > 0, wrong = bad;
        const uint32_t* mask = a.mask + ((int64_t)b * a.drafts + r) * a.words;
        for (int t = 0; t < T; ++t) {
            if (!(mask[t / 32] >> (t % 32) & 1)) continue;
            any = true;
            float kk[4], vv[4];
            const int64_t at = (int64_t)b * a.drafts + t;
            row4(a.k + at * a.k_stride + h * kD, kk);
            row4(a.v + at * a.v_stride + h * kD, vv);
            wrong = wrong || __any_sync(kFull, !(isfinite(vv[0]) && isfinite(vv[1]) && isfinite(vv[2]) && isfinite(vv[3])));
            visit(warp_sum(q[i][0] * kk[0] + q[i][1] * kk[1] + q[i][2] * kk[2] + q[i][3] * kk[3]), vv, m[i], l[i], acc[i]);
        }
        if (wrong || (any && m[i] == -INFINITY)) l[i] = NAN;
        const float inv = l[i] > 0.f ? 1.f / l[i] : l[i];   // (0 for nothing seen; NaN stays)
        const float o[4] = {acc[i][0] * inv, acc[i][1] * inv, acc[i][2] * inv, acc[i][3] * inv};
        const int64_t at = ((int64_t)b * a.drafts + r) * a.n_q + h * a.G + row % a.G;
        if (a.out_bf16) {
            const __nv_bfloat162 x = __floats2bfloat162_rn(o[0], o[1]), y = __floats2bfloat162_rn(o[2], o[3]);
            reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at * kD)[lane] =
                make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
        } else {
            reinterpret_cast<float4*>(static_cast<float*>(a.out) + at * kD)[lane] = make_float4(o[0], o[1], o[2], o[3]);
        }
    }
}

namespace {

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// How a call is cut: CTAs that share a unit's query rows (128 each, or 256 where
// there are more: `wide`), and ranges of cached tokens, as many as fill the GPU with them.
struct TreePlan {
    bool wide;
    int row_tiles, rows_pad, ranges;
};
TreePlan tree_plan(const kvarn_config& c, int drafts, int q_dtype) {
    const int R = drafts * (c.n_q_heads / c.n_kv_heads);
    TreePlan p{R > kPRows && q_dtype == KVARN_BF16, 0, (R + 31) / 32 * 32, 0};
    const int rows = p.wide ? 2 * kPRows : kPRows;
    p.row_tiles = (R + rows - 1) / rows;
    const int ctas = p.wide || q_dtype == KVARN_FP32 ? 1 : 2;   // an SM
    p.ranges = (int)(ctas * current_device_sms() / p.row_tiles);
    return p;
}

size_t tree_ws_bytes(const kvarn_config& c, int32_t batch, int32_t drafts, int32_t) {
    if (batch == 0) return kWsHeader;
    const TreePlan p = tree_plan(c, drafts, KVARN_BF16), q = tree_plan(c, drafts, KVARN_FP32);
    if (p.ranges <= 0 || q.ranges <= 0) return 0;
    const size_t units = (size_t)batch * c.n_kv_heads, ranges = p.ranges > q.ranges ? p.ranges : q.ranges;
    return align256(kWsHeader + units * 2 * sizeof(int32_t)) + (units + ranges) * 33 * p.rows_pad * sizeof(float4);
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
    const size_t need = tree_ws_bytes(c, batch, drafts, max_blocks);
    if (need == 0) return KVARN_ERR_CUDA;
    if (workspace_bytes < need) return KVARN_ERR_WORKSPACE;
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
    const TreePlan plan = tree_plan(c, drafts, q_dtype);
    a.B = c.block_size;
    a.unit_map = (int32_t*)((uint8_t*)workspace + kWsHeader);
    const int64_t units = (int64_t)batch * c.n_kv_heads;
    a.partials = (float4*)((uint8_t*)workspace + align256(kWsHeader + units * 2 * sizeof(int32_t)));
    a.row_tiles = plan.row_tiles;
    a.rows_pad = plan.rows_pad;
    a.ranges = plan.ranges;
    a.late = max_blocks > 0;
    if constexpr (!PACKED) {
        cudaError_t e = max_blocks > 0 ? launch_tree_bf16(a, plan.wide, st) : cudaSuccess;
        if (e != cudaSuccess) return KVARN_ERR_CUDA;
        e = launch_tree_join<false>(a, st);
        return e == cudaSuccess ? KVARN_OK : KVARN_ERR_CUDA;
    }
    const dim3 grid((drafts * a.G + kSimpleRows - 1) / kSimpleRows, c.n_kv_heads, batch);
    const cudaError_t e = dispatch(c, [&](auto b, auto w) {
        return launch_pdl(tree_simple_kernel<decltype(b)::value, decltype(w)::value, PACKED>, grid, 128, 0, st, a);
    });
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
    return tree_ws_bytes(c, batch, drafts, max_blocks_per_seq);
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
