// append_rope.cu -- a step's keys and values appended to a paged cache with
// the head norms and the rotary position rotation on the way, and the step's
// queries normed and rotated in the same launch: into bf16 pages
// (append_rope_bf16_kernel) or the packed cache with its staging buffer
// (append_rope_kernel).
//
// Per token and head (q and k; v is copied):
//   y = x w / sqrt(mean(x^2) + eps)            (where a norm weight is given)
//   y_a' = y_a cos - y_b sin, y_b' = y_b cos + y_a sin   for every pair (a, b)
// with the angle rope_pos * inv_freq[pair] (rope.cuh), all in fp32, rounded
// once to the output's type. A key is rounded to bf16 before it is staged or
// quantised, so that a block quantised from a prompt holds the same bytes as
// one whose tokens came one by one through the staging buffer.
//
// Bound: every q, k and v row is read and written once (512 bytes a row), so
// memory for prompts and latency for a decode step.
#include "host_checks.h"
#include "quantize.cuh"
#include "rope.cuh"

namespace kvarn {

struct RopeAppendArgs {
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;
    int64_t q_stride, k_stride, v_stride;   // elements from one token's rows to the next's
    const uint16_t* q_weight;
    const uint16_t* k_weight;
    void* q_out;
    int q_out_fp32;
    const int32_t* pos;
    const int32_t* rope_pos;
    const int32_t* cu;        // token offsets of the sequences; nullptr: token b is sequence b's
    int64_t n_tokens;
    int batch;
    int n_q, n_kv;
    uint8_t* pool;
    uint16_t* staging;
    int64_t n_pool_blocks;
    int64_t block_bytes;
    const int32_t* block_table;
    int max_blocks;
    uint32_t* err;
};

__device__ __forceinline__ void load_weight(const uint16_t* w, int lane, float (&v)[4]) {
    if (w) unpack_bf4(reinterpret_cast<const uint2*>(w)[lane], v);
}

__device__ __forceinline__ void store_q(const RopeAppendArgs& a, int64_t row, int lane, const float (&x)[4]) {
    if (a.q_out_fp32)
        reinterpret_cast<float4*>(static_cast<float*>(a.q_out) + row * kD)[lane] = make_float4(x[0], x[1], x[2], x[3]);
    else
        reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.q_out) + row * kD)[lane] = pack_bf4(x);
}

// The sequence of token row t: the number of ends cu[1 .. batch] at or before
// t, counted by the warp (32-way search, then one round over what is left).
// -1 for a row behind the last sequence; -2 where cu is not ascending around t.
__device__ __forceinline__ int sequence_of(const RopeAppendArgs& a, int64_t t, int lane) {
    if (!a.cu) return (int)t;
    int lo = 0, n = a.batch;   // ends lo + 1 .. lo + n are undecided
    while (n > 32) {
        const int step = (n + 31) / 32;
        const int at = min(lo + (lane + 1) * step, lo + n);
        const int below = __popc(__ballot_sync(kFull, a.cu[at] <= t));
        const int skip = min(below * step, n);
        lo += skip;
        n = min(step, n - skip);
    }
    const bool passed = lane < n && a.cu[lo + 1 + lane] <= t;
    const int b = lo + __popc(__ballot_sync(kFull, passed));
    if (b >= a.batch) return -1;
    const int c0 = a.cu[b];
    return c0 >= 0 && c0 <= t && t < a.cu[b + 1] ? b : -2;
}

// ---------------------------------------------------------------- bf16 pages
// One warp per (token, run of `rows` of its n_q + 2 n_kv head rows).
template <int B>
__global__ void __launch_bounds__(128) append_rope_bf16_kernel(RopeAppendArgs a, const __grid_constant__ kvarn_rope r,
                                                               int rows, int runs) {
    wait_prior_grids();
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int64_t t = item / runs;
    if (t >= a.n_tokens) return;
    const int b = sequence_of(a, t, lane);
    if (b < 0) {
        if (b == -2 && lane == 0) raise_error(a.err, KVARN_DEVERR_POSITION);
        return;
    }
    const int64_t i = a.cu ? t - a.cu[b] : 0;
    const int64_t at = (int64_t)a.pos[b] + i;
    if (a.pos[b] < 0 || at >= (int64_t)a.max_blocks * B) {
        if (lane == 0) raise_error(a.err, KVARN_DEVERR_POSITION);
        return;
    }
    const int64_t phys = a.block_table[(int64_t)b * a.max_blocks + at / B];
    const bool ok = phys >= 0 && phys < a.n_pool_blocks;
    if (!ok && lane == 0) raise_error(a.err, KVARN_DEVERR_BLOCK_ID);
    const RopeLane rl = rope_lane(r, (a.rope_pos ? (int64_t)a.rope_pos[b] : (int64_t)a.pos[b]) + i, lane);
    float qw[4], kw[4];
    load_weight(a.q_weight, lane, qw);
    load_weight(a.k_weight, lane, kw);
    uint16_t* page = reinterpret_cast<uint16_t*>(a.pool + phys * a.block_bytes) + (at % B) * kD;
    const int r0 = (int)(item % runs) * rows, r1 = min(r0 + rows, a.n_q + 2 * a.n_kv);
    for (int j = r0; j < r1; ++j) {
        float x[4];
        if (j < a.n_q) {
            if (!a.q) continue;
            unpack_bf4(reinterpret_cast<const uint2*>(a.q + t * a.q_stride + (int64_t)j * kD)[lane], x);
            if (a.q_weight) head_norm(x, qw, r.eps);
            rope_apply(rl, x);
            store_q(a, t * a.n_q + j, lane, x);
        } else if (j < a.n_q + a.n_kv) {
            const int h = j - a.n_q;
            unpack_bf4(reinterpret_cast<const uint2*>(a.k + t * a.k_stride + (int64_t)h * kD)[lane], x);
            if (a.k_weight) head_norm(x, kw, r.eps);
            rope_apply(rl, x);
            if (ok) reinterpret_cast<uint2*>(page + (int64_t)(2 * h) * B * kD)[lane] = pack_bf4(x);
        } else {
            const int h = j - a.n_q - a.n_kv;
            const uint2 u = reinterpret_cast<const uint2*>(a.v + t * a.v_stride + (int64_t)h * kD)[lane];
            if (ok) reinterpret_cast<uint2*>(page + (int64_t)(2 * h + 1) * B * kD)[lane] = u;
        }
    }
}

// ---------------------------------------------------------------- packed cache
// A unit is the part of one sequence's new tokens that falls into one block.
// Unit u of all sequences, warp-cooperative: the sequence (-1: none) and the
// unit's index within it.
template <int B>
__device__ __forceinline__ int unit_of(const RopeAppendArgs& a, int64_t u, int lane, int& j, bool& bad) {
    bad = false;
    if (!a.cu) {
        j = 0;
        return (int)u;
    }
    int64_t before = 0;
    int found = -1;
    for (int b0 = 0; b0 < a.batch && (found < 0 || u == 0); b0 += 32) {   // (unit 0 checks every sequence)
        const int b = b0 + lane;
        int64_t n = 0;
        bool wrong = false;
        if (b < a.batch) {
            const int64_t c0 = a.cu[b], c1 = a.cu[b + 1], p = a.pos[b];
            wrong = c0 < 0 || c1 < c0 || c1 > a.n_tokens || (c1 > c0 && (p < 0 || p + (c1 - c0) > (int64_t)a.max_blocks * B));
            if (!wrong && c1 > c0) n = (p + (c1 - c0) - 1) / B - p / B + 1;
        }
        bad |= __any_sync(kFull, wrong);
        int64_t inc = n;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const int64_t o = __shfl_up_sync(kFull, inc, m);
            if (lane >= m) inc += o;
        }
        const int64_t excl = before + inc - n;
        const uint32_t hit = __ballot_sync(kFull, n > 0 && u >= excl && u < excl + n);
        if (hit) {
            const int src = __ffs(hit) - 1;
            found = b0 + src;
            j = (int)(u - __shfl_sync(kFull, excl, src));
        }
        before += __shfl_sync(kFull, inc, 31);
    }
    return found;
}

// grid (units, n_kv, 2 or 3): z = 0 keys, 1 values, 2 the G query heads of kv
// head y. A unit that completes its block quantises it (rows before `pos`
// from staging); another one writes staging rows. Where a sequence's first
// block takes staged rows and its last block stays incomplete, one CTA does
// both, the last block's staging rows after the first block has been read.
template <int B, int BITS>
__global__ void __launch_bounds__(quant_threads<B>(), B == 64 ? 2 : 3) append_rope_kernel(RopeAppendArgs a,
                                                                            const __grid_constant__ kvarn_rope r,
                                                                            QuantParams p) {
    wait_prior_grids();
    __shared__ QuantSmem<B, BITS> q;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int h = blockIdx.y, kind = blockIdx.z;
    int j;
    bool bad_args;
    const int b = unit_of<B>(a, blockIdx.x, lane, j, bad_args);
    if (bad_args && blockIdx.x == 0 && h == 0 && kind == 0 && tid == 0) raise_error(a.err, KVARN_DEVERR_POSITION);
    if (b < 0) return;
    const int64_t t0 = a.cu ? a.cu[b] : b;                      // the sequence's first token row
    const int64_t pos = a.pos[b];
    const int64_t end = pos + (a.cu ? a.cu[b + 1] - t0 : 1);    // its length after this call
    if (pos < 0 || end > (int64_t)a.max_blocks * B) {           // (decode; unit_of skips such sequences otherwise)
        if (tid == 0 && h == 0 && kind == 0) raise_error(a.err, KVARN_DEVERR_POSITION);
        return;
    }
    const int64_t turn0 = (a.rope_pos ? (int64_t)a.rope_pos[b] : pos) - pos;
    const int64_t blk = pos / B + j;
    const int64_t lo = max(pos, blk * B), hi = min(end, (blk + 1) * B);
    float w[4];

    if (kind == 2) {
        const int G = a.n_q / a.n_kv;
        load_weight(a.q_weight, lane, w);
        for (int64_t x = lo + warp; x < hi; x += quant_warps<B>()) {
            const RopeLane rl = rope_lane(r, turn0 + x, lane);
            const int64_t t = t0 + (x - pos);
            for (int g = 0; g < G; ++g) {
                float v[4];
                unpack_bf4(reinterpret_cast<const uint2*>(a.q + t * a.q_stride + (int64_t)(h * G + g) * kD)[lane], v);
                if (a.q_weight) head_norm(v, w, r.eps);
                rope_apply(rl, v);
                store_q(a, t * a.n_q + h * G + g, lane, v);
            }
        }
        return;
    }

    uint16_t* stage = a.staging + (((int64_t)b * a.n_kv + h) * 2 + kind) * B * kD;
    if (kind == 0) load_weight(a.k_weight, lane, w);
    // the new row of position x (this lane's 4 channels), rounded to bf16
    auto new_row = [&](int64_t x) -> uint2 {
        const int64_t t = t0 + (x - pos);
        if (kind == 1) return reinterpret_cast<const uint2*>(a.v + t * a.v_stride + (int64_t)h * kD)[lane];
        float v[4];
        unpack_bf4(reinterpret_cast<const uint2*>(a.k + t * a.k_stride + (int64_t)h * kD)[lane], v);
        if (a.k_weight) head_norm(v, w, r.eps);
        rope_apply(rope_lane(r, turn0 + x, lane), v);
        return pack_bf4(v);
    };
    auto stage_rows = [&](int64_t from, int64_t to) {
        for (int64_t x = from + warp; x < to; x += quant_warps<B>())
            reinterpret_cast<uint2*>(stage + (x % B) * kD)[lane] = new_row(x);
    };
    if (hi < (blk + 1) * B) {   // the block stays incomplete
        if (j == 0 || pos % B == 0) stage_rows(lo, hi);
        return;
    }
    const int64_t phys = a.block_table[(int64_t)b * a.max_blocks + blk];
    const bool ok = phys >= 0 && phys < a.n_pool_blocks;
    if (!ok && tid == 0) raise_error(a.err, KVARN_DEVERR_BLOCK_ID);
    p.kind = kind;
    zero_code_words<B, BITS>(q, tid);
    float x[kRowsPerWarp][4];
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kRowsPerWarp; ++i) {
        const int64_t at = blk * B + warp * kRowsPerWarp + i;
        unpack_bf4(at < lo ? reinterpret_cast<const uint2*>(stage + (at % B) * kD)[lane] : new_row(at), x[i]);
#pragma unroll
        for (int c = 0; c < 4; ++c) bad |= !isfinite(x[i][c]);
    }
    if (__syncthreads_or(bad) && tid == 0) raise_error(a.err, KVARN_DEVERR_NONFINITE);
    if (ok) {
        quantize_tile<B, BITS>(x, p, q, warp, lane);
        store_image<B, BITS>(q, a.pool + phys * a.block_bytes + (int64_t)(2 * h + kind) * head_block_bytes(B, BITS), tid);
    }
    // the staged rows of this block have been read (the barrier above)
    if (j == 0 && pos % B != 0 && end % B != 0 && end / B > blk) stage_rows(end / B * B, end);
}

// ---------------------------------------------------------------- host side
namespace {

int check_rope(const kvarn_rope* r) {
    if (!r) return KVARN_ERR_INVALID_ARG;
    if (r->rotary_dim < 0 || r->rotary_dim > kD) return KVARN_ERR_INVALID_ARG;
    if (r->rotary_dim % 16) return KVARN_ERR_UNSUPPORTED;
    if (r->layout != KVARN_ROPE_HALF && r->layout != KVARN_ROPE_INTERLEAVED) return KVARN_ERR_INVALID_ARG;
    if (!isfinite(r->scale) || !(r->eps >= 0.0f) || isinf(r->eps)) return KVARN_ERR_INVALID_ARG;
    return KVARN_OK;
}

// Everything but the cache's own buffers; fills the kernels' arguments.
int check_append(const kvarn_config* cfg, const kvarn_rope* rope, void* pool, int64_t n_pool_blocks,
                 const int32_t* block_table, int32_t max_blocks, const int32_t* pos, const int32_t* rope_pos,
                 const int32_t* cu_tokens, int64_t n_tokens, int32_t batch, const void* q, const void* k, const void* v,
                 int64_t q_stride, int64_t k_stride, int64_t v_stride, const void* q_weight, const void* k_weight,
                 void* q_out, int32_t q_out_dtype, void* workspace, kvarn_config* c, RopeAppendArgs* a) {
    int s = check_config(cfg, c);
    if (s != KVARN_OK) return s;
    if ((s = check_rope(rope)) != KVARN_OK) return s;
    if (q_out_dtype != KVARN_BF16 && q_out_dtype != KVARN_FP32) return KVARN_ERR_INVALID_ARG;
    if (batch < 0 || n_tokens < 0 || max_blocks < 0 || n_pool_blocks < 0 || n_pool_blocks > 0x7fffffff)
        return KVARN_ERR_INVALID_ARG;
    if (!cu_tokens && n_tokens != batch) return KVARN_ERR_INVALID_ARG;
    if ((int64_t)max_blocks * c->block_size > 0x7fffffff || c->n_kv_heads > 65535) return KVARN_ERR_INVALID_ARG;
    if (n_tokens > 0x7fffffff / (c->n_q_heads + 2 * (int64_t)c->n_kv_heads)) return KVARN_ERR_INVALID_ARG;
    if (batch == 0 || n_tokens == 0) return KVARN_OK;
    if (!pool || !block_table || !pos || !k || !v || !workspace || (!q != !q_out)) return KVARN_ERR_INVALID_ARG;
    if (!aligned(pool, 16) || !aligned(workspace, 16) || !aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) ||
        !aligned(q_out, 16) || !aligned(q_weight, 16) || !aligned(k_weight, 16) || !aligned(block_table, 4) ||
        !aligned(pos, 4) || !aligned(rope_pos, 4) || !aligned(cu_tokens, 4))
        return KVARN_ERR_INVALID_ARG;
    if (k_stride < (int64_t)c->n_kv_heads * kD || v_stride < (int64_t)c->n_kv_heads * kD || k_stride % 8 || v_stride % 8)
        return KVARN_ERR_INVALID_ARG;
    if (q && (q_stride < (int64_t)c->n_q_heads * kD || q_stride % 8)) return KVARN_ERR_INVALID_ARG;
    *a = {};
    a->q = (const uint16_t*)q;
    a->k = (const uint16_t*)k;
    a->v = (const uint16_t*)v;
    a->q_stride = q_stride;
    a->k_stride = k_stride;
    a->v_stride = v_stride;
    a->q_weight = (const uint16_t*)q_weight;
    a->k_weight = (const uint16_t*)k_weight;
    a->q_out = q_out;
    a->q_out_fp32 = q_out_dtype == KVARN_FP32;
    a->pos = pos;
    a->rope_pos = rope_pos;
    a->cu = cu_tokens;
    a->n_tokens = n_tokens;
    a->batch = batch;
    a->n_q = c->n_q_heads;
    a->n_kv = c->n_kv_heads;
    a->pool = (uint8_t*)pool;
    a->n_pool_blocks = n_pool_blocks;
    a->block_table = block_table;
    a->max_blocks = max_blocks;
    a->err = (uint32_t*)workspace;
    return KVARN_OK;
}

}  // namespace
}  // namespace kvarn

using namespace kvarn;

extern "C" {

int kvarn_rope_init(kvarn_rope* rope, int32_t rotary_dim, int32_t layout, const double* inv_freq, float scale,
                    float eps) {
    if (!rope) return KVARN_ERR_INVALID_ARG;
    kvarn_rope r = {};
    r.rotary_dim = rotary_dim;
    r.layout = layout;
    r.scale = scale;
    r.eps = eps;
    const int s = check_rope(&r);
    if (s != KVARN_OK) return s;
    if (rotary_dim > 0 && !inv_freq) return KVARN_ERR_INVALID_ARG;
    for (int i = 0; i < rotary_dim / 2; ++i) {
        if (!(fabs(inv_freq[i]) <= 1048576.0)) return KVARN_ERR_INVALID_ARG;
        // (volatile: the product is rounded before the difference, on every host)
        const volatile double turns = inv_freq[i] * 0.15915494309189533577;   // 1 / (2 pi): per position
        const double f = turns - floor(turns);                                // exact, in [0, 1]
        // high and low halves: each product and difference below is exact
        const double hi = floor(f * 0x1p32), lo = (f * 0x1p32 - hi) * 0x1p32;
        r.turns[i] = ((uint64_t)hi << 32) + (uint64_t)floor(lo + 0.5);   // (a whole turn wraps to 0)
    }
    *rope = r;
    return KVARN_OK;
}

int kvarn_append_rope_bf16(const kvarn_config* cfg, const kvarn_rope* rope, void* kv_pool, int64_t n_pool_blocks,
                           const int32_t* block_table, int32_t max_blocks_per_seq, const int32_t* pos,
                           const int32_t* rope_pos, const int32_t* cu_tokens, int64_t n_tokens, int32_t batch,
                           const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride,
                           int64_t v_stride, const void* q_weight, const void* k_weight, void* q_out,
                           int32_t q_out_dtype, void* workspace, void* stream) {
    kvarn_config c;
    RopeAppendArgs a;
    const int s = check_append(cfg, rope, kv_pool, n_pool_blocks, block_table, max_blocks_per_seq, pos, rope_pos,
                               cu_tokens, n_tokens, batch, q, k, v, q_stride, k_stride, v_stride, q_weight, k_weight,
                               q_out, q_out_dtype, workspace, &c, &a);
    if (s != KVARN_OK || batch == 0 || n_tokens == 0) return s;
    a.block_bytes = (int64_t)c.n_kv_heads * 2 * c.block_size * kD * 2;
    const int all = c.n_q_heads + 2 * c.n_kv_heads;
    const int rows = n_tokens >= 1024 ? 16 : 4;
    const int runs = (all + rows - 1) / rows;
    const unsigned grid = (unsigned)((n_tokens * runs + 3) / 4);
    const cudaError_t e = c.block_size == 32
                              ? launch_pdl(append_rope_bf16_kernel<32>, grid, 128, 0, (cudaStream_t)stream, a, *rope, rows, runs)
                              : launch_pdl(append_rope_bf16_kernel<64>, grid, 128, 0, (cudaStream_t)stream, a, *rope, rows, runs);
    return e == cudaSuccess ? KVARN_OK : KVARN_ERR_CUDA;
}

int kvarn_append_rope(const kvarn_config* cfg, const kvarn_rope* rope, void* pool, int64_t n_pool_blocks, void* staging,
                      const int32_t* block_table, int32_t max_blocks_per_seq, const int32_t* pos,
                      const int32_t* rope_pos, const int32_t* cu_tokens, int64_t n_tokens, int32_t batch, const void* q,
                      const void* k, const void* v, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                      const void* q_weight, const void* k_weight, void* q_out, int32_t q_out_dtype, void* workspace,
                      void* stream) {
    kvarn_config c;
    RopeAppendArgs a;
    const int s = check_append(cfg, rope, pool, n_pool_blocks, block_table, max_blocks_per_seq, pos, rope_pos, cu_tokens,
                               n_tokens, batch, q, k, v, q_stride, k_stride, v_stride, q_weight, k_weight, q_out,
                               q_out_dtype, workspace, &c, &a);
    if (s != KVARN_OK || batch == 0 || n_tokens == 0) return s;
    if (!staging || !aligned(staging, 16)) return KVARN_ERR_INVALID_ARG;
    a.staging = (uint16_t*)staging;
    a.block_bytes = block_bytes_of(c);
    const QuantParams p = make_params(c, 0);
    // units: a sequence of n tokens touches at most (n + 2 B - 2) / B blocks
    const int64_t units = cu_tokens ? n_tokens / c.block_size + 2 * (int64_t)batch : batch;
    if (units > 0x7fffffff) return KVARN_ERR_INVALID_ARG;
    const dim3 grid((unsigned)units, c.n_kv_heads, q ? 3 : 2);
    const cudaError_t e = dispatch(c, [&](auto b, auto w) {
        constexpr int B = decltype(b)::value, BITS = decltype(w)::value;
        return launch_pdl(append_rope_kernel<B, BITS>, grid, quant_threads<B>(), 0, (cudaStream_t)stream, a, *rope, p);
    });
    return e == cudaSuccess ? KVARN_OK : KVARN_ERR_CUDA;
}

}  // extern "C"
