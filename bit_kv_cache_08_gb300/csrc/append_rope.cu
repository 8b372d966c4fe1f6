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
// memory for prompts and latency for a decode step. 32 760 prompt tokens of 48
// rows (805 MB) into bf16 pages take 128 us, 0.93 of the measured copy
// bandwidth, with 4 rows a half-warp in flight (with 2 and 1 it took 10 and 60
// us more); with few rows a token its lookups and angles weigh more (12 rows:
// 50 us for 201 MB). A decode step of 64 tokens takes 5 us as a graph node, into
// the packed cache 8 where no token completes its block, 14 where one does and
// 36 where all do (2 bits, 1024 head-blocks; a CTA per kv head and kind, which
// quantises then). 32 760 prompt tokens into the packed cache take 526 us.
#include "attn_common.cuh"
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

__device__ __forceinline__ void load_weight(const uint16_t* w, const RopeLane& p, float (&v)[8]) {
    if (!w) return;
    unpack_bf4(*reinterpret_cast<const uint2*>(w + p.c0), v);
    unpack_bf4(*reinterpret_cast<const uint2*>(w + p.c1), v + 4);
}

// A loaded row normed (where there is a weight) and rotated.
__device__ __forceinline__ void turn_row(const uint2 (&u)[2], const RopeLane& p, bool norm, const float (&w)[8], float eps,
                                         float (&x)[8]) {
    unpack_bf4(u[0], x);
    unpack_bf4(u[1], x + 4);
    if (norm) head_norm(x, w, eps);
    rope_apply(p, x);
}

__device__ __forceinline__ void store_row(uint16_t* row, const RopeLane& p, const float (&x)[8]) {
    *reinterpret_cast<uint2*>(row + p.c0) = pack_bf4(x);
    *reinterpret_cast<uint2*>(row + p.c1) = pack_bf4(x + 4);
}
__device__ __forceinline__ void store_q(const RopeAppendArgs& a, int64_t row, const RopeLane& p, const float (&x)[8]) {
    if (a.q_out_fp32) {
        float* out = static_cast<float*>(a.q_out) + row * kD;
        *reinterpret_cast<float4*>(out + p.c0) = make_float4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<float4*>(out + p.c1) = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        store_row(static_cast<uint16_t*>(a.q_out) + row * kD, p, x);
    }
}

// A ragged sequence whose tokens cannot all be placed: offsets that descend or
// leave the token rows, or tokens beyond the block table. None of them is.
__device__ __forceinline__ bool bad_sequence(const RopeAppendArgs& a, int b, int64_t capacity) {
    const int64_t c0 = a.cu[b], c1 = a.cu[b + 1], p = a.pos[b];
    return c0 < 0 || c1 < c0 || c1 > a.n_tokens || (c1 > c0 && (p < 0 || p + (c1 - c0) > capacity));
}

// The sequence of token row t: the number of ends cu[1 .. batch] at or before
// t, counted by the warp (32-way search, then one round over what is left).
// -1 for a row outside every sequence (also where offsets around it descend).
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
    return c0 >= 0 && c0 <= t && t < a.cu[b + 1] ? b : -1;
}

// ---------------------------------------------------------------- bf16 pages
// One warp per (token, run): the run-th part of the token's query, key and
// value rows.
constexpr int kRowBatch = 4;
template <int B>
__global__ void __launch_bounds__(128) append_rope_bf16_kernel(RopeAppendArgs a, const __grid_constant__ kvarn_rope r,
                                                               uint32_t runs) {
    __shared__ uint64_t turns[64];
    copy_turns(r, turns);
    __syncthreads();
    wait_prior_grids();
    const int lane = threadIdx.x & 31;
    // (items and heads * runs stay below 2^32: the host's bounds)
    const uint32_t item = blockIdx.x * 4 + (threadIdx.x >> 5), run = runs == 1 ? 0u : item % runs;
    const int64_t t = runs == 1 ? item : item / runs, capacity = (int64_t)a.max_blocks * B;
    if (a.cu)   // the grid's threads look at every sequence, with rows here or not
        for (int64_t x = blockIdx.x * 128ll + threadIdx.x; x < a.batch; x += gridDim.x * 128ll)
            if (bad_sequence(a, (int)x, capacity)) raise_error(a.err, KVARN_DEVERR_POSITION);
    if (t >= a.n_tokens) return;
    const int b = sequence_of(a, t, lane);
    if (b < 0) return;
    const int64_t i = a.cu ? t - a.cu[b] : 0;
    const int64_t at = (int64_t)a.pos[b] + i;
    if (a.cu) {
        if (bad_sequence(a, b, capacity)) return;
    } else if (a.pos[b] < 0 || at >= capacity) {
        if (lane == 0) raise_error(a.err, KVARN_DEVERR_POSITION);
        return;
    }
    const int64_t phys = a.block_table[(int64_t)b * a.max_blocks + at / B];
    const bool ok = phys >= 0 && phys < a.n_pool_blocks;
    if (!ok && lane == 0) raise_error(a.err, KVARN_DEVERR_BLOCK_ID);
    const int half = lane >> 4;
    const RopeLane rl = rope_lane(r, turns, (a.rope_pos ? (int64_t)a.rope_pos[b] : (int64_t)a.pos[b]) + i, lane & 15);
    float qw[8], kw[8];
    load_weight(a.q_weight, rl, qw);
    load_weight(a.k_weight, rl, kw);
    uint16_t* page = reinterpret_cast<uint16_t*>(a.pool + phys * a.block_bytes) + (at % B) * kD;
    // the half-warps take the rows of a kind in turn, kRowBatch each at a time;
    // all loads of a batch are in flight (and in place they come before its stores)
    auto rows_of = [&](int heads, const uint16_t* src, auto&& put) {
        const int h0 = runs == 1 ? 0 : heads * run / runs, h1 = runs == 1 ? heads : heads * (run + 1) / runs;
        for (int j0 = h0; j0 < h1; j0 += 2 * kRowBatch) {
            uint2 u[kRowBatch][2];
#pragma unroll
            for (int k = 0; k < kRowBatch; ++k)   // (a half without a row repeats the last: the norm's shuffles need it)
                load_row(src + (int64_t)min(j0 + 2 * k + half, h1 - 1) * kD, rl, u[k]);
#pragma unroll
            for (int k = 0; k < kRowBatch; ++k)
                if (j0 + 2 * k < h1) put(u[k], j0 + 2 * k + half, j0 + 2 * k + half < h1);
        }
    };
    if (a.q)
        rows_of(a.n_q, a.q + t * a.q_stride, [&](const uint2 (&u)[2], int j, bool real) {
            float x[8];
            turn_row(u, rl, a.q_weight != nullptr, qw, r.eps, x);
            if (real) store_q(a, t * a.n_q + j, rl, x);
        });
    rows_of(a.n_kv, a.k + t * a.k_stride, [&](const uint2 (&u)[2], int j, bool real) {
        float x[8];
        turn_row(u, rl, a.k_weight != nullptr, kw, r.eps, x);
        if (real && ok) store_row(page + (int64_t)(2 * j) * B * kD, rl, x);
    });
    rows_of(a.n_kv, a.v + t * a.v_stride, [&](const uint2 (&u)[2], int j, bool real) {
        if (!real || !ok) return;
        uint16_t* row = page + (int64_t)(2 * j + 1) * B * kD;
        *reinterpret_cast<uint2*>(row + rl.c0) = u[0];
        *reinterpret_cast<uint2*>(row + rl.c1) = u[1];
    });
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
            wrong = bad_sequence(a, b, (int64_t)a.max_blocks * B);
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
// head y (of a decode step: with the keys). A unit that completes its block quantises it (rows before `pos`
// from staging); another one writes staging rows. Where a sequence's first
// block takes staged rows and its last block stays incomplete, one CTA does
// both, the last block's staging rows after the first block has been read.
template <int B, int BITS>
__global__ void __launch_bounds__(quant_threads<B>(), B == 64 ? 2 : 3) append_rope_kernel(RopeAppendArgs a,
                                                                            const __grid_constant__ kvarn_rope r,
                                                                            QuantParams p) {
    __shared__ uint64_t turns[64];
    copy_turns(r, turns);
    __syncthreads();
    wait_prior_grids();
    __shared__ QuantSmem<B, BITS> q;
    __shared__ __align__(16) uint16_t tile[B * kD];   // the completed block's rows
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
    const int hw = tid >> 4, l = tid & 15;                      // half-warp, lane in it
    constexpr int kHalves = 2 * quant_warps<B>();
    const RopeLane groups = rope_lane(r, turns, 0, l);                 // (for the channel groups)
    float w[8];

    if (a.q && (kind == 2 || (kind == 0 && !a.cu))) {           // (a decode step's few query rows ride with the keys)
        const int G = a.n_q / a.n_kv, rows = (int)(hi - lo) * G;
        load_weight(a.q_weight, groups, w);
        for (int x0 = 0; x0 < rows; x0 += kHalves) {
            if (x0 + (hw & ~1) >= rows) break;                  // (whole warps)
            const int x = min(x0 + hw, rows - 1), g = x % G;
            const int64_t at = lo + x / G, t = t0 + (at - pos);
            const RopeLane rl = rope_lane(r, turns, turn0 + at, l);
            uint2 u[2];
            load_row(a.q + t * a.q_stride + (int64_t)(h * G + g) * kD, rl, u);
            float v[8];
            turn_row(u, rl, a.q_weight != nullptr, w, r.eps, v);
            if (x0 + hw < rows) store_q(a, t * a.n_q + h * G + g, rl, v);
        }
        if (kind == 2) return;
    }

    uint16_t* stage = a.staging + (((int64_t)b * a.n_kv + h) * 2 + kind) * B * kD;
    if (kind == 0) load_weight(a.k_weight, groups, w);
    // new rows of positions from .. to - 1, rounded to bf16, to row (position % B) of dst
    auto new_rows = [&](int64_t from, int64_t to, uint16_t* dst) {
        const int rows = (int)(to - from);
        for (int x0 = 0; x0 < rows; x0 += kHalves) {
            if (x0 + (hw & ~1) >= rows) break;                  // (whole warps)
            const int64_t at = from + min(x0 + hw, rows - 1), t = t0 + (at - pos);
            uint16_t* row = dst + (at % B) * kD;
            uint2 u[2];
            if (kind == 1) {
                load_row(a.v + t * a.v_stride + (int64_t)h * kD, groups, u);
                if (x0 + hw < rows) {
                    *reinterpret_cast<uint2*>(row + groups.c0) = u[0];
                    *reinterpret_cast<uint2*>(row + groups.c1) = u[1];
                }
            } else {
                const RopeLane rl = rope_lane(r, turns, turn0 + at, l);
                load_row(a.k + t * a.k_stride + (int64_t)h * kD, rl, u);
                float v[8];
                turn_row(u, rl, a.k_weight != nullptr, w, r.eps, v);
                if (x0 + hw < rows) store_row(row, rl, v);
            }
        }
    };
    if (hi < (blk + 1) * B) {   // the block stays incomplete
        if (j == 0 || pos % B == 0) new_rows(lo, hi, stage);
        return;
    }
    const int64_t phys = a.block_table[(int64_t)b * a.max_blocks + blk];
    const bool ok = phys >= 0 && phys < a.n_pool_blocks;
    if (!ok && tid == 0) raise_error(a.err, KVARN_DEVERR_BLOCK_ID);
    p.kind = kind;
    zero_code_words<B, BITS>(q, tid);
    new_rows(lo, hi, tile);
    for (int64_t x = blk * B + warp; x < lo; x += quant_warps<B>())
        reinterpret_cast<uint2*>(tile + (x % B) * kD)[lane] = reinterpret_cast<const uint2*>(stage + (x % B) * kD)[lane];
    __syncthreads();
    float x[kRowsPerWarp][4];
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kRowsPerWarp; ++i) {
        unpack_bf4(reinterpret_cast<const uint2*>(tile + (warp * kRowsPerWarp + i) * kD)[lane], x[i]);
#pragma unroll
        for (int c = 0; c < 4; ++c) bad |= !isfinite(x[i][c]);
    }
    if (__syncthreads_or(bad) && tid == 0) raise_error(a.err, KVARN_DEVERR_NONFINITE);
    if (ok) {
        quantize_tile<B, BITS>(x, p, q, warp, lane);
        store_image<B, BITS>(q, a.pool + phys * a.block_bytes + (int64_t)(2 * h + kind) * head_block_bytes(B, BITS), tid);
    }
    // the staged rows of this block have been read (the barriers above)
    if (j == 0 && pos % B != 0 && end % B != 0 && end / B > blk) new_rows(end / B * B, end, stage);
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

// The fraction of rate / (2 pi) in units of 2^-64, to the nearest: 1 / (2 pi)
// as the sum of two doubles (a relative 2^-108), its product with the rate as
// the rounded one with the first, that one's exact remainder and the small one
// with the second, so that whole turns of a large rate take no bits of the rest.
uint64_t turns_of(double rate) {
    // (volatile: the product is rounded before the remainder, on every host)
    const volatile double turns = rate * 0x1.45f306dc9c883p-3;
    const double rest = fma(rate, 0x1.45f306dc9c883p-3, -turns) - rate * 0x1.6b01ec5417056p-57;
    const double f = turns - floor(turns);                                 // exact, in [0, 1)
    const double hi = floor(f * 0x1p32), lo = (f * 0x1p32 - hi) * 0x1p32;   // exact
    // (rest is below 2^-35 of a turn; the sum wraps at a whole one)
    return ((uint64_t)hi << 32) + (uint64_t)(int64_t)floor(lo + rest * 0x1p64 + 0.5);
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
        r.turns[i] = turns_of(fabs(inv_freq[i]));
        if (inv_freq[i] < 0) r.turns[i] = 0 - r.turns[i];
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
    // a warp of its own for every 4 rows of a token, fewer where the tokens alone
    // give 16 warps to an SM: each looks the token's place up and makes its angles
    // (as a graph, 1407 tokens of 60 rows: 15.0, 9.3, 8.5, 8.5 and 10.1 us with 64,
    // 20, 16, 12 and 8)
    const int64_t rows = c.n_q_heads + 2 * (int64_t)c.n_kv_heads, warps = current_device_sms() * 16;
    int64_t runs = (warps + n_tokens - 1) / n_tokens, most = (rows + 3) / 4;
    if (most * rows > 0xffffffffll) most = 0xffffffffll / rows;
    runs = runs < most ? runs : most;
    runs = runs > 1 ? runs : 1;
    const unsigned grid = (unsigned)((n_tokens * runs + 3) / 4);
    const cudaError_t e = c.block_size == 32
                              ? launch_pdl(append_rope_bf16_kernel<32>, grid, 128, 0, (cudaStream_t)stream, a, *rope, (uint32_t)runs)
                              : launch_pdl(append_rope_bf16_kernel<64>, grid, 128, 0, (cudaStream_t)stream, a, *rope, (uint32_t)runs);
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
    const dim3 grid((unsigned)units, c.n_kv_heads, q && cu_tokens ? 3 : 2);
    const cudaError_t e = dispatch(c, [&](auto b, auto w) {
        constexpr int B = decltype(b)::value, BITS = decltype(w)::value;
        return launch_pdl(append_rope_kernel<B, BITS>, grid, quant_threads<B>(), 0, (cudaStream_t)stream, a, *rope, p);
    });
    return e == cudaSuccess ? KVARN_OK : KVARN_ERR_CUDA;
}

}  // extern "C"
