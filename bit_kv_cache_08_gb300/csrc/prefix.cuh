// prefix.cuh -- what the shared-prefix kernels over bf16 pages and over the
// packed cache share: their arguments, and the softmax of one tensor-core tile.
#pragma once
#include "attn_common.cuh"
#include "tcgen05.cuh"

namespace kvarn {

constexpr int kPRows = 128;   // query rows of a tensor-core tile

struct PrefixArgs {
    const void* q;
    const uint8_t* pool;
    const int32_t* table;        // physical blocks of the prefix
    const int32_t* lens;         // prefix tokens each sequence sees
    float* partials;             // see partial_row
    uint32_t* err;
    int64_t n_pool_blocks, block_bytes;
    int q_dtype;
    int n_blocks;                // of the prefix
    int batch, n_q, n_kv, G;
    int splits;
    float sm_scale;
    uint32_t flags;
    uint32_t sb[4];
};

// The prefix tokens sequence b sees; a length outside [0, max_len] (flagged by
// the merge) sees none.
__device__ __forceinline__ int prefix_len(const int32_t* lens, int b, int max_len) {
    const int L = lens[b];
    return L < 0 || L > max_len ? 0 : L;
}

// The most any sequence sees (warp-cooperative).
__device__ __forceinline__ int prefix_most(const PrefixArgs& a, int max_len, int lane) {
    int most = 0;
    for (int b = lane; b < a.batch; b += 32) most = max(most, prefix_len(a.lens, b, max_len));
    return __reduce_max_sync(kFull, most);
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Bytes of the 128-byte-swizzled K-major operand row r, 16-byte unit u (0..7),
// within its 64-element column block.
__device__ __forceinline__ uint32_t swizzled(int r, int u) { return (uint32_t)(r * 128 + ((u ^ (r & 7)) << 4)); }

// a b + c with 16-bit a and b (the low or the high half of a register) and
// fp32 c: the product is exact, the sum rounds once.
__device__ __forceinline__ float fma_half(uint32_t a, uint32_t b, float c, bool high_a, bool high_b) {
    const uint16_t x = high_a ? (uint16_t)(a >> 16) : (uint16_t)a, y = high_b ? (uint16_t)(b >> 16) : (uint16_t)b;
    float d;
    asm("fma.rn.f32.f16 %0, %1, %2, %3;" : "=f"(d) : "h"(x), "h"(y), "f"(c));
    return d;
}
// c - a for a bf16 a.
__device__ __forceinline__ float minus_bf16(uint32_t a, float c, bool high) {
    const uint16_t x = high ? (uint16_t)(a >> 16) : (uint16_t)a;
    float d;
    asm("fma.rn.f32.bf16 %0, %1, %2, %3;" : "=f"(d) : "h"(x), "h"((uint16_t)0xbf80), "f"(c));
    return d;
}

// Two fp32 values as pairs of 16-bit halves, hi = RN(x) and lo = RN(x - hi):
// together within 2^-16 (bf16) or 2^-22 (HALF: fp16, normal halves) of x.
template <bool HALF>
__device__ __forceinline__ void split_pair(float x, float y, uint32_t& hi, uint32_t& lo) {
    if (HALF) {
        hi = pack_h2(x, y);
        lo = pack_h2(fma_half(hi, 0xbc00u, x, false, false), fma_half(hi, 0xbc00u, y, true, false));
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        hi = *reinterpret_cast<const uint32_t*>(&h);
        const __nv_bfloat162 l = __floats2bfloat162_rn(minus_bf16(hi, x, false), minus_bf16(hi, y, true));
        lo = *reinterpret_cast<const uint32_t*>(&l);
    }
}

// P in the tensor memory of S: a weight's two halves take the place of its
// score, so 16 columns of S become 8 of high and 8 of low halves.
constexpr uint32_t kPLow = 8;

// One thread's row of an online softmax (everything in the log2 domain): the
// reference m that P and O are relative to, and the sum l.
struct RowState {
    float m, l;
};

// The softmax of a TOK-token tile by the 128 threads of a stream, a row each:
// reads S (fp32) at my_s, writes P (two 16-bit halves, HALF: fp16, else bf16)
// over it, and rescales O at my_o. A weight is 2^(scale s + bias - m + lift):
// bias is the tile's value exponent (V is stored times 2^-bias), lift a
// constant that keeps small fp16 weights out of the subnormals. The reference
// grows only past 2^8 of what is there, so P stays within 2^(8 + lift) and O is
// seldom touched; o_idle() waits until no product writes O (false: gave up).
// `shown`: tokens of the tile that this row sees. The caller waits for S
// before; each of the stream's 4 warps arrives on p_ready.
// S stays in registers (CHUNK = TOK) or is read twice, CHUNK columns at a
// time, where the kernel has too few of them.
template <int TOK, int CHUNK, bool HALF, typename Idle>
__device__ __forceinline__ bool softmax_tile(uint32_t my_s, uint32_t my_o, int shown, float scale, float bias, float unbias,
                                             float lift, bool first, RowState& st, uint64_t* p_ready, Idle&& o_idle) {
    uint32_t x[CHUNK];
    const bool cut = __any_sync(kFull, shown < TOK);
    auto load = [&](int c0) {
#pragma unroll
        for (int c = 0; c < CHUNK; c += 32) tmem_ld32(my_s + c0 + c, x + c);
        tmem_wait_ld();
        if (cut) {
#pragma unroll
            for (int i = 0; i < CHUNK; ++i)
                if (c0 + i >= shown) x[i] = 0xff800000u;   // -inf, whatever was there
        }
    };
    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int c0 = 0; c0 < TOK; c0 += CHUNK) {
        load(c0);
#pragma unroll
        for (int i = 0; i < CHUNK; i += 2)   // (three-input maxima)
            mx[(i >> 1) & 3] = fmaxf(fmaxf(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), mx[(i >> 1) & 3]);
    }
    const float top = fmaf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), scale, bias);
    const bool grow = top - st.m > 8.f;            // (from -inf at once; false where nothing is shown)
    if (!first && __any_sync(kFull, grow)) {
        if (!o_idle()) return false;
        const float f = grow && st.m != -INFINITY ? ex2(st.m - top) : 1.f;
        st.l *= f;
#pragma unroll
        for (int c = 0; c < kD; c += 16) {
            uint32_t o[16];
            tmem_ld16(my_o + c, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
            tmem_st16(my_o + c, o);
        }
    }
    if (grow) st.m = top;
    const float off = st.m == -INFINITY ? 0.f : bias + lift - st.m;
    const float2 scale2 = make_float2(scale, scale), off2 = make_float2(off, off);
    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
    for (int c0 = 0; c0 < TOK; c0 += CHUNK) {
        if (CHUNK < TOK) load(c0);
#pragma unroll
        for (int c = 0; c < CHUNK; c += 16) {
            uint32_t y[16];   // high halves, low halves
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
                const float2 e = __ffma2_rn(make_float2(__uint_as_float(x[c + i]), __uint_as_float(x[c + i + 1])), scale2, off2);
                const float2 p = make_float2(ex2(e.x), ex2(e.y));
                sum[(i >> 1) & 1] = __fadd2_rn(sum[(i >> 1) & 1], p);
                split_pair<HALF>(p.x, p.y, y[i >> 1], y[8 + (i >> 1)]);
            }
            tmem_st16(my_s + c0 + c, y);   // (over columns of S that have been read)
        }
    }
    tmem_wait_st();
    tc_fence_before();
    warp_arrive(p_ready);
    st.l += ((sum[0].x + sum[0].y) + (sum[1].x + sum[1].y)) * unbias;
    return true;
}

// Partials are laid out [slot][kv head][batch * G rows][kPartialStride], so
// that a warp's 32 rows are one run of memory.
__host__ __device__ __forceinline__ int64_t partial_row(int64_t slot, int n_kv, int h, int64_t R, int64_t row) {
    return ((slot * n_kv + h) * R + row) * kPartialStride;
}

// A warp's 32 rows of a stream's result (m in the log2 domain, l, O) as the
// merge's partials: each thread writes its row to shared memory (the 528-byte
// pitch keeps the 16-byte stores apart in the banks) and one bulk copy takes
// the rows that exist; straight from the threads, rows 528 bytes apart, the
// stores took 2-5 us. `stage`: 32 * 528 bytes of the warp's own, not read by
// products any more. An empty stream's O is zero.
__device__ __forceinline__ void store_partials(const PrefixArgs& a, int slot, int row0, int h, uint8_t* stage, bool empty,
                                               float m, float l, uint32_t my_o, int lane) {
    float* mine = reinterpret_cast<float*>(stage) + lane * kPartialStride;
    *reinterpret_cast<float4*>(mine) = make_float4(m, l, 0.f, 0.f);
#pragma unroll
    for (int c = 0; c < kD; c += 32) {
        uint32_t o[32];
        if (empty) {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = 0u;
        } else {
            tmem_ld32(my_o + c, o);
            tmem_wait_ld();
        }
#pragma unroll
        for (int i = 0; i < 32; i += 4)
            *reinterpret_cast<uint4*>(mine + 4 + c + i) = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
    }
    fence_async_smem();
    __syncwarp();
    const int64_t R = (int64_t)a.batch * a.G;
    const int rows = (int)min((int64_t)32, R - row0);
    if (lane == 0 && rows > 0) {
        bulk_s2g(a.partials + partial_row(slot, a.n_kv, h, R, row0), stage, (uint32_t)rows * kPartialStride * 4);
        bulk_store_wait();
    }
    __syncwarp();
}

}  // namespace kvarn
