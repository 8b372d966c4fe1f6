// tree.cuh -- what the kernels of the attention for a tree of drafted tokens
// share: their arguments, how the cached tokens are cut, and the partials.
#pragma once
#include "prefix.cuh"

namespace kvarn {

struct TreeArgs {
    const void* q;               // [batch][drafts][n_q][128]
    const uint8_t* pool;
    const uint16_t* staging;     // packed cache
    const int32_t* table;
    const int32_t* lens;         // cached tokens
    const uint16_t *k, *v;       // drafted rows, [batch * drafts] of k_stride / v_stride elements
    const uint32_t* mask;        // [batch][drafts][words]
    const int32_t* draft_lens;   // nullptr: drafts
    void* out;
    uint32_t* err;
    float4* partials;            // see tree_partial; of few rows, see few
    int32_t* unit_map;           // (first, last) range of each unit
    uint16_t* turned;            // packed cache: the rotated queries, two fp16 halves, and their scales
    float* turned_scale;
    int64_t n_pool_blocks, block_bytes, k_stride, v_stride;
    int q_dtype, out_bf16;
    int max_blocks, B, batch, drafts, words;
    int n_q, n_kv, G;
    int row_tiles, rows_pad;     // CTAs that share a unit's query rows; the rows, to a multiple of 32
    int ranges;                  // that the tiles of all units are cut into, at most
    int extra;                   // rows 128 .. 135 of bf16 pages have two partials, kExtraRows apart
    int few;                     // > 0: so many partials of each row from the prefill kernel, in its layout
    int late;                    // the join comes behind a kernel of this call
    float sm_scale;
    uint32_t flags;
    uint32_t sb[4];
};

// The drafts of sequence b; -1: a length outside 0 .. drafts (flagged by the join).
__device__ __forceinline__ int tree_rows(const TreeArgs& a, int b) {
    if (a.draft_lens == nullptr) return a.drafts;
    const int T = a.draft_lens[b];
    return T < 0 || T > a.drafts ? -1 : T;
}

// The cached tokens of sequence b that lie in blocks (PACKED: complete ones); 0
// where a length is out of its range or there is no draft to see them.
template <bool PACKED>
__device__ __forceinline__ int tree_tokens(const TreeArgs& a, int b) {
    const int L = a.lens[b];
    if (L < 0 || (int64_t)L > (int64_t)a.max_blocks * a.B || tree_rows(a, b) <= 0) return 0;
    return PACKED ? L / a.B * a.B : L;
}

// A unit is a (sequence, kv head). The tiles (of TOK tokens) of all units lie end to end, sequence by
// sequence, kv head by kv head, and range r of the n in use takes tiles
// [r W / n, (r + 1) W / n) of the W, so that ragged lengths are balanced; a range
// writes a partial for each unit that it touches, in slot unit + range.
struct TreeCursor {
    int b, h, t, tiles, tokens;   // tile t of `tiles`, which hold `tokens`
};
template <int TOK, bool PACKED>
__device__ __forceinline__ void tree_enter(const TreeArgs& a, TreeCursor& c) {
    c.tokens = tree_tokens<PACKED>(a, c.b);
    c.tiles = (c.tokens + TOK - 1) / TOK;
}
// All tiles (warp-cooperative); where x is one of them, c is put there.
template <int TOK, bool PACKED>
__device__ __forceinline__ int64_t tree_locate(const TreeArgs& a, int64_t x, int lane, TreeCursor& c) {
    int64_t before = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 32) {
        const int b = b0 + lane;
        const int64_t mine = b < a.batch ? (int64_t)((tree_tokens<PACKED>(a, b) + TOK - 1) / TOK) * a.n_kv : 0;
        int64_t upto = mine;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const int64_t o = __shfl_up_sync(kFull, upto, m);
            if (lane >= m) upto += o;
        }
        upto += before;
        const uint32_t hit = __ballot_sync(kFull, x >= upto - mine && x < upto);
        if (hit) {
            const int src = __ffs(hit) - 1;
            const int64_t in = x - __shfl_sync(kFull, upto - mine, src);
            c.b = b0 + src;
            tree_enter<TOK, PACKED>(a, c);
            c.h = (int)(in / c.tiles);
            c.t = (int)(in % c.tiles);
        }
        before = __shfl_sync(kFull, upto, 31);
    }
    return before;
}
// The next unit that has tiles (the caller knows that there is one).
template <int TOK, bool PACKED>
__device__ __forceinline__ void tree_next(const TreeArgs& a, TreeCursor& c) {
    c.t = 0;
    if (++c.h < a.n_kv) return;
    c.h = 0;
    do {
        ++c.b;
        tree_enter<TOK, PACKED>(a, c);
    } while (c.tiles == 0);
}
// Ranges in use.
__device__ __forceinline__ int64_t tree_ranges(int64_t W, int ranges) { return W < ranges ? W : ranges; }

// Rows beyond 128 that the bf16 kernel takes beside a row tile (tree_bf16.cu).
constexpr int kExtraRows = 8;

// Partials: [slot][33][rows_pad] of four floats, (m, l, -, -) and then four channels at a
// time: a warp's 32 rows of four channels are one run of memory for the kernel that
// writes them, a row a thread, and 8 rows of them for the join, which holds them as
// fragments of a product.
__device__ __forceinline__ float4* tree_partial(const TreeArgs& a, int64_t slot, int quad, int row) {
    return a.partials + (slot * 33 + quad) * a.rows_pad + row;
}

// softmax_tile (prefix.cuh) with S read from tensor memory twice, 32 columns at a time in
// rolled loops: a fifth of its instructions in memory, for kernels whose warps' code together
// does not fit the instruction caches. The reference moves when a score passes it by 8 and is put kBelow
// below the largest one: weights are at most 2^(8 + lift), and the row's largest is at least
// 2^(lift + kBelow). With a lift of 7 that is 2^11 .. 2^15, and fp16 halves, whose steps end at 2^-24,
// hold every weight within 2^-36 of the row's largest: an output of many small weights beside a large one
// (a first token that takes most of the attention and has next to no value) is made of those. A
// reference above the largest score moves less often (48 x 16 drafts over 8192 4-bit tokens 392 us a call
// at 2^4 above, 397 at the score, 401 so, 407 at 2^6 below), but 2^4 above holds them within 2^-28 alone.
constexpr float kBelow = 4.f;
template <int TOK, bool HALF, typename Idle>
__device__ __forceinline__ bool softmax_rolled(uint32_t my_s, uint32_t my_o, int shown, float scale, float bias, float unbias, float lift,
                                               bool first, RowState& st, uint64_t* p_ready, Idle&& o_idle) {
    const bool cut = __any_sync(kFull, shown < TOK);
    auto load = [&](int c0, uint32_t (&x)[32]) {
        tmem_ld32(my_s + c0, x);
        tmem_wait_ld();
        if (cut) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (c0 + i >= shown) x[i] = 0xff800000u;   // -inf, whatever was there
        }
    };
    float mx = -INFINITY;
#pragma unroll 1
    for (int c0 = 0; c0 < TOK; c0 += 32) {
        uint32_t x[32];
        load(c0, x);
        float y[4] = {mx, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < 32; i += 2)                    // (three-input maxima)
            y[(i >> 1) & 3] = fmaxf(fmaxf(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), y[(i >> 1) & 3]);
        mx = fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3]));
    }
    const float top = fmaf(mx, scale, bias);
    const bool grow = top - st.m > 8.f;                    // (from -inf at once; false where nothing is shown)
    const float ref = top - kBelow;
    if (!first && __any_sync(kFull, grow)) {
        if (!o_idle()) return false;
        const float f = grow && st.m != -INFINITY ? ex2(st.m - ref) : 1.f;
        st.l *= f;
#pragma unroll 1
        for (int c = 0; c < kD; c += 32) {
            uint32_t o[32];
            tmem_ld32(my_o + c, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
            tmem_st32(my_o + c, o);
        }
    }
    if (grow) st.m = ref;
    const float off = st.m == -INFINITY ? 0.f : bias + lift - st.m;
    const float2 scale2 = make_float2(scale, scale), off2 = make_float2(off, off);
    float2 sum = make_float2(0.f, 0.f);
#pragma unroll 1
    for (int c0 = 0; c0 < TOK; c0 += 32) {
        uint32_t x[32];
        load(c0, x);
#pragma unroll
        for (int c = 0; c < 32; c += 16) {
            uint32_t y[16];                                // high halves, low halves
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
                const float2 e = __ffma2_rn(make_float2(__uint_as_float(x[c + i]), __uint_as_float(x[c + i + 1])), scale2, off2);
                const float2 p = make_float2(ex2(e.x), ex2(e.y));
                sum = __fadd2_rn(sum, p);
                split_pair<HALF>(p.x, p.y, y[i >> 1], y[8 + (i >> 1)]);
            }
            tmem_st16(my_s + c0 + c, y);                   // (over columns of S that have been read)
        }
    }
    tmem_wait_st();
    tc_fence_before();
    warp_arrive(p_ready);
    st.l += (sum.x + sum.y) * unbias;
    return true;
}

// ---------------------------------------------------------------- products in runs
// Products of one step as one piece of PTX, for a whole warp with the same operands in all lanes: the lane
// that issues is elected once, and a product costs the additions to its operands alone. (A product at a time,
// each with an election of its own, took 70 to 80 cycles beside busy warps on the same scheduler,
// where the tensor core takes one in 32 to 64.) Operand %0 is the shape, %1 the descriptors' high word.
//   TREE_TS(d, a, +, b, +, p)  [d] (+)= A at tensor memory a + times B at descriptor b +; p: none, one
//   TREE_SS                    the same with A at a descriptor
#define TREE_RUN                                                                                                              \
    "{\n .reg .pred e, none, one;\n .reg .b32 ta, tb;\n .reg .b64 da, db;\n elect.sync _|e, 0xffffffff;\n"                   \
    " setp.ne.u32 none, %2, 0;\n setp.ne.u32 one, 1, 0;\n"
#define TREE_TS(d, a, a_off, b, b_off, p)                                                                                     \
    " add.u32 ta, " a ", " a_off ";\n add.u32 tb, " b ", " b_off ";\n mov.b64 db, {tb, %1};\n"                               \
    " @e tcgen05.mma.cta_group::1.kind::f16 [" d "], [ta], db, %0, " p ";\n"
#define TREE_SS(d, a, a_off, b, b_off, p)                                                                                     \
    " add.u32 ta, " a ", " a_off ";\n add.u32 tb, " b ", " b_off ";\n mov.b64 da, {ta, %1};\n mov.b64 db, {tb, %1};\n"       \
    " @e tcgen05.mma.cta_group::1.kind::f16 [" d "], da, db, %0, " p ";\n"

// S = Q K^T of bf16 tiles: Q and K as 64-channel blocks, BLOCK bytes apart in K.
template <int BLOCK>
__device__ __forceinline__ void run_qk_bf16(uint32_t d, uint32_t q, uint32_t k, uint32_t shape, bool acc) {
    static_assert(BLOCK == 8192 || BLOCK == 16384, "tiles of 64 or 128 tokens");
#define TREE_QK(q_at, k_at, p) TREE_SS("%3", "%4", q_at, "%5", k_at, p)
    if (BLOCK == 8192)
        asm volatile(TREE_RUN TREE_QK("0", "0", "none") TREE_QK("2", "2", "one") TREE_QK("4", "4", "one") TREE_QK("6", "6", "one")
                     TREE_QK("1024", "512", "one") TREE_QK("1026", "514", "one") TREE_QK("1028", "516", "one") TREE_QK("1030", "518", "one") "}\n"
                     ::"r"(shape), "r"(kOperandHigh), "r"((uint32_t)acc), "r"(d), "r"(q), "r"(k) : "memory");
    else
        asm volatile(TREE_RUN TREE_QK("0", "0", "none") TREE_QK("2", "2", "one") TREE_QK("4", "4", "one") TREE_QK("6", "6", "one")
                     TREE_QK("1024", "1024", "one") TREE_QK("1026", "1026", "one") TREE_QK("1028", "1028", "one") TREE_QK("1030", "1030", "one") "}\n"
                     ::"r"(shape), "r"(kOperandHigh), "r"((uint32_t)acc), "r"(d), "r"(q), "r"(k) : "memory");
#undef TREE_QK
}
// O (+)= P V of 64 tokens of bf16 tiles: 16 tokens are 8 columns of each half of P, and 2048 bytes of V's rows.
__device__ __forceinline__ void run_pv_bf16(uint32_t d, uint32_t p, uint32_t v, uint32_t shape, bool acc) {
#define TREE_PV(p_hi, p_lo, v_at, x) TREE_TS("%3", "%4", p_hi, "%5", v_at, x) TREE_TS("%3", "%4", p_lo, "%5", v_at, "one")
    asm volatile(TREE_RUN TREE_PV("0", "8", "0", "none") TREE_PV("16", "24", "128", "one") TREE_PV("32", "40", "256", "one")
                 TREE_PV("48", "56", "384", "one") "}\n"
                 ::"r"(shape), "r"(kOperandHigh), "r"((uint32_t)acc), "r"(d), "r"(p), "r"(v) : "memory");
#undef TREE_PV
    static_assert(kPLow == 8, "the halves of P");
}
// S = Q K'^T of a packed tile: high halves of Q in tensor memory (qh), low ones there too (ql) or, run_qk_packed_low,
// at a descriptor; K' high (kh) and low (kl).
__device__ __forceinline__ void run_qk_packed(uint32_t d, uint32_t qh, uint32_t ql, uint32_t kh, uint32_t kl, uint32_t shape) {
#define TREE_QK(t_at, k_at, x) \
    TREE_TS("%3", "%4", t_at, "%6", k_at, x) TREE_TS("%3", "%5", t_at, "%6", k_at, "one") TREE_TS("%3", "%4", t_at, "%7", k_at, "one")
    asm volatile(TREE_RUN TREE_QK("0", "0", "none") TREE_QK("8", "2", "one") TREE_QK("16", "4", "one") TREE_QK("24", "6", "one")
                 TREE_QK("32", "512", "one") TREE_QK("40", "514", "one") TREE_QK("48", "516", "one") TREE_QK("56", "518", "one") "}\n"
                 ::"r"(shape), "r"(kOperandHigh), "r"(0u), "r"(d), "r"(qh), "r"(ql), "r"(kh), "r"(kl) : "memory");
#undef TREE_QK
}
__device__ __forceinline__ void run_qk_packed_low(uint32_t d, uint32_t qa, uint32_t q, uint32_t kh, uint32_t kl, uint32_t shape) {
#define TREE_QK(t_at, q_at, k_at, x) \
    TREE_TS("%3", "%4", t_at, "%6", k_at, x) TREE_TS("%3", "%4", t_at, "%7", k_at, "one") TREE_SS("%3", "%5", q_at, "%6", k_at, "one")
    asm volatile(TREE_RUN TREE_QK("0", "0", "0", "none") TREE_QK("8", "2", "2", "one") TREE_QK("16", "4", "4", "one") TREE_QK("24", "6", "6", "one")
                 TREE_QK("32", "1024", "512", "one") TREE_QK("40", "1026", "514", "one") TREE_QK("48", "1028", "516", "one")
                 TREE_QK("56", "1030", "518", "one") "}\n"
                 ::"r"(shape), "r"(kOperandHigh), "r"(0u), "r"(d), "r"(qa), "r"(q), "r"(kh), "r"(kl) : "memory");
#undef TREE_QK
}
// O (+)= P V' of a packed tile: V' high (vh) and low (vl).
__device__ __forceinline__ void run_pv_packed(uint32_t d, uint32_t p, uint32_t vh, uint32_t vl, uint32_t shape, bool acc) {
#define TREE_PV(p_hi, p_lo, v_at, x) \
    TREE_TS("%3", "%4", p_hi, "%5", v_at, x) TREE_TS("%3", "%4", p_hi, "%6", v_at, "one") TREE_TS("%3", "%4", p_lo, "%5", v_at, "one")
    asm volatile(TREE_RUN TREE_PV("0", "8", "0", "none") TREE_PV("16", "24", "2", "one") TREE_PV("32", "40", "4", "one")
                 TREE_PV("48", "56", "6", "one") "}\n"
                 ::"r"(shape), "r"(kOperandHigh), "r"((uint32_t)acc), "r"(d), "r"(p), "r"(vh), "r"(vl) : "memory");
#undef TREE_PV
}

// A thread's row of a result (m in the log2 domain, l, O in tensor memory) as a partial.
__device__ __forceinline__ void tree_store(const TreeArgs& a, int64_t slot, int row, bool valid, float m, float l, uint32_t my_o) {
    if (valid) *tree_partial(a, slot, 0, row) = make_float4(m, l, 0.f, 0.f);
#pragma unroll
    for (int c = 0; c < kD; c += 32) {
        uint32_t o[32];
        tmem_ld32(my_o + c, o);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; i += 4)
            if (valid)
                *tree_partial(a, slot, 1 + (c + i) / 4, row) = make_float4(__uint_as_float(o[i]), __uint_as_float(o[i + 1]),
                                                                          __uint_as_float(o[i + 2]), __uint_as_float(o[i + 3]));
    }
}

}  // namespace kvarn
