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
    float4* partials;            // see tree_partial
    int32_t* unit_map;           // (first, last) range of each unit
    uint16_t* turned;            // packed cache: the rotated queries, two fp16 halves, and their scales
    float* turned_scale;
    int64_t n_pool_blocks, block_bytes, k_stride, v_stride;
    int q_dtype, out_bf16;
    int max_blocks, B, batch, drafts, words;
    int n_q, n_kv, G;
    int row_tiles, rows_pad;     // CTAs that share a unit's query rows; the rows, to a multiple of 32
    int ranges;                  // that the tiles of all units are cut into, at most
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

// Partials: [slot][33][rows_pad] of four floats, (m, l, -, -) and then four channels at a
// time: a warp's 32 rows of four channels are one run of memory for the kernel that
// writes them, a row a thread, and 8 rows of them for the join, which holds them as
// fragments of a product.
__device__ __forceinline__ float4* tree_partial(const TreeArgs& a, int64_t slot, int quad, int row) {
    return a.partials + (slot * 33 + quad) * a.rows_pad + row;
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
