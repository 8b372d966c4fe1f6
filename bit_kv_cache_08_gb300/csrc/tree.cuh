// tree.cuh -- what the kernels of the attention for a tree of drafted tokens share.
#pragma once
#include "attn_common.cuh"

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
    int64_t n_pool_blocks, block_bytes, k_stride, v_stride;
    int q_dtype, out_bf16;
    int max_blocks, batch, drafts, words;
    int n_q, n_kv, G;
    float sm_scale;
    uint32_t flags;
    uint32_t sb[4];
};

// The drafts of sequence b; a length outside 0 .. drafts is none (flagged).
__device__ __forceinline__ int tree_rows(const TreeArgs& a, int b) {
    if (a.draft_lens == nullptr) return a.drafts;
    const int T = a.draft_lens[b];
    return T < 0 || T > a.drafts ? -1 : T;
}

}  // namespace kvarn
