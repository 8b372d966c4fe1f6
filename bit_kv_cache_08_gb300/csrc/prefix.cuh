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
    float* partials;             // [splits][batch * n_q][kPartialStride]
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

}  // namespace kvarn
