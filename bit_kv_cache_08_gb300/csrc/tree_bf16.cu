// tree_bf16.cu -- drafted queries over the cached tokens of bf16 pages on the
// tensor cores.
//
// The R = drafts * G query rows of a (sequence, kv head) meet the same tokens, so
// that S = Q K^T, P = 2^(scale S - m) and O += P V are matrix products of R rows, and
// the pages are read once for all drafts. A CTA takes a range of tiles of tokens
// (tree.cuh), which may go on from one unit to the next, and leaves a partial (m, l, O) of each
// unit. Three forms:
//   NT 1  up to 128 rows and 64-token tiles, two CTAs an SM. HBM bounds it: two CTAs cover
//         each other's waits and ends of units. S of a tile runs under the softmax of the
//         tile before (two S in tensor memory, one O).
//   NT 2  up to 256 rows and 128-token tiles, a CTA an SM. The tensor core bounds it (three products
//         of 256 rows for 512 bytes a token): two row tiles share the keys and
//         values in shared memory and take turns, one in its products while the other is
//         in its softmax; products of 128 tokens read shared memory at the rate of the tensor core,
//         those of 64 do not.
//   extra NT 1, with up to 8 rows more on mma.sync by 4 warps of their own from the same tiles: a second
//         row tile costs as many products for 4 rows (33 drafts) as for 128.
// Per row tile:
//   S (128 rows, fp32)  tensor memory
//   softmax             128 threads, a row each; P as two bf16 halves over S, the A operand of
//   O (128 x 128 fp32)  tensor memory; V straight from its page rows
// Warps: 4 a row tile for the softmax, one that issues the products, one that copies pages (a tile copy
// per page and 64-channel half, swizzled; two stages each of K and V), across the
// units' borders: the next unit's pages are on their way while this one's result is
// stored and the next queries are loaded.
//
// Measured (8 kv heads, 4 query heads each, up to 8192 cached tokens a sequence, alone and cold): 16 x 16
// drafts 68 us for 393 MB (5.8 TB/s, 0.85 of a copy), 32 x 33 with extra rows 172 us for 808 MB (4.7 TB/s: extra
// rows and tcgen05 products share the tensor cores), 200 to 215 as two row tiles.
//
// Rounding: as in the shared prefix over bf16 pages (P two halves, 2^-16; an fp32
// query two, one more product).
#include "prefix_merge.cuh"
#include "tree.cuh"

#include <cuda.h>

namespace kvarn {

cudaError_t bf16_page_map(CUtensorMap* map, const uint8_t* pool, int64_t n_pool_blocks, int n_kv, int block_size);

constexpr int kTbQ = kPRows * kD * 2;        // bytes of a 128 x 128 query operand

struct TreeBf16Smem {
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_ready[2], v_clean[2], o_full[2], q_full, drained;
    uint32_t tmem;
    int stop;
};
constexpr int kTbHeader = 1024;
static_assert(sizeof(TreeBf16Smem) <= kTbHeader, "header");

template <bool Q32, int NT, bool EXTRA>
struct TreeBf16Form {
    static_assert(!Q32 || NT == 1, "an fp32 query is two operands");
    static_assert(!EXTRA || (!Q32 && NT == 1), "extra rows of bf16 queries beside one row tile");
    static constexpr int kExtra = EXTRA ? 4 : 0;                // warps
    static constexpr int kTok = 64 * NT, kKv = kTok * kD * 2;   // tokens of a tile, bytes of its K or V: two 64-channel blocks
    static constexpr int kSoft = 4 * NT, kThreads = 32 * (kSoft + 2 + kExtra);
    static constexpr int kQ = (Q32 ? 2 : 1) * NT * kTbQ;
    static constexpr uint32_t kColumns = 256 * NT;              // of tensor memory: two S, and NT O
    static constexpr size_t kSmem = 1024 + kTbHeader + kQ + 4 * kKv;
};

// The rows from 128 on (up to 8) of a range's units, on mma.sync by 4 warps from the tiles in shared memory:
// warp e takes tokens 32 (e / 2) .. + 31 of a tile and, of O, channels 64 (e % 2) .. + 63. What each half of
// the tokens gives is a partial of its own (the join adds them). The rows are the products' 8 columns:
//   S' = K Q'    A = 16 tokens of K by ldmatrix, B = the rows' queries, in registers
//   O' += V' P'  A = 16 channels of V by ldmatrix.trans, B = S' as two bf16 halves, transposed by movmatrix
__device__ __forceinline__ void ldmatrix4(uint32_t at, uint32_t (&x)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];" : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t at, uint32_t (&x)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];" : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
template <int TOK>
__device__ __forceinline__ void tree_extra_rows(const TreeArgs& a, TreeBf16Smem& s, TreeCursor c, const uint8_t* k_op, const uint8_t* v_op,
                                                int64_t range, int total, int e, int lane, int* stop) {
    static_assert(TOK == 64 && kExtraRows == 8, "two halves of 32 tokens, blocks of 64 channels with rows of 128 bytes");
    constexpr int kKv = TOK * kD * 2;
    const int gq = lane >> 2, tq = lane & 3, token0 = 32 * (e >> 1), block = e & 1;
    const float scale = a.sm_scale * kLog2e;
    int g = 0, cleaned = 0;
    bool ok = true;
    while (g < total && ok) {
        const int n = min(c.tiles - c.t, total - g), rows = tree_rows(a, c.b) * a.G;
        const bool cut = c.tokens % TOK != 0 && c.t + n == c.tiles;
        uint32_t q[8][2];                                // B fragments of 16 channels: row gq
        {
            const int row = kPRows + gq;
            const uint32_t* src = reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(a.q) +
                                                                    (((int64_t)c.b * a.drafts + row / a.G) * a.n_q + c.h * a.G + row % a.G) * kD);
#pragma unroll
            for (int k = 0; k < 8; ++k)
#pragma unroll
                for (int i = 0; i < 2; ++i) q[k][i] = row < rows ? src[8 * k + 4 * i + tq] : 0u;
        }
        // of rows 2 tq + x: channels 16 j + gq (o[j][x]) and + 8 (o[j][2 + x])
        float o[4][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        for (int i = 0; i < n && ok; ++i, ++g) {
            const int st = g & 1, shown = c.tokens - (c.t + i) * TOK - token0;   // tokens of this half that there are
            ok = warp_wait_or_stop(&s.k_full[st], (g >> 1) & 1, stop, kWaitLimit);
            if (!ok) break;
            float sc[2][4];                              // [16 tokens][token gq: rows 2 tq, 2 tq + 1; token gq + 8]
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                sc[t][0] = sc[t][1] = sc[t][2] = sc[t][3] = 0.f;
#pragma unroll
                for (int k = 0; k < 8; ++k) {            // matrices: tokens 0, 8 of the first 8 channels, of the others
                    uint32_t x[4];
                    ldmatrix4(smem_addr(k_op + st * kKv + (k >> 2) * (kKv / 2) +
                                        swizzled(token0 + 16 * t + 8 * (lane >> 3 & 1) + (lane & 7), 2 * (k & 3) + (lane >> 4))), x);
                    mma_bf16(sc[t], x[0], x[1], x[2], x[3], q[k][0], q[k][1]);
                }
            }
            warp_arrive(&s.k_empty[st]);
            float f[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                float top = -INFINITY;
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float& z = sc[t][2 * j + x];
                        z = 16 * t + 8 * j + gq < shown ? z * scale : -INFINITY;
                        top = fmaxf(top, z);
                    }
#pragma unroll
                for (int k = 4; k < 32; k <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, k));
                const bool grow = top - m[x] > 8.f;      // (from -inf at once; false where nothing is shown)
                f[x] = grow && m[x] != -INFINITY ? ex2(m[x] - top) : 1.f;
                if (grow) m[x] = top;
                const float off = m[x] == -INFINITY ? 0.f : m[x];
                float sum = 0.f;
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int j = 0; j < 2; ++j) sum += sc[t][2 * j + x] = ex2(sc[t][2 * j + x] - off);
                l[x] = l[x] * f[x] + sum;
            }
            if (__any_sync(kFull, f[0] != 1.f || f[1] != 1.f))
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    o[j][0] *= f[0];
                    o[j][1] *= f[1];
                    o[j][2] *= f[0];
                    o[j][3] *= f[1];
                }
            uint32_t p[2][2][2];                         // [16 tokens][half][8 tokens]: row gq, tokens 2 tq, 2 tq + 1
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    split_pair<false>(sc[t][2 * j], sc[t][2 * j + 1], p[t][0][j], p[t][1][j]);
                    p[t][0][j] = transposed(p[t][0][j]);
                    p[t][1][j] = transposed(p[t][1][j]);
                }
            ok = warp_wait_or_stop(&s.v_full[st], (g >> 1) & 1, stop, kWaitLimit);
            if (ok && cut && i == n - 1) ok = warp_wait_or_stop(&s.v_clean[st], cleaned >> st & 1, stop, kWaitLimit);
            if (!ok) break;
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j) {            // matrices: channels 0, 8 of the first 8 tokens, of the others
                    uint32_t x[4];
                    ldmatrix4_trans(smem_addr(v_op + st * kKv + block * (kKv / 2) +
                                              swizzled(token0 + 16 * t + 8 * (lane >> 4) + (lane & 7), 2 * j + (lane >> 3 & 1))), x);
                    mma_bf16(o[j], x[0], x[1], x[2], x[3], p[t][0][0], p[t][0][1]);
                    mma_bf16(o[j], x[0], x[1], x[2], x[3], p[t][1][0], p[t][1][1]);
                }
            warp_arrive(&s.v_empty[st]);
        }
        if (!ok) break;
        if (cut) cleaned ^= 1 << (g - 1 & 1);
        const int64_t slot = (int64_t)c.b * a.n_kv + c.h + range;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
#pragma unroll
            for (int k = 4; k < 32; k <<= 1) l[x] += __shfl_xor_sync(kFull, l[x], k);
            if (kPRows + 2 * tq + x >= rows) continue;
            const int row = kPRows + 2 * tq + x + kExtraRows * (e >> 1);
            if (block == 0 && gq == 0) *tree_partial(a, slot, 0, row) = make_float4(m[x], l[x], 0.f, 0.f);
#pragma unroll
            for (int j = 0; j < 8; ++j)                  // channels 64 block + 8 j + gq
                reinterpret_cast<float*>(tree_partial(a, slot, 1 + 16 * block + 2 * j + (gq >> 2), row))[gq & 3] = o[j >> 1][2 * (j & 1) + x];
        }
        if (g < total) tree_next<TOK, false>(a, c);
    }
}

template <int B, bool Q32, int NT, bool EXTRA>
__global__ void __launch_bounds__(TreeBf16Form<Q32, NT, EXTRA>::kThreads, Q32 || NT == 2 ? 1 : 2) tree_bf16_kernel(const __grid_constant__ CUtensorMap map, TreeArgs a) {
    wait_prior_grids();
    let_next_grid_start();   // the join
    using Form = TreeBf16Form<Q32, NT, EXTRA>;
    constexpr int TOK = Form::kTok, kKv = Form::kKv, kSoft = Form::kSoft;
    extern __shared__ uint8_t raw[];
    uint8_t* base = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);   // the swizzle's period
    TreeBf16Smem& s = *reinterpret_cast<TreeBf16Smem*>(base);
    uint8_t* q_op = base + kTbHeader;
    uint8_t* k_op = q_op + Form::kQ;
    uint8_t* v_op = k_op + 2 * kKv;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rt = blockIdx.x % a.row_tiles;
    const int64_t range = blockIdx.x / a.row_tiles;

    TreeCursor c = {};
    const int64_t W = tree_locate<TOK, false>(a, -1, lane, c), n_ranges = tree_ranges(W, a.ranges);
    if (range >= n_ranges) return;
    const int64_t x_beg = range * W / n_ranges;
    const int total = (int)((range + 1) * W / n_ranges - x_beg);   // tiles of this CTA
    tree_locate<TOK, false>(a, x_beg, lane, c);

    if (tid == 0) {
        s.stop = 0;
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.k_full[i], 1);
            mbar_init(&s.k_empty[i], 1 + Form::kExtra);
            mbar_init(&s.v_full[i], 1);
            mbar_init(&s.v_empty[i], 1 + Form::kExtra);
            mbar_init(&s.s_full[i], 1);
            mbar_init(&s.p_ready[i], 4);
            mbar_init(&s.v_clean[i], 1);
            mbar_init(&s.o_full[i], 1);
        }
        mbar_init(&s.q_full, kSoft);
        mbar_init(&s.drained, 1);
        fence_mbar_init();
    }
    if (warp == kSoft) tmem_alloc(&s.tmem, Form::kColumns);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // S (and P) at + TOK w: of tile g, w = g % 2 (NT 1), of row tile w (NT 2); O of a row tile at + 128
    const uint32_t tm_s = __reduce_max_sync(kFull, s.tmem), tm_o = tm_s + 2 * TOK;   // (uniform to the compiler)
    int* stop = &s.stop;
    int issued_k = 0, issued_v = 0;                      // tiles whose copies have been issued
    int g = 0;                                           // tiles of this CTA so far: stage g % 2, phase g / 2
    bool ok = true;

    if (warp == kSoft + 1) {
        // ---------------------------------------------------------- page copies
        // Keys of tile g + 2 right behind the values of tile g: what S(g) and the
        // product of P(g - 2), issued together, set free. (Keys and values of one tile
        // together had the keys wait for the values' stage: 64 x 16 drafts over 8K 342 us a call, 268 so.)
        constexpr int PPT = TOK / B;                // pages per tile
        struct {
            TreeCursor c;
            int held, held0;                             // lane i holds page held0 + i of the sequence
        } at[2] = {{c, -1, -32}, {c, -1, -32}};
        for (int step = 0; step < total + 2 && ok; ++step) {
#pragma unroll
            for (int kind = 1; kind >= 0; --kind) {      // V of tile step - 2, K of tile step
                const int i = kind ? step - 2 : step, st = i & 1;
                if (i < 0 || i >= total || !ok) continue;
                auto& me = at[kind];
                const int first = me.c.t * PPT, used = (me.c.tokens + B - 1) / B;   // pages: of the tile; that hold a token
                if (first >= me.held0 + 32) {            // (32 is a multiple of PPT, and so is every `first`)
                    me.held0 = first;
                    me.held = first + lane < used ? a.table[(int64_t)me.c.b * a.max_blocks + first + lane] : -1;
                    if (first + lane < used && (me.held < 0 || me.held >= a.n_pool_blocks)) {
                        raise_error(a.err, KVARN_DEVERR_BLOCK_ID);
                        me.held = -1;
                    }
                }
                const int p = lane >> 1, half = lane & 1;
                int page = __shfl_sync(kFull, me.held, (first - me.held0 + p) & 31);
                if (p >= PPT) page = -1;                 // (a page behind the end is -1 too)
                const uint32_t bytes = __popc(__ballot_sync(kFull, page >= 0)) * (B * 128);
                const int y = (int)(((int64_t)max(page, 0) * a.n_kv + me.c.h) * 2 * B);
                uint64_t* full = kind ? &s.v_full[st] : &s.k_full[st];
                if (i >= 2) ok = warp_wait_or_stop(kind ? &s.v_empty[st] : &s.k_empty[st], ((i >> 1) - 1) & 1, stop, kWaitLimit);
                if (!ok) break;
                if (lane == 0) mbar_arrive_expect_tx(full, bytes);
                __syncwarp();
                if (page >= 0)
                    tile_g2s((kind ? v_op : k_op) + st * kKv + half * (kKv / 2) + p * B * 128, &map, 64 * half, y + kind * B, full);
                __syncwarp();
                (kind ? issued_v : issued_k) = i + 1;
                // value rows behind the sequence's end: a weight of 0 times whatever the
                // page or an earlier tile holds must be 0
                const int valid = me.c.tokens - me.c.t * TOK;
                if (kind && valid < TOK) {
                    ok = warp_wait_or_stop(&s.v_full[st], (i >> 1) & 1, stop, kWaitLimit);
                    for (int r = valid * 8 + lane; r < TOK * 8; r += 32)
                        for (int k = 0; k < 2; ++k)
                            *reinterpret_cast<uint4*>(v_op + st * kKv + k * (kKv / 2) + r * 16) = make_uint4(0, 0, 0, 0);
                    fence_async_smem();
                    warp_arrive(&s.v_clean[st]);
                }
                if (++me.c.t == me.c.tiles && i + 1 < total) {
                    tree_next<TOK, false>(a, me.c);
                    me.held0 = -32;
                }
            }
        }
    } else if (EXTRA && warp > kSoft + 1) {
        // ---------------------------------------------------------- extra rows
        if constexpr (EXTRA) tree_extra_rows<TOK>(a, s, c, k_op, v_op, range, total, warp - (kSoft + 2), lane, stop);
    } else if (warp == kSoft) {
        // ---------------------------------------------------------- products
        constexpr uint32_t kQk = mma_shape(kMmaBf16, TOK, false), kPv = mma_shape(kMmaBf16, kD, true);
        const uint32_t q_desc = smem_operand(smem_addr(q_op), 16), k_desc = smem_operand(smem_addr(k_op), 16);
        const uint32_t v_desc = smem_operand(smem_addr(v_op), kKv / 2);
        int units = 0, cleaned = 0;                      // (cleaned: bit w, the phase of v_clean[w])
        ok = !(a.flags & KVARN_FLAG_TEST_WAIT_TIMEOUT);
        if (!ok && lane == 0) *stop = 1;                 // (test switch: as if the first wait had run out)
        while (g < total && ok) {
            // (through a warp reduction, whose result the compiler knows to be the same in
            // all lanes: a product's operands then stay in uniform registers)
            const int n = __reduce_min_sync(kFull, min(c.tiles - c.t, total - g));
            const bool cut = c.tokens % TOK != 0 && c.t + n == c.tiles;   // the last tile has rows behind the end
            ok = warp_wait_or_stop(&s.q_full, units & 1, stop, kWaitLimit);
            // O (+)= P V of step i - 2, then S = Q K^T of step i; a step is a tile (NT 1) or a
            // row tile of one, the second behind the first (NT 2)
            for (int i = 0; i < NT * n + 2 && ok; ++i) {
                const int j = i - 2, ti = g + i / NT, tj = g + (NT == 2 ? (i >> 1) - 1 : j);   // (tiles)
                const int w = NT == 2 ? i & 1 : ti & 1, x = NT == 2 ? w : 0;
                const bool lead = NT == 1 || w == 0, trail = NT == 1 || w == 1;
                if (j >= 0) {
                    if (lead) {
                        ok = ok && warp_wait_or_stop(&s.v_full[tj & 1], (tj >> 1) & 1, stop, kWaitLimit);
                        if (ok && cut && tj == g + n - 1) ok = warp_wait_or_stop(&s.v_clean[tj & 1], cleaned >> (tj & 1) & 1, stop, kWaitLimit);
                    }
                    ok = ok && warp_wait_or_stop(&s.p_ready[w], (NT == 2 ? tj : tj >> 1) & 1, stop, kWaitLimit);
                }
                if (!ok) break;
                if (j >= 0) {
                    tc_fence_after();
                    const uint32_t vd = v_desc + (tj & 1) * (kKv >> 4);
#pragma unroll
                    for (int k = 0; k < NT; ++k)          // 64 tokens
                        run_pv_bf16(tm_o + 128 * x, tm_s + TOK * w + 64 * k, vd + k * (8192 >> 4), kPv, j >= NT || k > 0);
                    if (trail) mma_commit(&s.v_empty[tj & 1]);
                    if (tj == g + n - 1) mma_commit(&s.o_full[x]);
                }
                // (the keys' wait comes behind the products that do not need them)
                if (i < NT * n && lead) ok = warp_wait_or_stop(&s.k_full[ti & 1], (ti >> 1) & 1, stop, kWaitLimit);
                if (!ok) break;
                tc_fence_after();
                if (i < NT * n) {
                    const uint32_t kd = k_desc + (ti & 1) * (kKv >> 4);
                    run_qk_bf16<kKv / 2>(tm_s + TOK * w, q_desc + x * (kTbQ >> 4), kd, kQk, false);
                    if (Q32) run_qk_bf16<kKv / 2>(tm_s + TOK * w, q_desc + (kTbQ >> 4), kd, kQk, true);   // (the low halves)
                    mma_commit(&s.s_full[w]);
                    if (trail) mma_commit(&s.k_empty[ti & 1]);
                }
            }
            if (cut) cleaned ^= 1 << (g + n - 1 & 1);
            g += n;
            ++units;
            if (g < total) tree_next<TOK, false>(a, c);
        }
        // products in flight end before the operands and tensor memory go
        mma_commit(&s.drained);
        if (!mbar_wait_bounded(&s.drained, 0, kWaitLimit)) *stop = 1;
    } else {
        // ---------------------------------------------------------- softmax
        const int x = warp >> 2;                         // row tile of the CTA
        const int r = rt * NT * kPRows + tid;            // this thread's query row of a unit
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t my_o = tm_o + 128 * x + lanes;
        const float scale = a.sm_scale * kLog2e;
        int units = 0;
        for (; g < total && ok; ++units) {
            const int n = min(c.tiles - c.t, total - g);
            const int rows = tree_rows(a, c.b) * a.G;
            const bool valid = r < rows, some = __any_sync(kFull, valid);
            // the query rows as a swizzled operand (rows behind the last draft: zeros):
            // a warp takes its own 32, two at a time, 8 channels a lane
            constexpr int kBatch = Q32 ? 4 : 8;
#pragma unroll 1
            for (int i0 = 0; i0 < 16; i0 += kBatch) {
                uint4 v0[kBatch], v1[Q32 ? kBatch : 1];
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const int row = rt * NT * kPRows + warp * 32 + 2 * (i0 + i) + (lane >> 4);
                    v0[i] = make_uint4(0, 0, 0, 0);
                    if (Q32) v1[i] = v0[i];
                    if (row < rows) {
                        const int64_t at = (((int64_t)c.b * a.drafts + row / a.G) * a.n_q + c.h * a.G + row % a.G) * kD + 8 * (lane & 15);
                        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.q) + at * (Q32 ? 4 : 2));
                        v0[i] = src[0];
                        if (Q32) v1[i] = src[1];
                    }
                }
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const int u = lane & 15;
                    uint8_t* dst = q_op + x * kTbQ + (u >> 3) * (kTbQ / 2) + swizzled((warp & 3) * 32 + 2 * (i0 + i) + (lane >> 4), u & 7);
                    if (Q32) {
                        const uint32_t f[8] = {v0[i].x, v0[i].y, v0[i].z, v0[i].w, v1[i].x, v1[i].y, v1[i].z, v1[i].w};
                        uint32_t hi[4], lo[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            split_pair<false>(__uint_as_float(f[2 * k]), __uint_as_float(f[2 * k + 1]), hi[k], lo[k]);
                        *reinterpret_cast<uint4*>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                        *reinterpret_cast<uint4*>(dst + kTbQ) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                    } else {
                        *reinterpret_cast<uint4*>(dst) = v0[i];
                    }
                }
            }
            fence_async_smem();
            tc_fence_before();                           // (the last unit's O has been read)
            warp_arrive(&s.q_full);
            RowState st{-INFINITY, 0.f};
            const int len = valid ? c.tokens : 0;
            for (int i = 0; i < n; ++i, ++g) {
                const int w = NT == 2 ? x : g & 1;
                ok = warp_wait_or_stop(&s.s_full[w], (NT == 2 ? g : g >> 1) & 1, stop, kWaitLimit);
                if (!ok) break;
                tc_fence_after();
                if (!some) {                             // (rows that nothing reads)
                    warp_arrive(&s.p_ready[w]);
                    continue;
                }
                ok = softmax_tile<TOK, EXTRA ? 32 : TOK, false>(tm_s + TOK * w + lanes, my_o, len - (c.t + i) * TOK, scale, 0.f, 1.f, 0.f, i == 0, st,
                                                   &s.p_ready[w], [&] {
                    // O is idle once the last product into it has completed: with two row
                    // tiles S came behind it, with one it has freed tile g - 1's values
                    if (NT == 2) return true;
                    const bool idle = warp_wait_or_stop(&s.v_empty[(g - 1) & 1], ((g - 1) >> 1) & 1, stop, kWaitLimit);
                    tc_fence_after();
                    return idle;
                });
                if (!ok) break;
            }
            // (the row tile's products are over: O is complete, its query's memory free)
            ok = ok && warp_wait_or_stop(&s.o_full[x], units & 1, stop, kWaitLimit);
            if (!ok) break;
            tc_fence_after();
            const int64_t u = (int64_t)c.b * a.n_kv + c.h;
            if (some) tree_store(a, u + range, r, valid, st.m, st.l, my_o);
            if (rt == 0 && tid == 0) {
                if (c.t == 0) a.unit_map[2 * u] = (int)range;
                if (c.t + n == c.tiles) a.unit_map[2 * u + 1] = (int)range;
            }
            if (g < total) tree_next<TOK, false>(a, c);
        }
        tc_fence_before();
    }
    __syncthreads();
    if (*stop) {   // a wait ran out: copies in flight land before the CTA ends
        if (tid == 0) raise_error(a.err, KVARN_DEVERR_WAIT_TIMEOUT);
        if (warp == kSoft + 1) {
            for (int i = max(0, issued_k - 2); i < issued_k; ++i) mbar_wait_bounded(&s.k_full[i & 1], (i >> 1) & 1, kWaitLimit);
            for (int i = max(0, issued_v - 2); i < issued_v; ++i) mbar_wait_bounded(&s.v_full[i & 1], (i >> 1) & 1, kWaitLimit);
        }
        __syncthreads();
    }
    if (warp == kSoft) {
        tc_fence_after();
        tmem_free(s.tmem, Form::kColumns);
    }
}

// ---------------------------------------------------------------- host side
namespace {

template <int B, bool Q32, int NT, bool EXTRA = false>
cudaError_t launch_tree_bf16_as(const CUtensorMap& map, const TreeArgs& a, cudaStream_t st) {
    using Form = TreeBf16Form<Q32, NT, EXTRA>;
    const auto fn = tree_bf16_kernel<B, Q32, NT, EXTRA>;
    static bool ready[64];
    int d = 0;
    cudaError_t e = cudaGetDevice(&d);
    if (e != cudaSuccess) return e;
    if (d < 0 || d >= 64) return cudaErrorInvalidDevice;
    if (!ready[d]) {
        e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Form::kSmem);
        if (e != cudaSuccess) return e;
        ready[d] = true;
    }
    return launch_pdl(fn, a.ranges * a.row_tiles, Form::kThreads, Form::kSmem, st, map, a);
}
template <int B>
cudaError_t launch_tree_bf16_block(const CUtensorMap& map, const TreeArgs& a, bool wide, cudaStream_t st) {
    return a.q_dtype == KVARN_FP32 ? launch_tree_bf16_as<B, true, 1>(map, a, st)
           : wide                  ? launch_tree_bf16_as<B, false, 2>(map, a, st)
           : a.extra               ? launch_tree_bf16_as<B, false, 1, true>(map, a, st)
                                   : launch_tree_bf16_as<B, false, 1>(map, a, st);
}

}  // namespace

cudaError_t launch_tree_bf16(const TreeArgs& a, bool wide, cudaStream_t st) {
    CUtensorMap map;
    const cudaError_t e = bf16_page_map(&map, a.pool, a.n_pool_blocks, a.n_kv, a.B);
    if (e != cudaSuccess) return e;
    return a.B == 32 ? launch_tree_bf16_block<32>(map, a, wide, st) : launch_tree_bf16_block<64>(map, a, wide, st);
}

}  // namespace kvarn
