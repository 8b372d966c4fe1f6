// tree_packed.cu -- drafted queries over the cached tokens of the packed cache on
// the tensor cores: the products of the shared prefix over the packed cache
// (prefix_packed.cu: S = Q K'^T and O += P V' in the rotated space, K', V', P and Q two
// fp16 halves each, three products of halves), for the rows of one sequence's drafts over
// that sequence's blocks, in ranges of tiles that go on from one unit to the next
// (tree.cuh).
//
// tree_rotate_kernel turns the queries once: H (sigma q) / sqrt(128), each row scaled by a
// power of two and split into two fp16 halves. In the main kernel a CTA has one or two
// tiles of 128 rows (NT), which share the built operands; Q's high half lies in tensor memory
// (64 columns a row tile), its low half in shared memory, beside S / P of two steps
// (2 x 64 columns) and O (128 a row tile).
// Warps: 4 a row tile for the softmax, one that issues the products, one that copies raw
// tiles and finds their exponents, 8 that build operands (packed_build.cuh).
#include "packed_build.cuh"
#include "host_checks.h"
#include "quantize.cuh"
#include "tree.cuh"

namespace kvarn {

constexpr int kTreeTopQuery = 14;    // a rotated query's channels up to 2^14

// ---------------------------------------------------------------- queries
// A warp a row: [unit][rows_pad][hi 128 | lo 128] fp16, and what the scores are to be
// multiplied with, 2^e, [unit][rows_pad].
__global__ void __launch_bounds__(256) tree_rotate_kernel(TreeArgs a) {
    wait_prior_grids();
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);   // of [batch][drafts][n_q]
    if (row >= (int64_t)a.batch * a.drafts * a.n_q) return;
    const int hq = (int)(row % a.n_q), r = (int)(row / a.n_q % a.drafts), b = (int)(row / a.n_q / a.drafts);
    if (r >= tree_rows(a, b)) return;
    float v[4];
    load_q4(a.q, a.q_dtype, row, lane, v);
    if (!(a.flags & KVARN_FLAG_NO_ROTATION)) {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] *= sign_of4(a.sb[0], a.sb[1], a.sb[2], a.sb[3], 4 * lane + k);
        fwht128(v, lane);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] *= kInvSqrtD;
    }
    const float big = warp_max(fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3]))));
    const int e = big > 0x1p-100f ? min(ceil_log2(big), 127) : -100;
    const float up = exp2i(kTreeTopQuery - e);
    uint32_t hi[2], lo[2];
    split_pair<true>(v[0] * up, v[1] * up, hi[0], lo[0]);
    split_pair<true>(v[2] * up, v[3] * up, hi[1], lo[1]);
    const int64_t to = ((int64_t)b * a.n_kv + hq / a.G) * a.rows_pad + r * a.G + hq % a.G;
    uint2* dst = reinterpret_cast<uint2*>(a.turned + to * 2 * kD);
    dst[lane] = make_uint2(hi[0], hi[1]);
    dst[32 + lane] = make_uint2(lo[0], lo[1]);
    if (lane == 0) a.turned_scale[to] = exp2i(e - kTreeTopQuery);
}

// ---------------------------------------------------------------- cached tokens
struct TreePackedSmem {
    // ready: a raw tile's exponents are known; raw_empty: its operands are built
    uint64_t raw_full[kMaxRaw], ready[kMaxRaw], raw_empty[kMaxRaw];
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_ready[2], o_full[2], q_full, drained;
    uint32_t tmem;
    int stop;
    // the exponents of the last tiles (see the prefix kernel: at most 6 are in use)
    int kexp[8], vexp[8];
};

template <int B, int BITS, int NT>
struct TreePackedLayout {
    static constexpr int kSoft = 4 * NT, kThreads = 32 * (kSoft + 2 + kBuildWarps);
    static constexpr int HB = head_block_bytes(B, BITS);
    static constexpr int kBlocks = kPkTok / B;                 // blocks per tile
    static constexpr int kRaw = kBlocks * 2 * HB;              // bytes of a raw tile: (K, V) per block
    static constexpr int kHeader = 1024;
    static_assert(sizeof(TreePackedSmem) <= kHeader, "header");
    static constexpr int kFixed = 1024 + kHeader + NT * kPkQ + 4 * kPkK + 4 * kPkV;
    static constexpr int kFit = (227 * 1024 - kFixed) / kRaw;
    static constexpr int kRawStages = kFit < kMaxRaw ? kFit : kMaxRaw;
    static_assert(kRawStages >= 2, "a raw tile in flight while another is built");
    static constexpr size_t bytes = kFixed + kRawStages * kRaw;
};

template <int B, int BITS, int NT>
__global__ void __launch_bounds__(TreePackedLayout<B, BITS, NT>::kThreads, 1) tree_packed_kernel(TreeArgs a) {
    wait_prior_grids();
    let_next_grid_start();   // the join
    using Lay = TreePackedLayout<B, BITS, NT>;
    constexpr int kSoft = Lay::kSoft, kRawStages = Lay::kRawStages, TOK = kPkTok;
    extern __shared__ uint8_t raw_smem[];
    uint8_t* base = raw_smem + ((1024 - (smem_addr(raw_smem) & 1023)) & 1023);
    TreePackedSmem& s = *reinterpret_cast<TreePackedSmem*>(base);
    uint8_t* q_lo = base + Lay::kHeader;          // [row tile]
    uint8_t* k_op = q_lo + NT * kPkQ;             // [stage][hi, lo]
    uint8_t* v_op = k_op + 4 * kPkK;              // [stage][hi, lo]
    uint8_t* raw = v_op + 4 * kPkV;               // [raw stage][block][K, V]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rt = blockIdx.x % a.row_tiles;
    const int64_t range = blockIdx.x / a.row_tiles;

    TreeCursor c = {};
    const int64_t W = tree_locate<TOK, true>(a, -1, lane, c), n_ranges = tree_ranges(W, a.ranges);
    if (range >= n_ranges) return;
    const int64_t x_beg = range * W / n_ranges;
    const int total = (int)((range + 1) * W / n_ranges - x_beg);   // tiles of this CTA
    tree_locate<TOK, true>(a, x_beg, lane, c);

    if (tid == 0) {
        s.stop = 0;
        for (int i = 0; i < kRawStages; ++i) {
            mbar_init(&s.raw_full[i], 1);
            mbar_init(&s.ready[i], 1);
            mbar_init(&s.raw_empty[i], kBuildWarps);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.k_full[i], kBuildWarps);
            mbar_init(&s.k_empty[i], 1);
            mbar_init(&s.v_full[i], kBuildWarps);
            mbar_init(&s.v_empty[i], 1);
            mbar_init(&s.s_full[i], 1);
            mbar_init(&s.p_ready[i], 4);
            mbar_init(&s.o_full[i], 1);
        }
        mbar_init(&s.q_full, kSoft);
        mbar_init(&s.drained, 1);
        fence_mbar_init();
    }
    if (warp == kSoft) tmem_alloc(&s.tmem, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // Q of row tile x at + 64 x; S (and P) at + 64 w, of tile g, w = g % 2 (NT 1), or of row
    // tile w (NT 2); O at + 128 x
    const uint32_t tm_q = s.tmem, tm_s = s.tmem + 128, tm_o = s.tmem + 256;
    int* stop = &s.stop;
    int fetched = 0;                              // raw tiles whose copies have been issued
    int g = 0;                                    // tiles of this CTA so far
    bool ok = true;

    if (warp == kSoft + 1) {
        // ---------------------------------------------------------- raw tiles and their exponents
        TreeCursor f = c;                         // of the copies
        int held = -1, held0 = -32;               // lane i holds block held0 + i of the sequence
        auto fetch = [&] {
            const int st = fetched % kRawStages, first = f.t * Lay::kBlocks, used = f.tokens / B;
            if (first >= held0 + 32) {            // (32 is a multiple of kBlocks, and so is every `first`)
                held0 = first;
                held = first + lane < used ? a.table[(int64_t)f.b * a.max_blocks + first + lane] : -1;
                if (first + lane < used && (held < 0 || held >= a.n_pool_blocks)) {
                    raise_error(a.err, KVARN_DEVERR_BLOCK_ID);
                    held = -1;
                }
            }
            int64_t page = __shfl_sync(kFull, held, (first - held0 + lane) & 31);   // lane x: block x of the tile
            if (lane >= Lay::kBlocks) page = -1;
            const uint32_t bytes = __popc(__ballot_sync(kFull, page >= 0)) * (2 * Lay::HB);
            if (lane == 0) mbar_arrive_expect_tx(&s.raw_full[st], bytes);
            __syncwarp();
            if (page >= 0)
                bulk_g2s(raw + st * Lay::kRaw + lane * 2 * Lay::HB, a.pool + page * a.block_bytes + (int64_t)(2 * f.h) * Lay::HB,
                         2 * Lay::HB, &s.raw_full[st]);
            ++fetched;
            if (++f.t == f.tiles && fetched < total) {
                tree_next<TOK, true>(a, f);
                held0 = -32;
            }
        };
        for (; g < total && ok; ++g) {
            // (one stage less in flight than there are: its wait is for tile g - 2)
            while (fetched < total && fetched < g + kRawStages - 1 && ok) {
                if (fetched >= kRawStages)        // the stage's last tile has been built
                    ok = warp_wait_or_stop(&s.raw_empty[fetched % kRawStages], (fetched / kRawStages - 1) & 1, stop, kWaitLimit);
                if (ok) fetch();
            }
            const int st = g % kRawStages;
            ok = ok && warp_wait_or_stop(&s.raw_full[st], (g / kRawStages) & 1, stop, kWaitLimit);
            if (!ok) break;
            const int x = lane / (32 / Lay::kBlocks);              // this lane's block
            const bool there = c.t * Lay::kBlocks + x < c.tokens / B;
            const uint8_t* hb = raw + st * Lay::kRaw + x * 2 * Lay::HB;
            const int ke = tile_exponent<B, BITS>(hb, there, lane), ve = tile_exponent<B, BITS>(hb + Lay::HB, there, lane);
            if (lane == 0) {
                s.kexp[g & 7] = ke;
                s.vexp[g & 7] = ve;
                mbar_arrive(&s.ready[st]);
            }
            if (++c.t == c.tiles && g + 1 < total) tree_next<TOK, true>(a, c);
        }
    } else if (warp > kSoft) {
        // ---------------------------------------------------------- operands from codes
        // warp bw: group grp of the 32 records of half sb, a record a lane
        const int bw = warp - (kSoft + 2), grp = bw & 3, sb = bw >> 2;
        for (; g < total && ok; ++g) {
            const int st = g % kRawStages, par = g & 1;
            ok = warp_wait_or_stop(&s.ready[st], (g / kRawStages) & 1, stop, kWaitLimit) &&
                 warp_wait_or_stop(&s.raw_full[st], (g / kRawStages) & 1, stop, kWaitLimit);
            if (!ok) break;
            const uint8_t* hb = raw + st * Lay::kRaw + (B == 64 ? 0 : sb) * 2 * Lay::HB;
            const bool there = B == 64 || c.t * Lay::kBlocks + sb < c.tokens / B;   // else its values are zero
            ok = build_keys<B, BITS>(hb, grp, sb, lane, &s.kexp[g & 7], k_op + par * 2 * kPkK, [&] {
                return g < 2 || warp_wait_or_stop(&s.k_empty[par], ((g >> 1) - 1) & 1, stop, kWaitLimit);
            });
            if (!ok) break;
            fence_async_smem();
            warp_arrive(&s.k_full[par]);
            ok = build_values<B, BITS>(hb + Lay::HB, there, grp, sb, lane, &s.vexp[g & 7], v_op + par * 2 * kPkV, [&] {
                return g < 2 || warp_wait_or_stop(&s.v_empty[par], ((g >> 1) - 1) & 1, stop, kWaitLimit);
            });
            if (!ok) break;
            fence_async_smem();
            warp_arrive(&s.v_full[par]);
            warp_arrive(&s.raw_empty[st]);
            if (B != 64 && ++c.t == c.tiles && g + 1 < total) tree_next<TOK, true>(a, c);
        }
    } else if (warp == kSoft) {
        // ---------------------------------------------------------- products
        constexpr uint32_t kQk = mma_shape(kMmaF16, TOK, false), kPv = mma_shape(kMmaF16, kD, false);
        const uint32_t q_desc = smem_operand(smem_addr(q_lo), 16), k_desc = smem_operand(smem_addr(k_op), 16);
        const uint32_t v_desc = smem_operand(smem_addr(v_op), 16);
        int units = 0;
        ok = !(a.flags & KVARN_FLAG_TEST_WAIT_TIMEOUT);
        if (!ok && lane == 0) *stop = 1;          // (test switch: as if the first wait had run out)
        while (g < total && ok) {
            const int n = __reduce_min_sync(kFull, min(c.tiles - c.t, total - g));   // (uniform to the compiler)
            ok = warp_wait_or_stop(&s.q_full, units & 1, stop, kWaitLimit);
            // O (+)= P V' of step i - 2, then S = Q K'^T of step i; a step is a tile (NT 1) or a
            // row tile of one, the second behind the first (NT 2)
            for (int i = 0; i < NT * n + 2 && ok; ++i) {
                const int j = i - 2, ti = g + i / NT, tj = g + (NT == 2 ? (i >> 1) - 1 : j);
                const int w = NT == 2 ? i & 1 : ti & 1, x = NT == 2 ? w : 0;
                const bool lead = NT == 1 || w == 0, trail = NT == 1 || w == 1;
                if (j >= 0) {
                    if (lead) ok = ok && warp_wait_or_stop(&s.v_full[tj & 1], (tj >> 1) & 1, stop, kWaitLimit);
                    ok = ok && warp_wait_or_stop(&s.p_ready[w], (NT == 2 ? tj : tj >> 1) & 1, stop, kWaitLimit);
                }
                if (!ok) break;
                if (j >= 0) {
                    tc_fence_after();
                    const uint32_t p = tm_s + 64 * w, vd = v_desc + (tj & 1) * (2 * kPkV >> 4);
#pragma unroll
                    for (int k = 0; k < TOK / 16; ++k) {          // hi hi, hi lo, lo hi
                        mma_ts(tm_o + 128 * x, p + 16 * k, vd + 2 * k, kPv, j >= NT || k > 0);
                        mma_ts(tm_o + 128 * x, p + 16 * k, vd + (kPkV >> 4) + 2 * k, kPv, true);
                        mma_ts(tm_o + 128 * x, p + 16 * k + kPLow, vd + 2 * k, kPv, true);
                    }
                    if (trail) mma_commit(&s.v_empty[tj & 1]);
                    if (tj == g + n - 1) mma_commit(&s.o_full[x]);
                }
                // (the keys' wait comes behind the products that do not need them)
                if (i < NT * n && lead) ok = warp_wait_or_stop(&s.k_full[ti & 1], (ti >> 1) & 1, stop, kWaitLimit);
                if (!ok) break;
                tc_fence_after();
                if (i < NT * n) {
                    const uint32_t kd = k_desc + (ti & 1) * (2 * kPkK >> 4), qa = tm_q + 64 * x, qd = q_desc + x * (kPkQ >> 4);
#pragma unroll
                    for (int k = 0; k < 24; ++k) {                // hi hi, hi lo, lo hi
                        const uint32_t kb = kd + (((k >> 3) == 1 ? kPkK >> 4 : 0) + (((k >> 2 & 1) * (kPkK / 2) + (k & 3) * 32) >> 4));
                        if (k < 16) mma_ts(tm_s + 64 * w, qa + 8 * (k & 7), kb, kQk, k > 0);
                        else mma_ss(tm_s + 64 * w, qd + (((k >> 2 & 1) * (kPkQ / 2) + (k & 3) * 32) >> 4), kb, kQk, true);
                    }
                    mma_commit(&s.s_full[w]);
                    if (trail) mma_commit(&s.k_empty[ti & 1]);
                }
            }
            g += n;
            ++units;
            if (g < total) tree_next<TOK, true>(a, c);
        }
        // products in flight end before the operands and tensor memory go
        mma_commit(&s.drained);
        if (!mbar_wait_bounded(&s.drained, 0, kWaitLimit)) *stop = 1;
    } else {
        // ---------------------------------------------------------- softmax
        const int x = warp >> 2;                                  // row tile of the CTA
        const int r = rt * NT * kPRows + tid;                     // this thread's query row of a unit
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t my_o = tm_o + 128 * x + lanes;
        int units = 0;
        for (; g < total && ok; ++units) {
            const int n = min(c.tiles - c.t, total - g);
            const bool valid = r < tree_rows(a, c.b) * a.G, some = __any_sync(kFull, valid);
            const int64_t u = (int64_t)c.b * a.n_kv + c.h;
            // the row's two halves (rows behind the last draft: zeros)
            const uint4* src = reinterpret_cast<const uint4*>(a.turned + (u * a.rows_pad + r) * 2 * kD);
#pragma unroll 1
            for (int k = 0; k < 4; ++k) {                         // 32 channels
                uint4 hi[4], lo[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    hi[i] = valid ? src[4 * k + i] : make_uint4(0, 0, 0, 0);
                    lo[i] = valid ? src[16 + 4 * k + i] : make_uint4(0, 0, 0, 0);
                }
                uint32_t y[16];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    y[4 * i] = hi[i].x;
                    y[4 * i + 1] = hi[i].y;
                    y[4 * i + 2] = hi[i].z;
                    y[4 * i + 3] = hi[i].w;
                    const int at = 4 * k + i;
                    *reinterpret_cast<uint4*>(q_lo + x * kPkQ + (at >> 3) * (kPkQ / 2) + swizzled((warp & 3) * 32 + lane, at & 7)) = lo[i];
                }
                tmem_st16(tm_q + 64 * x + 16 * k + lanes, y);
            }
            const float scale = valid ? a.sm_scale * kLog2e * a.turned_scale[u * a.rows_pad + r] : 0.f;
            tmem_wait_st();
            fence_async_smem();
            tc_fence_before();                                    // (the last unit's O has been read)
            warp_arrive(&s.q_full);
            RowState st{-INFINITY, 0.f};
            const int len = valid ? c.tokens : 0;
            for (int i = 0; i < n; ++i, ++g) {
                const int w = NT == 2 ? x : g & 1;
                ok = warp_wait_or_stop(&s.s_full[w], (NT == 2 ? g : g >> 1) & 1, stop, kWaitLimit);
                if (!ok) break;
                tc_fence_after();
                if (!some) {                                      // (rows that nothing reads)
                    warp_arrive(&s.p_ready[w]);
                    continue;
                }
                const int e = *reinterpret_cast<volatile int*>(&s.vexp[g & 7]);
                // (finite and not 0, so that what is masked stays masked)
                const float here = fminf(fmaxf(scale * exp2i(*reinterpret_cast<volatile int*>(&s.kexp[g & 7])), 0x1p-126f), 0x1p127f);
                ok = softmax_tile<TOK, NT == 2 ? 32 : 64, true>(tm_s + 64 * w + lanes, my_o, len - (c.t + i) * TOK, here, (float)e, exp2i(-e),
                                                               kLift, i == 0, st, &s.p_ready[w], [&] {
                    // O is idle once the last product into it has completed: with two row
                    // tiles S came behind it, with one it has freed tile g - 1's V stage
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
            if (some) tree_store(a, u + range, r, valid, st.m - kLift, st.l, my_o);
            if (rt == 0 && tid == 0) {
                if (c.t == 0) a.unit_map[2 * u] = (int)range;
                if (c.t + n == c.tiles) a.unit_map[2 * u + 1] = (int)range;
            }
            if (g < total) tree_next<TOK, true>(a, c);
        }
        tc_fence_before();
    }
    __syncthreads();
    if (*stop) {   // a wait ran out: copies in flight land before the CTA ends
        if (tid == 0) raise_error(a.err, KVARN_DEVERR_WAIT_TIMEOUT);
        if (warp == kSoft + 1)
            for (int i = max(0, fetched - kRawStages); i < fetched; ++i)
                mbar_wait_bounded(&s.raw_full[i % kRawStages], (i / kRawStages) & 1, kWaitLimit);
        __syncthreads();
    }
    if (warp == kSoft) {
        tc_fence_after();
        tmem_free(s.tmem, 512);
    }
}

// ---------------------------------------------------------------- host side
namespace {

template <int B, int BITS, int NT>
cudaError_t launch_tree_packed_as(const TreeArgs& a, cudaStream_t st) {
    using Lay = TreePackedLayout<B, BITS, NT>;
    static_assert(Lay::bytes <= 227 * 1024, "shared memory of one CTA");
    static bool ready[64];
    int d = 0;
    cudaError_t e = cudaGetDevice(&d);
    if (e != cudaSuccess) return e;
    if (d < 0 || d >= 64) return cudaErrorInvalidDevice;
    if (!ready[d]) {
        e = cudaFuncSetAttribute(tree_packed_kernel<B, BITS, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Lay::bytes);
        if (e != cudaSuccess) return e;
        ready[d] = true;
    }
    return launch_pdl(tree_packed_kernel<B, BITS, NT>, a.ranges * a.row_tiles, Lay::kThreads, Lay::bytes, st, a);
}

}  // namespace

cudaError_t launch_tree_packed(const kvarn_config& c, const TreeArgs& a, bool wide, cudaStream_t st) {
    const int64_t rows = (int64_t)a.batch * a.drafts * a.n_q;
    const cudaError_t e = launch_pdl(tree_rotate_kernel, (unsigned)((rows + 7) / 8), 256, 0, st, a);
    if (e != cudaSuccess) return e;
    return dispatch(c, [&](auto b, auto w) {
        constexpr int B = decltype(b)::value, BITS = decltype(w)::value;
        return wide ? launch_tree_packed_as<B, BITS, 2>(a, st) : launch_tree_packed_as<B, BITS, 1>(a, st);
    });
}

}  // namespace kvarn
