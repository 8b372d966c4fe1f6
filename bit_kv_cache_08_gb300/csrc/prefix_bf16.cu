// prefix_bf16.cu -- the shared prefix over bf16 pages on the tensor cores.
//
// Per kv head, R = batch * G query rows meet every prefix token: S = Q K^T,
// P = 2^(scale S - m), O += P V with the running row maximum m and sum l of
// an online softmax. A CTA owns up to 256 rows of one head and a range of
// 128-token tiles, and writes (m, l, O) partials for the merge.
//
// Two streams run through the tensor core in turn, so that one multiplies
// while the other is in its softmax: with more than 128 rows, two row tiles
// over the same K/V tiles; with fewer, one row tile over even and odd K/V
// tiles (their partials are joined at the end). Per stream:
//   S (128 x 128 fp32)   tensor memory; K and Q tiles from shared memory
//   softmax              128 threads, a row each: S to registers, P (two
//                        bf16 halves) back over S in tensor memory as the A
//                        operands of
//   O (128 x 128 fp32)   tensor memory; V straight from its page rows
//                        (contraction across rows, so no transposition)
// O is rescaled only when a row's maximum has grown by more than 2^8 since
// the reference it was accumulated with (P stays within 2^8; the result is
// the same up to rounding).
//
// Warps: 0-3 and 4-7 softmax of the two streams, 8 issues the products, 9
// copies pages (a tile copy per page and 64-channel half, swizzled), two
// stages each of K and V.
//
// Rounding: scores are exact products summed in fp32 (an fp32 query is split
// into two bf16 halves, two products); P is split into two halves of V's type,
// two products, within 2^-16, as the decode attention does. (P rounded to one
// bf16 value left errors of 2^-9 of sum p |v|, for 14 us of 119 at 128 x 32 768.)
//
// Measured (32 query heads on 8 kv heads, 128 channels; alone and cold): 512
// rows a head behind 32 768 tokens in 79 us; its products (34 GFLOP of scores,
// 69 of the two halves of P) at 1.31 PFLOP/s, 0.69 of a library bf16 product;
// 256 rows behind 8192 in 23. The tensor pipe is busy 64 % of the time and HBM
// a quarter: the bound is a step's chain (product, softmax, products and the
// waits between), of which two streams hide the larger part. Timing stand-ins
// of a whole call, with P in one half (119.5 us then): no exponentials 115.6, no
// softmax 109.5, an eighth of the products 111, no pages after the first two
// tiles 119.3. A product warp for each stream (124), half a row a thread (129),
// S read twice in fewer registers (131) and fewer token ranges (132) were slower.
#include "prefix.cuh"

#include <cuda.h>

namespace kvarn {

constexpr int kTileTok = 128;
constexpr int kOperand = kPRows * kD * 2;           // bytes of a 128 x 128 16-bit operand
constexpr int kHalfOperand = kOperand / 2;          // its 64-element column block

struct Bf16Smem {
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_ready[2], o_full[2], v_clean, drained;
    uint32_t tmem;
    int stop;
};
constexpr int kBf16Header = 1024;
static_assert(sizeof(Bf16Smem) <= kBf16Header, "header");
static_assert(8 * 32 * kPartialStride * 4 <= 5 * kOperand, "the partials' staging fits the operands' memory");

// MODE 0: 256 rows; 1: 128 rows; 2: 128 rows, fp32 query in two halves
constexpr int bf16_q_tiles(int mode) { return mode == 1 ? 1 : 2; }
constexpr size_t bf16_prefix_smem(int mode) { return 1024 + kBf16Header + (size_t)(bf16_q_tiles(mode) + 4) * kOperand; }

template <int B, int MODE>
__global__ void __launch_bounds__(320, 1) prefix_bf16_kernel(const __grid_constant__ CUtensorMap map, PrefixArgs a) {
    wait_prior_grids();
    let_next_grid_start();   // the own tokens' split kernel
    extern __shared__ uint8_t raw[];
    // operands on 1024-byte boundaries (the swizzle's period)
    uint8_t* base = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
    Bf16Smem& s = *reinterpret_cast<Bf16Smem*>(base);
    uint8_t* q_op = base + kBf16Header;
    uint8_t* k_op = q_op + bf16_q_tiles(MODE) * kOperand;
    uint8_t* v_op = k_op + 2 * kOperand;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    constexpr int kRowsCta = MODE == 0 ? 2 * kPRows : kPRows;
    const int h = blockIdx.z, R = a.batch * a.G, row0 = blockIdx.y * kRowsCta;
    const int max_len = a.n_blocks * B;

    const int most = prefix_most(a, max_len, lane);
    const int tiles = (most + kTileTok - 1) / kTileTok;
    const int t_beg = (int)((int64_t)tiles * blockIdx.x / a.splits), t_end = (int)((int64_t)tiles * (blockIdx.x + 1) / a.splits);
    const int n = t_end - t_beg;                       // K/V tiles
    const int steps = MODE == 0 ? 2 * n : n;           // (stream, tile) items: stream = step % 2

    if (tid == 0) {
        s.stop = 0;
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.k_full[i], 1);
            mbar_init(&s.k_empty[i], 1);
            mbar_init(&s.v_full[i], 1);
            mbar_init(&s.v_empty[i], 1);
            mbar_init(&s.s_full[i], 1);
            mbar_init(&s.p_ready[i], 4);
            mbar_init(&s.o_full[i], 1);
        }
        mbar_init(&s.v_clean, 1);
        mbar_init(&s.drained, 1);
        fence_mbar_init();
    }
    if (warp == 8) tmem_alloc(&s.tmem, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = s.tmem;
    int* stop = &s.stop;
    const uint32_t tm_s = tm, tm_o = tm + 256;         // S (and P) of stream w at + 128 w, O likewise

    if (warp != 9) {
        // ---- the query rows as swizzled operands (rows behind the batch:
        // zeros), loads in batches, while warp 9 starts on the pages
        constexpr int kBatch = MODE == 2 ? 4 : 8;
        for (int i0 = tid; i0 < kRowsCta * 16; i0 += kBatch * 288) {
            uint4 x[MODE == 2 ? 2 * kBatch : kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const int i = i0 + j * 288, row = row0 + (i >> 4);   // 8-channel unit i % 16 of row i / 16
                const int64_t at = ((int64_t)(row / a.G) * a.n_q + h * a.G + row % a.G) * kD + 8 * (i & 15);
                const bool there = i < kRowsCta * 16 && row < R;
                if (MODE == 2) {
                    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const float*>(a.q) + at);
                    x[2 * j] = there ? src[0] : make_uint4(0, 0, 0, 0);
                    x[2 * j + 1] = there ? src[1] : make_uint4(0, 0, 0, 0);
                } else {
                    x[j] = there ? *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + at) : make_uint4(0, 0, 0, 0);
                }
            }
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const int i = i0 + j * 288, r = i >> 4, u = i & 15;
                if (i >= kRowsCta * 16) break;
                uint8_t* dst = q_op + (r / kPRows) * kOperand + (u >> 3) * kHalfOperand + swizzled(r % kPRows, u & 7);
                if (MODE == 2) {
                    const uint4 lo4 = x[2 * j], hi4 = x[2 * j + 1];
                    const uint32_t f[8] = {lo4.x, lo4.y, lo4.z, lo4.w, hi4.x, hi4.y, hi4.z, hi4.w};
                    uint32_t ph[4], pl[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 v = make_float2(__uint_as_float(f[2 * k]), __uint_as_float(f[2 * k + 1]));
                        const __nv_bfloat162 b = __floats2bfloat162_rn(v.x, v.y);
                        const float2 bf = __bfloat1622float2(b);
                        const __nv_bfloat162 c = __floats2bfloat162_rn(v.x - bf.x, v.y - bf.y);
                        ph[k] = *reinterpret_cast<const uint32_t*>(&b);
                        pl[k] = *reinterpret_cast<const uint32_t*>(&c);
                    }
                    *reinterpret_cast<uint4*>(dst) = make_uint4(ph[0], ph[1], ph[2], ph[3]);
                    *reinterpret_cast<uint4*>(dst + kOperand) = make_uint4(pl[0], pl[1], pl[2], pl[3]);
                } else {
                    *reinterpret_cast<uint4*>(dst) = x[j];
                }
            }
        }
        fence_async_smem();
        asm volatile("bar.sync 1, 288;" ::: "memory");
    }

    int done_k = 0, done_v = 0;                        // tiles whose copies warp 9 has issued
    if (warp == 9) {
        // ---------------------------------------------------------- page copies
        constexpr int PPT = kTileTok / B;              // pages per tile
        const int used = (most + B - 1) / B;           // pages that hold a visible token
        bool ok = true;
        for (int i = 0; i < n && ok; ++i) {
            const int t = t_beg + i, st = i & 1;
            int page = -1;
            const int p = lane >> 1, half = lane & 1;  // lanes 0 .. 2 PPT - 1 copy
            if (p < PPT && t * PPT + p < used) {
                page = a.table[t * PPT + p];
                if (page < 0 || page >= a.n_pool_blocks) {
                    raise_error(a.err, KVARN_DEVERR_BLOCK_ID);
                    page = -1;
                }
            }
            const uint32_t bytes = __popc(__ballot_sync(kFull, page >= 0)) * (B * 128);
            const int y = (int)(((int64_t)max(page, 0) * a.n_kv + h) * 2 * B);
            for (int kind = 0; kind < 2; ++kind) {
                uint64_t* full = kind ? &s.v_full[st] : &s.k_full[st];
                if (i >= 2) ok = warp_wait_or_stop(kind ? &s.v_empty[st] : &s.k_empty[st], ((i >> 1) - 1) & 1, stop, kWaitLimit);
                if (!ok) break;
                if (lane == 0) mbar_arrive_expect_tx(full, bytes);
                __syncwarp();
                if (page >= 0)
                    tile_g2s((kind ? v_op : k_op) + st * kOperand + half * kHalfOperand + p * B * 128, &map, 64 * half,
                             y + kind * B, full);
                __syncwarp();
                (kind ? done_v : done_k) = i + 1;
            }
            // value rows behind every sequence's prefix: a weight of 0 times
            // whatever the page or an earlier tile holds must be 0
            const int valid = most - t * kTileTok;
            if (ok && valid < kTileTok) {
                ok = warp_wait_or_stop(&s.v_full[st], (i >> 1) & 1, stop, kWaitLimit);
                for (int x = valid * 8 + lane; x < kTileTok * 8; x += 32)
                    for (int c = 0; c < 2; ++c)
                        *reinterpret_cast<uint4*>(v_op + st * kOperand + c * kHalfOperand + x * 16) = make_uint4(0, 0, 0, 0);
                fence_async_smem();
                warp_arrive(&s.v_clean);
            }
        }
    } else if (warp == 8) {
        // ---------------------------------------------------------- products
        if (steps > 0) {
            constexpr uint32_t kQk = mma_shape(kMmaBf16, kTileTok, false), kPv = mma_shape(kMmaBf16, kD, true);
            const uint32_t q_desc = smem_operand(smem_addr(q_op), 16), k_desc = smem_operand(smem_addr(k_op), 16);
            const uint32_t v_desc = smem_operand(smem_addr(v_op), kHalfOperand);
            bool ok = !(a.flags & KVARN_FLAG_TEST_WAIT_TIMEOUT);
            if (!ok && lane == 0) *stop = 1;                      // (test switch: as if the first wait had run out)
            for (int i = 0; i < steps + 2 && ok; ++i) {           // O (+)= P V of step j, then S = Q K^T of step i
                const int j = i - 2, w = i & 1, tj = MODE == 0 ? j >> 1 : j, ti = MODE == 0 ? i >> 1 : i;
                if (i < steps && (MODE != 0 || w == 0)) ok = warp_wait_or_stop(&s.k_full[ti & 1], (ti >> 1) & 1, stop, kWaitLimit);
                if (j >= 0) {
                    if (MODE != 0 || w == 0) {
                        ok = ok && warp_wait_or_stop(&s.v_full[tj & 1], (tj >> 1) & 1, stop, kWaitLimit);
                        if (ok && most - (t_beg + tj) * kTileTok < kTileTok) ok = warp_wait_or_stop(&s.v_clean, 0, stop, kWaitLimit);
                    }
                    ok = ok && warp_wait_or_stop(&s.p_ready[w], (j >> 1) & 1, stop, kWaitLimit);
                }
                if (!ok) break;
                tc_fence_after();
                if (j >= 0) {
                    const uint32_t p = tm_s + 128 * w, vd = v_desc + (tj & 1) * (kOperand >> 4);
#pragma unroll
                    for (int k = 0; k < kTileTok / 16; ++k) {     // 16 tokens: 8 columns of each half of P, 2048 bytes of V rows
                        mma_ts(tm_o + 128 * w, p + 16 * k, vd + k * (2048 >> 4), kPv, j >= 2 || k > 0);
                        mma_ts(tm_o + 128 * w, p + 16 * k + kPLow, vd + k * (2048 >> 4), kPv, true);
                    }
                    if (MODE != 0 || w == 1) mma_commit(&s.v_empty[tj & 1]);
                    if (j + 2 >= steps) mma_commit(&s.o_full[w]);
                }
                if (i < steps) {
                    const uint32_t qd = q_desc + (MODE == 0 ? w * (kOperand >> 4) : 0), kd = k_desc + (ti & 1) * (kOperand >> 4);
#pragma unroll
                    for (int k = 0; k < (MODE == 2 ? 16 : 8); ++k) {   // (k >= 8: the query's low halves)
                        const uint32_t off = ((k >> 2 & 1) * kHalfOperand + (k & 3) * 32) >> 4;
                        mma_ss(tm_s + 128 * w, qd + (k >> 3) * (kOperand >> 4) + off, kd + off, kQk, k > 0);
                    }
                    mma_commit(&s.s_full[w]);
                    if (MODE != 0 || w == 1) mma_commit(&s.k_empty[ti & 1]);
                }
            }
            // products in flight end before the operands and tensor memory go
            mma_commit(&s.drained);
            if (!mbar_wait_bounded(&s.drained, 0, kWaitLimit)) *stop = 1;
        }
    } else {
        // ---------------------------------------------------------- softmax
        const int w = warp >> 2;                                  // stream
        const int r = (MODE == 0 ? w * kPRows : 0) + (warp & 3) * 32 + lane;
        const int row = row0 + r;
        const int len = row < R ? prefix_len(a.lens, row / a.G, max_len) : 0;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t my_s = tm_s + 128 * w + lanes, my_o = tm_o + 128 * w + lanes;
        const float scale = a.sm_scale * kLog2e;
        RowState st{-INFINITY, 0.f};
        const int items = steps > w ? (steps - w + 1) / 2 : 0;
        bool ok = true;
        for (int j = 0; j < items; ++j) {
            const int t = t_beg + (MODE == 0 ? j : 2 * j + w);
            ok = warp_wait_or_stop(&s.s_full[w], j & 1, stop, kWaitLimit);
            if (!ok) break;
            tc_fence_after();
            // (the products that S waited for include the last one into O)
            softmax_tile<kTileTok, kTileTok, false>(my_s, my_o, len - t * kTileTok, scale, 0.f, 1.f, 0.f, j == 0, st, &s.p_ready[w],
                                          [] { return true; });
        }
        // both streams' products are over before the operands' memory is reused
        for (int x = 0; x < 2 && ok; ++x)
            if (steps > x) ok = warp_wait_or_stop(&s.o_full[x], 0, stop, kWaitLimit);
        tc_fence_after();
        if (ok)
            store_partials(a, MODE == 0 ? blockIdx.x : 2 * blockIdx.x + w, row - lane, h, q_op + warp * 32 * kPartialStride * 4,
                           items == 0, st.m, st.l, my_o, lane);
        tc_fence_before();
    }
    __syncthreads();
    if (*stop) {   // a wait ran out: copies in flight land before the CTA ends
        if (tid == 0) raise_error(a.err, KVARN_DEVERR_WAIT_TIMEOUT);
        if (warp == 9) {
            for (int i = max(0, done_k - 2); i < done_k; ++i) mbar_wait_bounded(&s.k_full[i & 1], (i >> 1) & 1, kWaitLimit);
            for (int i = max(0, done_v - 2); i < done_v; ++i) mbar_wait_bounded(&s.v_full[i & 1], (i >> 1) & 1, kWaitLimit);
        }
        __syncthreads();
    }
    if (warp == 8) {
        tc_fence_after();
        tmem_free(tm, 512);
    }
}

// ---------------------------------------------------------------- host side
namespace {

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's tensor-map encoder, looked up once (a host function: the same for every device).
EncodeTiled encode_tiled() {
    static const EncodeTiled fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            p = nullptr;
        return (EncodeTiled)p;
    }();
    return fn;
}

}  // namespace

// Tile copies of 64 channels of a page's K or V rows of one kv head, 128-byte
// swizzled: rows of 128 channels, page after page, (K, V) of each kv head.
cudaError_t bf16_page_map(CUtensorMap* map, const uint8_t* pool, int64_t n_pool_blocks, int n_kv, int block_size) {
    const EncodeTiled enc = encode_tiled();
    if (!enc) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {(cuuint64_t)kD, (cuuint64_t)n_pool_blocks * n_kv * 2 * block_size};
    const cuuint64_t strides[1] = {kD * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)block_size}, one[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint8_t*>(pool), dims, strides, box, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

namespace {

template <int B, int MODE>
cudaError_t launch_mode(const CUtensorMap& map, const PrefixArgs& p, cudaStream_t st) {
    constexpr int rows = MODE == 0 ? 2 * kPRows : kPRows;
    static bool ready[64];
    int d = 0;
    cudaError_t e = cudaGetDevice(&d);
    if (e != cudaSuccess) return e;
    if (d < 0 || d >= 64) return cudaErrorInvalidDevice;
    if (!ready[d]) {
        e = cudaFuncSetAttribute(prefix_bf16_kernel<B, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)bf16_prefix_smem(MODE));
        if (e != cudaSuccess) return e;
        ready[d] = true;
    }
    const dim3 grid(p.splits, (p.batch * p.G + rows - 1) / rows, p.n_kv);
    return launch_pdl(prefix_bf16_kernel<B, MODE>, grid, 320, bf16_prefix_smem(MODE), st, map, p);
}

}  // namespace

cudaError_t launch_prefix_bf16(const PrefixArgs& p, int block_size, cudaStream_t st) {
    CUtensorMap map;
    const cudaError_t e = bf16_page_map(&map, p.pool, p.n_pool_blocks, p.n_kv, block_size);
    if (e != cudaSuccess) return e;
    const int64_t R = (int64_t)p.batch * p.G;
    const int mode = p.q_dtype == KVARN_FP32 ? 2 : (R > kPRows ? 0 : 1);
    if (block_size == 32)
        return mode == 0 ? launch_mode<32, 0>(map, p, st) : (mode == 1 ? launch_mode<32, 1>(map, p, st) : launch_mode<32, 2>(map, p, st));
    return mode == 0 ? launch_mode<64, 0>(map, p, st) : (mode == 1 ? launch_mode<64, 1>(map, p, st) : launch_mode<64, 2>(map, p, st));
}

}  // namespace kvarn
