// prefix_packed.cu -- the shared prefix over the packed cache on the tensor
// cores: each 64-token tile of codes is turned into 16-bit operands once and
// multiplied with 128 query rows.
//
// Everything runs in the rotated space (the query rows are rotated here, the
// merge rotates back). Per kv head and up to 256 of its batch * G query rows
// (two tiles of 128, which share the built operands), over the CTA's range of
// 64-token tiles:
//   S = Q K'^T (128 x 64, fp32)   K' = (code s + z) R C 2^-k, its largest value
//       at most 2^15, and Q (scaled likewise, a row at a time) are each split
//       into two fp16 halves, and three products (hi hi, hi lo, lo hi) keep
//       2^-22 of each factor: a score is exponentiated, so its error must not
//       grow with the size of the scores (with bf16 halves it was 2^-16 of
//       sum |q k|). The exponents go into the scale of the scores.
//   P = 2^(S - m), O += P V'      P and V' are each split into two fp16 halves,
//       three products (2^-22): V' is (code s + z) R C 2^-e, the tile's exponent
//       e making its largest value at most 2^15, so that the low halves of
//       values down to 2^-18 of it are normal; e enters the exponent of P, so
//       P V' needs no other scale. (One fp16 value each left errors of 2^-12 of
//       sum p |v|, for 23 us of 205 at 128 x 32 768, 4 bits.)
// Tensor memory: Q's high half as the A operand (64 columns a row tile; its
// low half stays in shared memory), S / P of two steps (2 x 64), O (128 a row
// tile) -- 512 columns with two row tiles. K' and V' have two stages each.
// With two row tiles a step is one of them and the streams take turns in the
// tensor core; with one, steps are tiles, and the two S let the products of
// one run under the softmax of the other.
//
// Warps: 4 a row tile for the softmax (a row a thread), one that issues the
// products, one that copies raw tiles and finds their exponents, 8 that build
// operands without meeting at a barrier: one group's share of a record of the
// packed format (K: 4 tokens x 8 channels, V: 8 tokens x 4 channels) is four
// whole 16-byte units of the swizzled operand rows, so a lane reads a record's
// words and writes units. A build and the two softmax tiles that share it cost
// about 10 700 warp-instructions.
//
// Measured (32 query heads on 8 kv heads; alone and cold): 512 rows a head
// behind 32 768 4-bit tokens in 187 us, 256 rows behind 8192 2-bit tokens in 40,
// 20 behind 1111 in 17. Three products of the scores and three of the values make
// 206 GFLOP of the first, 1.10 PFLOP/s; the tensor pipe is busy 54 % of the time,
// the SM issues 47 %, HBM idles. As there, a step's chain bounds it, not one
// unit. Timing stand-ins of a whole call, with one product of the values (183.5
// us then): no softmax 174.6, a quarter of the building 170.2, one product in
// eight 145.9. One row tile for more than 128 rows took 292 us (each tile built
// twice), 16 builder warps gained nothing, half a row a thread 218.
#include "prefix.cuh"

#include "host_checks.h"
#include "quantize.cuh"

namespace kvarn {

constexpr int kPkTok = 64;                       // tokens of a tile
constexpr int kPkK = kPkTok * kD * 2;            // bytes of one 64 x 128 fp16 operand (two 64-channel blocks)
constexpr int kPkV = kD * kPkTok * 2;            // 128 channel rows x 64 tokens, fp16
constexpr int kPkQ = kPRows * kD * 2;            // 128 query rows, fp16
constexpr int kMaxRaw = 4;                       // stages of raw tiles, at most
constexpr int kBuildWarps = 8;
static_assert(kMaxRaw + 2 <= 8, "exponents in flight");
static_assert(2 * kPkV == kD * kD * 2, "the rotation matrix fits V's first stage");
constexpr float kLift = 7.f;                     // P up to 2^(8 + 7), small weights normal down to 2^-21
constexpr int kTopExp = 15;                      // K' and V' up to 2^15: halves of small values stay normal
constexpr int kTopQuery = 11;                    // the query's channels up to 2^11, rotated up to sqrt(128) times that

struct PackedSmem {
    // ready: a raw tile's exponent is known; raw_empty: its operands are built
    uint64_t raw_full[kMaxRaw], ready[kMaxRaw], raw_empty[kMaxRaw];
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_ready[2], o_full[2], q_done, drained;
    uint32_t tmem;
    int stop;
    // the exponents of the last tiles: the raw tiles' warp is at most kMaxRaw tiles ahead of
    // the V' that is built, which is at most two ahead of the softmax that reads e
    int kexp[8], vexp[8];
    int16_t qexp[2 * kPRows];   // of the query rows
};

template <int B, int BITS, int NT>   // NT: row tiles of a CTA
struct PackedLayout {
    static constexpr int kSoft = 4 * NT;                       // softmax warps
    static constexpr int kThreads = 32 * (kSoft + 2 + kBuildWarps);
    static constexpr int HB = head_block_bytes(B, BITS);
    static constexpr int kBlocks = kPkTok / B;                 // blocks per tile
    static constexpr int kRaw = kBlocks * 2 * HB;              // bytes of a raw tile: (K, V) per block
    static constexpr int kHeader = (sizeof(PackedSmem) + 1023) / 1024 * 1024;
    static constexpr int kFixed = 1024 + kHeader + NT * kPkQ + 4 * kPkK + 4 * kPkV;
    static constexpr int kFit = (227 * 1024 - kFixed) / kRaw;  // (2 with two row tiles and 4-bit blocks of 32 tokens)
    static constexpr int kRawStages = kFit < kMaxRaw ? kFit : kMaxRaw;
    static_assert(kRawStages >= 2, "a raw tile in flight while another is built");
    static constexpr size_t bytes = kFixed + kRawStages * kRaw;
};

__device__ __forceinline__ uint32_t sign_word(uint32_t s0, uint32_t s1, uint32_t s2, uint32_t s3, int w) {
    return w == 0 ? s0 : w == 1 ? s1 : w == 2 ? s2 : s3;
}
// Pair j of a record word as fp16 code 2^-9 (attn_common.cuh); for 3-bit
// codes jh is the pair's place in the high-bit word.
template <int BITS>
__device__ __forceinline__ uint32_t code_pair(uint32_t w, uint32_t w8, uint32_t hw, int j, int jh) {
    if constexpr (BITS == 2) return code2_s(w, w8, j);
    else if constexpr (BITS == 3) return code3_s(w, w8, hw, j, jh);
    else return code4_s(w, w8, j);
}

template <int B, int BITS, int NT>
__global__ void __launch_bounds__(PackedLayout<B, BITS, NT>::kThreads, 1) prefix_packed_kernel(PrefixArgs a) {
    wait_prior_grids();
    let_next_grid_start();   // the own tokens' split kernel
    using Lay = PackedLayout<B, BITS, NT>;
    constexpr int kSoft = Lay::kSoft, kRawStages = Lay::kRawStages;
    extern __shared__ uint8_t raw_smem[];
    uint8_t* base = raw_smem + ((1024 - (smem_addr(raw_smem) & 1023)) & 1023);
    PackedSmem& s = *reinterpret_cast<PackedSmem*>(base);
    uint8_t* q_lo = base + Lay::kHeader;          // [row tile]
    uint8_t* k_op = q_lo + NT * kPkQ;             // [stage][hi, lo]
    uint8_t* v_op = k_op + 4 * kPkK;              // [stage][hi, lo]; first the rotation matrix
    uint8_t* raw = v_op + 4 * kPkV;               // [raw stage][block][K, V]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int h = blockIdx.z, R = a.batch * a.G, row0 = blockIdx.y * NT * kPRows;
    const int max_len = a.n_blocks * B;

    const int most = prefix_most(a, max_len, lane);
    const int tiles = (most + kPkTok - 1) / kPkTok;
    const int t_beg = (int)((int64_t)tiles * blockIdx.x / a.splits), t_end = (int)((int64_t)tiles * (blockIdx.x + 1) / a.splits);
    const int n = t_end - t_beg;                  // tiles
    const int steps = NT * n;                     // step i: stream i % 2, tile i / NT

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
        }
        for (int i = 0; i < 2; ++i) mbar_init(&s.o_full[i], 1);
        mbar_init(&s.q_done, 1);
        mbar_init(&s.drained, 1);
        fence_mbar_init();
    }
    if (warp == kSoft) tmem_alloc(&s.tmem, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = s.tmem;
    int* stop = &s.stop;
    // Q of row tile w at + 64 w, S of stream w at + 64 w, O at + 128 w
    const uint32_t tm_q = tm, tm_s = tm + 128, tm_o = tm + 256;
    const int used = (most + B - 1) / B;          // blocks that hold a visible token
    auto fetch = [&](int i) {                     // (the raw tiles' warp) tile i into its stage
        const int st = i % kRawStages, b0 = (t_beg + i) * Lay::kBlocks;
        int64_t page = -1;                        // lane x: block x of the tile
        if (lane < Lay::kBlocks && b0 + lane < used) {
            page = a.table[b0 + lane];
            if (page < 0 || page >= a.n_pool_blocks) {
                raise_error(a.err, KVARN_DEVERR_BLOCK_ID);
                page = -1;
            }
        }
        const uint32_t bytes = __popc(__ballot_sync(kFull, page >= 0)) * (2 * Lay::HB);
        if (lane == 0) mbar_arrive_expect_tx(&s.raw_full[st], bytes);
        __syncwarp();
        if (page >= 0)
            bulk_g2s(raw + st * Lay::kRaw + lane * 2 * Lay::HB, a.pool + page * a.block_bytes + (int64_t)(2 * h) * Lay::HB,
                     2 * Lay::HB, &s.raw_full[st]);
    };
    int fetched = 0;
    if (warp == kSoft + 1)
        for (; fetched < kRawStages - 1 && fetched < n; ++fetched) fetch(fetched);

    // ---- the query rows: each is scaled by the power of two that brings its
    // largest channel to 2^11; their rotation H (sigma q) / sqrt(128) is itself a
    // product on the tensor core, of signs and of q in fp16 (a bf16 one is exact
    // down to 2^-25 of the largest) or, for an fp32 one, of its two fp16 halves;
    // without rotation H is the identity. Then the rows are split into two fp16
    // halves: the high one to tensor memory, the low one to its operand. (A row a
    // warp or a thread through butterflies took 7-14 us of a call.)
    const bool q32 = a.q_dtype == KVARN_FP32, rotate = !(a.flags & KVARN_FLAG_NO_ROTATION);
    {
        constexpr int kBatch = 4;
        for (int i0 = tid; i0 < NT * kPRows * 16; i0 += kBatch * Lay::kThreads) {
            uint4 x[kBatch], y[kBatch];                                  // (y: channels 4 .. 7 of an fp32 unit)
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const int i = i0 + j * Lay::kThreads, row = row0 + (i >> 4);
                const int64_t at = ((int64_t)(row / a.G) * a.n_q + h * a.G + row % a.G) * kD + 8 * (i & 15);
                x[j] = y[j] = make_uint4(0, 0, 0, 0);
                if (i < NT * kPRows * 16 && row < R) {
                    const char* src = static_cast<const char*>(a.q) + at * (q32 ? 4 : 2);
                    x[j] = *reinterpret_cast<const uint4*>(src);
                    if (q32) y[j] = *reinterpret_cast<const uint4*>(src + 16);
                }
            }
            if (i0 == tid)                                               // H, in V's first stage, under the loads
                for (int i = tid; i < kD * 16; i += Lay::kThreads) {
                    const int r = i >> 4, u = i & 15;
                    uint32_t w[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int c = 8 * u + 2 * k;
                        w[k] = rotate ? 0x3c003c00u ^ (__popc(r & c) & 1) << 15 ^ (uint32_t)(__popc(r & (c + 1)) & 1) << 31
                                      : (r == c ? 0x3c00u : 0u) | (r == c + 1 ? 0x3c000000u : 0u);
                    }
                    *reinterpret_cast<uint4*>(v_op + (u >> 3) * (kPkQ / 2) + swizzled(r, u & 7)) = make_uint4(w[0], w[1], w[2], w[3]);
                }
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const int i = i0 + j * Lay::kThreads, r = i >> 4, u = i & 15;
                if (i >= NT * kPRows * 16) break;
                uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w}, lo[4];
                float f[8];
                if (q32) {
                    const uint32_t u8[8] = {w[0], w[1], w[2], w[3], y[j].x, y[j].y, y[j].z, y[j].w};
#pragma unroll
                    for (int k = 0; k < 8; ++k) f[k] = __uint_as_float(u8[k]);
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        f[2 * k] = __uint_as_float(w[k] << 16);
                        f[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
                    }
                }
                float big = 0.f;                                         // (a row: 16 lanes next to one another)
#pragma unroll
                for (int k = 0; k < 8; ++k) big = fmaxf(big, fabsf(f[k]));
#pragma unroll
                for (int m = 8; m >= 1; m >>= 1) big = fmaxf(big, __shfl_xor_sync(kFull, big, m));
                const int e = big > 0x1p-100f ? ceil_log2(big) : -100;
                if (u == 0) s.qexp[r] = (int16_t)e;
                const float up = exp2i(kTopQuery - e);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (q32) split_pair<true>(f[2 * k] * up, f[2 * k + 1] * up, w[k], lo[k]);
                    else w[k] = pack_h2(f[2 * k] * up, f[2 * k + 1] * up);
                }
                const uint32_t sg = rotate ? sign_word(a.sb[0], a.sb[1], a.sb[2], a.sb[3], u >> 2) >> (8 * (u & 3)) : 0u;
                const uint32_t at = (r / kPRows) * kPkQ + (u >> 3) * (kPkQ / 2) + swizzled(r % kPRows, u & 7);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t flip = (sg >> (2 * k) & 1u) << 15 | (sg >> (2 * k + 1) & 1u) << 31;
                    w[k] ^= flip;
                    if (q32) lo[k] ^= flip;
                }
                *reinterpret_cast<uint4*>(q_lo + at) = make_uint4(w[0], w[1], w[2], w[3]);
                if (q32) *reinterpret_cast<uint4*>(k_op + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);   // in K's stages
            }
        }
    }
    fence_async_smem();
    __syncthreads();
    if (warp <= kSoft) {
        if (warp == kSoft) {
            constexpr uint32_t kRot = mma_shape(kMmaF16, kD, false);
            const uint32_t q_desc = smem_operand(smem_addr(q_lo), 16), l_desc = smem_operand(smem_addr(k_op), 16);
            const uint32_t h_desc = smem_operand(smem_addr(v_op), 16);
#pragma unroll 1
            for (int k = 0; k < (q32 ? 16 : 8) * NT; ++k) {
                const int part = k / (8 * NT), x = k / 8 % NT;
                const uint32_t off = ((k >> 2 & 1) * (kPkQ / 2) + (k & 3) * 32) >> 4;
                mma_ss(tm_o + 128 * x, (part ? l_desc : q_desc) + x * (kPkQ >> 4) + off, h_desc + off, kRot, part > 0 || (k & 7) > 0);
            }
            mma_commit(&s.q_done);
        }
        const bool ok = warp_wait_or_stop(&s.q_done, 0, stop, kWaitLimit);
        tc_fence_after();
        if (warp < kSoft && ok) {
            const float norm = rotate ? kInvSqrtD : 1.f;
            const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
            uint8_t* lo_row = q_lo + (warp >> 2) * kPkQ;
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {                                // 32 channels
                uint32_t v[32];
                tmem_ld32(tm_o + 128 * (warp >> 2) + 32 * c + lanes, v);
                tmem_wait_ld();
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    uint32_t lo[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float x0 = __uint_as_float(v[8 * u + 2 * k]) * norm, x1 = __uint_as_float(v[8 * u + 2 * k + 1]) * norm;
                        split_pair<true>(x0, x1, v[4 * u + k], lo[k]);
                    }
                    *reinterpret_cast<uint4*>(lo_row + (c >> 1) * (kPkQ / 2) + swizzled((warp & 3) * 32 + lane, 4 * (c & 1) + u)) =
                        make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
                tmem_st16(tm_q + 64 * (warp >> 2) + 16 * c + lanes, v);
            }
            tmem_wait_st();
            fence_async_smem();
        }
        tc_fence_before();
        asm volatile("bar.sync 1, %0;" ::"n"(32 * (kSoft + 1)) : "memory");   // the product warp waits for the rows
        tc_fence_after();
    }

    if (warp == kSoft + 1) {
        // ---------------------------------------------------------- raw tiles and their exponents
        bool ok = true;
        for (int i = 0; i < n && ok; ++i) {
            // (one stage less in flight than there are: its wait is for tile i - 2)
            for (; fetched < n && fetched < i + kRawStages - 1 && ok; ++fetched) {
                if (fetched >= kRawStages)        // the stage's last tile has been built
                    ok = warp_wait_or_stop(&s.raw_empty[fetched % kRawStages], (fetched / kRawStages - 1) & 1, stop, kWaitLimit);
                if (!ok) break;
                fetch(fetched);
            }
            const int st = i % kRawStages;
            ok = ok && warp_wait_or_stop(&s.raw_full[st], (i / kRawStages) & 1, stop, kWaitLimit);
            if (!ok) break;
            // 2^e over the tile's keys and over its values: the largest (|zero|, |top
            // level|) R times the largest C (a lane: 8 (group, token) pairs, 4 or 8 channels)
            constexpr int kPer = 32 / Lay::kBlocks;                // lanes per block
            const int x = lane / kPer, at = 8 * (lane % kPer);
            const bool there = (t_beg + i) * Lay::kBlocks + x < used;
            auto exponent = [&](const uint8_t* hb) {
                float vmax = 0.f, cmax = 0.f;
                if (there) {
                    const uint4 su = *reinterpret_cast<const uint4*>(hb + off_s(B, BITS) + 2 * at);
                    const uint4 zu = *reinterpret_cast<const uint4*>(hb + off_z(B, BITS) + 2 * at);
                    const uint4 ru = *reinterpret_cast<const uint4*>(hb + off_R(B, BITS) + 2 * (at % B));
                    const uint32_t sw[4] = {su.x, su.y, su.z, su.w}, zw[4] = {zu.x, zu.y, zu.z, zu.w}, rw[4] = {ru.x, ru.y, ru.z, ru.w};
                    constexpr float kTop = (float)((1 << BITS) - 1);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 sf = __half22float2(u32_as_h2(sw[k])), zf = __half22float2(u32_as_h2(zw[k]));
                        const float2 rf = __half22float2(u32_as_h2(rw[k]));
                        vmax = fmaxf(vmax, fmaxf(fabsf(zf.x), fabsf(fmaf(sf.x, kTop, zf.x))) * fabsf(rf.x));
                        vmax = fmaxf(vmax, fmaxf(fabsf(zf.y), fabsf(fmaf(sf.y, kTop, zf.y))) * fabsf(rf.y));
                    }
                    constexpr int kCh = kD / kPer;
#pragma unroll
                    for (int k = 0; k < kCh; k += 2) {
                        const float2 cf = __half22float2(
                            u32_as_h2(*reinterpret_cast<const uint32_t*>(hb + off_C(B, BITS) + 2 * (kCh * (lane % kPer) + k))));
                        cmax = fmaxf(cmax, fmaxf(fabsf(cf.x), fabsf(cf.y)));
                    }
                }
                const float bound = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(vmax))) *
                                    __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(cmax)));
                // (the clamps keep 2^-e and 2^e finite)
                return (bound > 0x1p-60f ? min(ceil_log2(bound), 100) : -60) - kTopExp;
            };
            const uint8_t* hb = raw + st * Lay::kRaw + x * 2 * Lay::HB;
            const int ke = exponent(hb), ve = exponent(hb + Lay::HB);
            if (lane == 0) {
                s.kexp[i & 7] = ke;
                s.vexp[i & 7] = ve;
                mbar_arrive(&s.ready[st]);
            }
        }
    } else if (warp > kSoft) {
        // ---------------------------------------------------------- operands from codes
        // warp bw: group g of the 32 records of half sb, a record a lane
        const int bw = warp - (kSoft + 2), g = bw & 3, sb = bw >> 2, ra = lane >> 2, rb = lane & 3;
        const int half0 = B == 64 ? 32 * sb : 0;          // the half's first token within its block
        // (code 2^-9) s + z 2^-9, times the rest of the value's factors and 2^9
        constexpr float kUp = 512.f;
        bool ok = true;
        for (int i = 0; i < n && ok; ++i) {
            const int st = i % kRawStages, par = i & 1;
            ok = warp_wait_or_stop(&s.ready[st], (i / kRawStages) & 1, stop, kWaitLimit) &&
                 warp_wait_or_stop(&s.raw_full[st], (i / kRawStages) & 1, stop, kWaitLimit);
            if (!ok) break;
            const uint8_t* hb = raw + st * Lay::kRaw + (B == 64 ? 0 : sb) * 2 * Lay::HB;
            const bool there = (t_beg + i) * Lay::kBlocks + (B == 64 ? 0 : sb) < used;   // else its values are zero
            // ---- K: 4 tokens 4 ra + k of the half, channels 32 g + 8 rb .. + 7
            {
                const uint8_t* codes = hb + (half0 + lane) * 16 * BITS;
                uint32_t w[4], hw[4];              // token k's word with this group's fields at its low end
                const uint4* src = reinterpret_cast<const uint4*>(codes);
                if constexpr (BITS == 4) {         // word 4 k + g
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint4 u = src[k];
                        w[k] = g == 0 ? u.x : g == 1 ? u.y : g == 2 ? u.z : u.w;
                    }
                } else {                           // word 2 k + g / 2, fields 4 (g % 2) ..
                    const uint4 u = src[0], v = src[1];
                    w[0] = (g & 2 ? u.y : u.x) >> 8 * (g & 1);
                    w[1] = (g & 2 ? u.w : u.z) >> 8 * (g & 1);
                    w[2] = (g & 2 ? v.y : v.x) >> 8 * (g & 1);
                    w[3] = (g & 2 ? v.w : v.z) >> 8 * (g & 1);
                    if constexpr (BITS == 3) {     // high bits in word 8 + k from bit 4 g
                        const uint4 x = src[2];
                        hw[0] = x.x >> 4 * g; hw[1] = x.y >> 4 * g; hw[2] = x.z >> 4 * g; hw[3] = x.w >> 4 * g;
                    }
                }
                const int t0 = half0 + 4 * ra;
                const uint2 su = *reinterpret_cast<const uint2*>(hb + off_s(B, BITS) + 2 * (g * B + t0));
                const uint2 zu = *reinterpret_cast<const uint2*>(hb + off_z(B, BITS) + 2 * (g * B + t0));
                const uint2 ru = *reinterpret_cast<const uint2*>(hb + off_R(B, BITS) + 2 * t0);
                const uint4 cu = *reinterpret_cast<const uint4*>(hb + off_C(B, BITS) + 2 * (32 * g + 8 * rb));
                float2 cc[4] = {__half22float2(u32_as_h2(cu.x)), __half22float2(u32_as_h2(cu.y)),
                                __half22float2(u32_as_h2(cu.z)), __half22float2(u32_as_h2(cu.w))};
                if (i >= 2) ok = warp_wait_or_stop(&s.k_empty[par], ((i >> 1) - 1) & 1, stop, kWaitLimit);
                if (i == 0 && q32) ok = warp_wait_or_stop(&s.q_done, 0, stop, kWaitLimit);   // (the query's low half was here)
                if (!ok) break;
                uint8_t* dst = k_op + par * 2 * kPkK + (g >> 1) * (kPkK / 2);
                const float up = kUp * exp2i(-*reinterpret_cast<volatile int*>(&s.kexp[i & 7]));
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t step = k < 2 ? su.x : su.y;
                    const float2 z2 = __half22float2(u32_as_h2(k < 2 ? zu.x : zu.y)), r2 = __half22float2(u32_as_h2(k < 2 ? ru.x : ru.y));
                    const float zero = ((k & 1) ? z2.y : z2.x) * kCodeScale, fac = ((k & 1) ? r2.y : r2.x) * up;
                    const uint32_t w8 = w[k] >> 8;
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        const uint32_t f = code_pair<BITS>(w[k], w8, hw[k], p, p);
                        float2 y = make_float2(fma_half(f, step, zero, false, k & 1), fma_half(f, step, zero, true, k & 1));
                        y = __fmul2_rn(__fmul2_rn(y, make_float2(fac, fac)), cc[p]);
                        split_pair<true>(y.x, y.y, hi[p], lo[p]);
                    }
                    const uint32_t at = swizzled(32 * sb + 4 * ra + k, 4 * (g & 1) + rb);
                    // (an absent half's scores are masked, whatever its raw bytes were)
                    *reinterpret_cast<uint4*>(dst + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4*>(dst + kPkK + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
                fence_async_smem();
                warp_arrive(&s.k_full[par]);
            }
            // ---- V: channels 32 g + 4 ra + k, 8 tokens 8 rb .. + 7 of the half
            {
                const uint8_t* vb = hb + Lay::HB;
                const uint8_t* codes = vb + (half0 + lane) * 16 * BITS;
                uint32_t w[4], hw = 0;             // 4-bit: word 4 g + k; else 2 g + k / 2, and its high bits in word 8 + g
                if constexpr (BITS == 4) {
                    const uint4 u = reinterpret_cast<const uint4*>(codes)[g];
                    w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
                } else {
                    const uint2 u = reinterpret_cast<const uint2*>(codes)[g];
                    w[0] = w[1] = u.x;
                    w[2] = w[3] = u.y;
                    if constexpr (BITS == 3) hw = reinterpret_cast<const uint32_t*>(codes)[8 + g];
                }
                const int t0 = half0 + 8 * rb;
                const uint4 su = *reinterpret_cast<const uint4*>(vb + off_s(B, BITS) + 2 * (g * B + t0));
                const uint4 zu = *reinterpret_cast<const uint4*>(vb + off_z(B, BITS) + 2 * (g * B + t0));
                const uint4 ru = *reinterpret_cast<const uint4*>(vb + off_R(B, BITS) + 2 * t0);
                const uint2 cu = *reinterpret_cast<const uint2*>(vb + off_C(B, BITS) + 2 * (32 * g + 4 * ra));
                const uint32_t sw[4] = {su.x, su.y, su.z, su.w}, zw[4] = {zu.x, zu.y, zu.z, zu.w}, rw[4] = {ru.x, ru.y, ru.z, ru.w};
                // (warps of an absent half, whose raw bytes may be anything, write zeros)
                const float up = kUp * exp2i(-*reinterpret_cast<volatile int*>(&s.vexp[i & 7]));
                float2 zero[4], fac[4];            // token pairs
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    zero[p] = __fmul2_rn(__half22float2(u32_as_h2(zw[p])), make_float2(kCodeScale, kCodeScale));
                    fac[p] = __fmul2_rn(__half22float2(u32_as_h2(rw[p])), make_float2(up, up));
                }
                const float2 c01 = __half22float2(u32_as_h2(cu.x)), c23 = __half22float2(u32_as_h2(cu.y));
                const float cf[4] = {c01.x, c01.y, c23.x, c23.y};
                if (i >= 2) ok = warp_wait_or_stop(&s.v_empty[par], ((i >> 1) - 1) & 1, stop, kWaitLimit);
                if (i == 0) ok = warp_wait_or_stop(&s.q_done, 0, stop, kWaitLimit);   // (H was here)
                if (!ok) break;
                uint8_t* dst = v_op + par * 2 * kPkV;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t w8 = w[k] >> 8;
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int p = 0; p < 4; ++p) {                 // tokens 2p, 2p + 1
                        const int j = BITS == 4 ? p : 4 * (p >> 1) + 2 * (p & 1) + (k & 1);
                        const uint32_t f = code_pair<BITS>(w[k], w8, hw, j, 8 * (k >> 1) + j);
                        float2 y = make_float2(fma_half(f, sw[p], zero[p].x, false, false), fma_half(f, sw[p], zero[p].y, true, true));
                        y = __fmul2_rn(__fmul2_rn(y, fac[p]), make_float2(cf[k], cf[k]));
                        split_pair<true>(y.x, y.y, hi[p], lo[p]);
                        if (!there) hi[p] = lo[p] = 0u;
                    }
                    const uint32_t at = swizzled(32 * g + 4 * ra + k, 4 * sb + rb);
                    *reinterpret_cast<uint4*>(dst + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4*>(dst + kPkV + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
                fence_async_smem();
                warp_arrive(&s.v_full[par]);
                warp_arrive(&s.raw_empty[st]);
            }
        }
    } else if (warp == kSoft) {
        // ---------------------------------------------------------- products
        if (steps > 0) {
            constexpr uint32_t kQk = mma_shape(kMmaF16, kPkTok, false), kPv = mma_shape(kMmaF16, kD, false);
            const uint32_t q_desc = smem_operand(smem_addr(q_lo), 16), k_desc = smem_operand(smem_addr(k_op), 16);
            const uint32_t v_desc = smem_operand(smem_addr(v_op), 16);
            bool ok = !(a.flags & KVARN_FLAG_TEST_WAIT_TIMEOUT);
            if (!ok && lane == 0) *stop = 1;                      // (test switch: as if the first wait had run out)
            for (int i = 0; i < steps + 2 && ok; ++i) {           // O (+)= P V' of step j, then S = Q K'^T of step i
                const int j = i - 2, w = i & 1, tj = j / NT, ti = i / NT, x = NT == 2 ? w : 0;
                if (i < steps && (NT == 1 || w == 0)) ok = warp_wait_or_stop(&s.k_full[ti & 1], (ti >> 1) & 1, stop, kWaitLimit);
                if (j >= 0) {
                    if (NT == 1 || w == 0) ok = ok && warp_wait_or_stop(&s.v_full[tj & 1], (tj >> 1) & 1, stop, kWaitLimit);
                    ok = ok && warp_wait_or_stop(&s.p_ready[w], (j >> 1) & 1, stop, kWaitLimit);
                }
                if (!ok) break;
                tc_fence_after();
                if (j >= 0) {
                    const uint32_t p = tm_s + 64 * w, vd = v_desc + (tj & 1) * (2 * kPkV >> 4);
#pragma unroll
                    for (int k = 0; k < kPkTok / 16; ++k) {       // hi hi, hi lo, lo hi
                        mma_ts(tm_o + 128 * x, p + 16 * k, vd + 2 * k, kPv, tj > 0 || k > 0);
                        mma_ts(tm_o + 128 * x, p + 16 * k, vd + (kPkV >> 4) + 2 * k, kPv, true);
                        mma_ts(tm_o + 128 * x, p + 16 * k + kPLow, vd + 2 * k, kPv, true);
                    }
                    if (NT == 1 || w == 1) mma_commit(&s.v_empty[tj & 1]);
                    if (j + NT >= steps) mma_commit(&s.o_full[x]);
                }
                if (i < steps) {
                    const uint32_t kd = k_desc + (ti & 1) * (2 * kPkK >> 4), qa = tm_q + 64 * x, qd = q_desc + x * (kPkQ >> 4);
#pragma unroll
                    for (int k = 0; k < 24; ++k) {                // hi hi, hi lo, lo hi
                        const uint32_t kb = kd + (((k >> 3) == 1 ? kPkK >> 4 : 0) + (((k >> 2 & 1) * (kPkK / 2) + (k & 3) * 32) >> 4));
                        if (k < 16) mma_ts(tm_s + 64 * w, qa + 8 * (k & 7), kb, kQk, k > 0);
                        else mma_ss(tm_s + 64 * w, qd + (((k >> 2 & 1) * (kPkQ / 2) + (k & 3) * 32) >> 4), kb, kQk, true);
                    }
                    mma_commit(&s.s_full[w]);
                    if (NT == 1 || w == 1) mma_commit(&s.k_empty[ti & 1]);
                }
            }
            // products in flight end before the operands and tensor memory go
            mma_commit(&s.drained);
            if (!mbar_wait_bounded(&s.drained, 0, kWaitLimit)) *stop = 1;
        }
    } else {
        // ---------------------------------------------------------- softmax
        const int x = warp >> 2;                                  // row tile
        const int row = row0 + warp * 32 + lane;
        const int len = row < R ? prefix_len(a.lens, row / a.G, max_len) : 0;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t my_o = tm_o + 128 * x + lanes;
        const float scale = a.sm_scale * kLog2e * exp2i(s.qexp[warp * 32 + lane] - kTopQuery);
        RowState st{-INFINITY, 0.f};
        bool ok = true;
        for (int i = 0; i < n && ok; ++i) {                       // tile
            const int w = NT == 2 ? x : i & 1, j = NT == 2 ? i : i >> 1;
            ok = warp_wait_or_stop(&s.s_full[w], j & 1, stop, kWaitLimit);
            if (!ok) break;
            tc_fence_after();
            const int e = *reinterpret_cast<volatile int*>(&s.vexp[i & 7]);
            // (finite and not 0, so that what is masked stays masked)
            const float here = fminf(fmaxf(scale * exp2i(*reinterpret_cast<volatile int*>(&s.kexp[i & 7])), 0x1p-126f), 0x1p127f);
            ok = softmax_tile<kPkTok, NT == 2 ? 32 : 64, true>(tm_s + 64 * w + lanes, my_o, len - (t_beg + i) * kPkTok, here, (float)e,
                                                        exp2i(-e), kLift, i == 0, st, &s.p_ready[w], [&] {
                // O is idle once the last product into it has completed: with two row
                // tiles S came behind it, with one it has freed tile i - 1's V stage
                if (NT == 2) return true;
                const bool idle = warp_wait_or_stop(&s.v_empty[(i - 1) & 1], ((i - 1) >> 1) & 1, stop, kWaitLimit);
                tc_fence_after();
                return idle;
            });
        }
        // every stream's products are over before the operands' memory is reused
        for (int k = 0; k < NT && n > 0 && ok; ++k) ok = warp_wait_or_stop(&s.o_full[k], 0, stop, kWaitLimit);
        tc_fence_after();
        if (ok) store_partials(a, blockIdx.x, row - lane, h, q_lo + warp * 32 * kPartialStride * 4, n == 0, st.m - kLift, st.l, my_o, lane);
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
        tmem_free(tm, 512);
    }
}

// ---------------------------------------------------------------- host side
template <int B, int BITS, int NT>
cudaError_t launch_packed_tiles(const PrefixArgs& p, cudaStream_t st) {
    using Lay = PackedLayout<B, BITS, NT>;
    static_assert(Lay::bytes <= 227 * 1024, "shared memory of one CTA");
    static_assert(Lay::kSoft * 32 * kPartialStride * 4 <= NT * kPkQ + 4 * kPkK + 4 * kPkV, "the partials' staging fits the operands' memory");
    static bool ready[64];
    int d = 0;
    cudaError_t e = cudaGetDevice(&d);
    if (e != cudaSuccess) return e;
    if (d < 0 || d >= 64) return cudaErrorInvalidDevice;
    if (!ready[d]) {
        e = cudaFuncSetAttribute(prefix_packed_kernel<B, BITS, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Lay::bytes);
        if (e != cudaSuccess) return e;
        ready[d] = true;
    }
    const dim3 grid(p.splits, (p.batch * p.G + NT * kPRows - 1) / (NT * kPRows), p.n_kv);
    return launch_pdl(prefix_packed_kernel<B, BITS, NT>, grid, Lay::kThreads, Lay::bytes, st, p);
}

cudaError_t launch_prefix_packed(const kvarn_config& c, const PrefixArgs& p, cudaStream_t st) {
    return dispatch(c, [&](auto b, auto w) {
        constexpr int B = decltype(b)::value, BITS = decltype(w)::value;
        return (int64_t)p.batch * p.G > kPRows ? launch_packed_tiles<B, BITS, 2>(p, st) : launch_packed_tiles<B, BITS, 1>(p, st);
    });
}

}  // namespace kvarn
