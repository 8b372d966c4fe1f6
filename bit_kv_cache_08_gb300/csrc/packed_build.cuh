// packed_build.cuh -- 64-token tiles of the packed cache as operands of the
// tensor core, for the kernels that multiply them with many query rows: the tiles' sizes and
// the reading of codes, which the shared prefix (prefix_packed.cu) and draft trees
// (tree_packed.cu) have in common, and the prefix's builders. (Draft trees build with fp16 arithmetic
// from levels prepared ahead, 4 warps for keys and 4 for values.)
//
// The prefix's: K' (64 tokens x 128 channels, channels along the contraction) and V' (128 channels x 64
// tokens, tokens along it) hold (code s + z) R C under a power of two of the tile's, each value
// as two fp16 halves. 8 warps build them without meeting at a barrier: one group's
// share of a record of the packed format (K: 4 tokens x 8 channels, V: 8 tokens x 4
// channels) is four whole 16-byte units of the swizzled operand rows, so a lane reads a
// record's words and writes units.
#pragma once
#include "prefix.cuh"

namespace kvarn {

constexpr int kPkTok = 64;                       // tokens of a tile
constexpr int kPkK = kPkTok * kD * 2;            // bytes of one 64 x 128 fp16 operand (two 64-channel blocks)
constexpr int kPkV = kD * kPkTok * 2;            // 128 channel rows x 64 tokens, fp16
constexpr int kPkQ = kPRows * kD * 2;            // 128 query rows, fp16
constexpr int kMaxRaw = 4;                       // stages of raw tiles, at most
constexpr int kBuildWarps = 8;
static_assert(kMaxRaw + 2 <= 8, "exponents in flight");
constexpr float kLift = 7.f;                     // P up to 2^(8 + 7); weights normal down to 2^-21 of the reference's
constexpr int kTopExp = 15;                      // K' and V' up to 2^15: halves of small values stay normal

// Pair j of a record word as fp16 code 2^-9 (attn_common.cuh); for 3-bit
// codes jh is the pair's place in the high-bit word.
template <int BITS>
__device__ __forceinline__ uint32_t code_pair(uint32_t w, uint32_t w8, uint32_t hw, int j, int jh) {
    if constexpr (BITS == 2) return code2_s(w, w8, j);
    else if constexpr (BITS == 3) return code3_s(w, w8, hw, j, jh);
    else return code4_s(w, w8, j);
}

// The power of two over a tile's keys or values (warp-cooperative): the largest (|zero|,
// |top level|) R times the largest C, a lane 8 (group, token) pairs and 4 or 8 channels of
// its block's head-block hb; `there`: the block is.
template <int B, int BITS>
__device__ __forceinline__ int tile_exponent(const uint8_t* hb, bool there, int lane) {
    constexpr int kPer = 32 / (kPkTok / B);              // lanes per block
    const int at = 8 * (lane % kPer);
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
}

// (code 2^-9) s + z 2^-9, times the rest of the value's factors and 2^9
constexpr float kBuildUp = 512.f;

// K' of group g of the 32 records of half sb of a tile, a record a lane: tokens 4 (lane / 4) + k,
// channels 32 g + 8 (lane % 4) .. + 7. hb: the half's K head-block; exponent: of the
// tile; ready(): waits until dst (hi, then lo) may be written (false: gave up).
template <int B, int BITS, typename Ready>
__device__ __forceinline__ bool build_keys(const uint8_t* hb, int g, int sb, int lane, const int* exponent, uint8_t* dst, Ready&& ready) {
    const int ra = lane >> 2, rb = lane & 3;
    const int half0 = B == 64 ? 32 * sb : 0;             // the half's first token within its block
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
    if (!ready()) return false;
    dst += (g >> 1) * (kPkK / 2);
    const float up = kBuildUp * exp2i(-*reinterpret_cast<const volatile int*>(exponent));
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
    return true;
}

// V' likewise: channels 32 g + 4 (lane / 4) + k, tokens 8 (lane % 4) .. + 7 of the half. vb: the
// half's V head-block; `there`: the half is (else, whatever its raw bytes are, its
// values are zeros).
template <int B, int BITS, typename Ready>
__device__ __forceinline__ bool build_values(const uint8_t* vb, bool there, int g, int sb, int lane, const int* exponent, uint8_t* dst,
                                             Ready&& ready) {
    const int ra = lane >> 2, rb = lane & 3;
    const int half0 = B == 64 ? 32 * sb : 0;
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
    const float up = kBuildUp * exp2i(-*reinterpret_cast<const volatile int*>(exponent));
    float2 zero[4], fac[4];            // token pairs
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        zero[p] = __fmul2_rn(__half22float2(u32_as_h2(zw[p])), make_float2(kCodeScale, kCodeScale));
        fac[p] = __fmul2_rn(__half22float2(u32_as_h2(rw[p])), make_float2(up, up));
    }
    const float2 c01 = __half22float2(u32_as_h2(cu.x)), c23 = __half22float2(u32_as_h2(cu.y));
    const float cf[4] = {c01.x, c01.y, c23.x, c23.y};
    if (!ready()) return false;
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
    return true;
}

}  // namespace kvarn
