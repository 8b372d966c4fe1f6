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
// (64 columns a row tile), beside S / P of two steps (2 x 64 columns) and O (128 a row tile); its
// low half too, where one row tile leaves room, else in shared memory.
// Warps: 4 a row tile for the softmax, one that issues the products, one that copies raw
// tiles and prepares the levels of their keys, one for those of the values, 8 that build
// operands, as in packed_build.cuh without meeting at a barrier.
//
// Measured (48 sequences x 16 drafts, up to 8192 4-bit tokens, 8 kv heads): 400 us a call, this kernel alone
// and cold 365, about 2900 cycles a tile of 64 tokens. The tensor core is busy 1480 of them (six products of halves),
// a warp that builds 1500, shared memory about as long (64 KB of operands written, 96 KB read by the products; the
// LSU's share was 29 % of a smaller call): no unit is saturated, each waits for the others in turn. Rows are the
// products' M, so that 32 cost what 128 do, and the width of a code does not matter: 2-bit tokens take as
// long as 4-bit ones, and longer than bf16 pages (64 x 8 drafts 490 us, 253). Not faster: four S in tensor
// memory and products of P three steps behind, 8 + 8 builder warps, two streams of softmax, rows of up to
// 64 held twice so that P V is two products.
#include "packed_build.cuh"
#include "host_checks.h"
#include "quantize.cuh"
#include "tree.cuh"

namespace kvarn {

constexpr int kTreeBuild = 4;        // warps that build a tile's keys, and as many its values
constexpr int kTreeTopQuery = 14;    // a rotated query's channels up to 2^14
constexpr uint32_t kQLow = 384;      // column of the queries' low halves (one row tile)

// ---------------------------------------------------------------- queries
// A warp a row: [unit][rows_pad][hi 128 | lo 128] fp16, and what the scores are to be
// multiplied with, 2^e, [unit][rows_pad].
__global__ void __launch_bounds__(256) tree_rotate_kernel(TreeArgs a) {
    wait_prior_grids();
    let_next_grid_start();   // the cached tokens' kernel, whose first operands need no query
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

// ---------------------------------------------------------------- operands from codes
// A value is (code S + Z) C with S = s R and Z = z R of its (token, group), C of its
// channel. Two warps prepare S and Z of a tile's keys and of its values: scaled by a
// power of two of the tile's (the largest level up to 2^6, the largest C up to 2^9, so that
// products reach 2^15) and split at a quantum u of the (token, group)'s own, the power of two
// with its largest level within 2040 u:
//   Sh, Zh  multiples of u: every level code Sh + Zh is one of up to 2047 u, exact in fp16
//   Sl, Zl  the rests, up to u / 2: a level's rest code Sl + Zl is up to 2 u (2 bits), 4 u (3), 8 u (4)
// The builder warps then need fp16 arithmetic only, on pairs:
//   Lh = code Sh + Zh (exact), Ll = code Sl + Zl (within 2^-9 u at 4 bits),
//   hi = RN(Lh C), lo = RN(RN(Lh C - hi) + Ll C)  (Lh C - hi is exact)
// so that hi + lo is within 2^-18 of the (token, group)'s largest level times C (2^-20 at 2
// bits), plus 2^-22 of itself. In fp32 (a mixed multiply-add, two products and a split into halves
// by conversions, as the shared prefix builds) a pair costs half as many instructions again, several of
// them at lower rates. That alone gained nothing while the builders waited for their raw
// tiles (48 x 16 drafts over 8192 4-bit tokens: 448 us with either); with rings of raw
// tiles and 4 warps each for keys and values it is 390.
constexpr int kTopLevel = 6, kTopChannel = 9;
constexpr float kCodeUp = 512.f;      // (codes come as code 2^-9)
constexpr int kRest = 4 * kPkTok * 2; // bytes of one plane of rests: [block][4][B] fp16

// S and Z of a head-block hb of the tile (its 8 (group, token) pairs of this lane), Sh 2^9 and Zh
// in place of s and z, Sl 2^9 and Zl at rest; returns the tile's exponent, and C's in
// c_exp. `there`: the lane's block is.
template <int B, int BITS>
__device__ __forceinline__ int prepare_levels(uint8_t* hb, bool there, int lane, uint8_t* rest, int& c_exp) {
    constexpr int kPer = 32 / (kPkTok / B), kCh = kD / kPer;   // lanes and channels of a block
    constexpr float kTop = (float)((1 << BITS) - 1);
    const int at = 8 * (lane % kPer);
    float S[8], Z[8], top[8], vmax = 0.f, cmax = 0.f;
    if (there) {
        const uint4 su = *reinterpret_cast<const uint4*>(hb + off_s(B, BITS) + 2 * at);
        const uint4 zu = *reinterpret_cast<const uint4*>(hb + off_z(B, BITS) + 2 * at);
        const uint4 ru = *reinterpret_cast<const uint4*>(hb + off_R(B, BITS) + 2 * (at % B));
        const uint32_t sw[4] = {su.x, su.y, su.z, su.w}, zw[4] = {zu.x, zu.y, zu.z, zu.w}, rw[4] = {ru.x, ru.y, ru.z, ru.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 rf = __half22float2(u32_as_h2(rw[k]));
            const float2 sf = __fmul2_rn(__half22float2(u32_as_h2(sw[k])), rf), zf = __fmul2_rn(__half22float2(u32_as_h2(zw[k])), rf);
            S[2 * k] = sf.x, S[2 * k + 1] = sf.y, Z[2 * k] = zf.x, Z[2 * k + 1] = zf.y;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            top[k] = fmaxf(fabsf(Z[k]), fabsf(fmaf(S[k], kTop, Z[k])));
            vmax = fmaxf(vmax, top[k]);
        }
#pragma unroll
        for (int k = 0; k < kCh; k += 2) {
            const float2 cf = __half22float2(
                u32_as_h2(*reinterpret_cast<const uint32_t*>(hb + off_C(B, BITS) + 2 * (kCh * (lane % kPer) + k))));
            cmax = fmaxf(cmax, fmaxf(fabsf(cf.x), fabsf(cf.y)));
        }
    }
    vmax = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(vmax)));
    cmax = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(cmax)));
    // (the clamps keep every power of two below finite)
    const int v_exp = (vmax > 0x1p-60f ? min(ceil_log2(vmax), 60) : -60) - kTopLevel;
    c_exp = (cmax > 0x1p-30f ? min(ceil_log2(cmax), 30) : -30) - kTopChannel;
    if (there) {
        const float down = exp2i(-v_exp);
        uint32_t sh[4], zh[4], sl[4], zl[4];
        float y[4][2];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float s0 = S[k] * down, z0 = Z[k] * down;
            // 1.5 2^23 u, u = 2^(e - 10), 2^e the power of two below the largest level and a
            // little: adding and subtracting it rounds to multiples of u
            const uint32_t e = __float_as_uint(fmaf(top[k] * down, 0x1p-7f, top[k] * down)) & 0x7f800000u;
            const float round = __uint_as_float(max(e, 0x08000000u) + (13u << 23)) * 1.5f;
            const float a = __fsub_rn(__fadd_rn(s0, round), round), b = __fsub_rn(__fadd_rn(z0, round), round);
            y[0][k & 1] = a * kCodeUp;
            y[1][k & 1] = b;
            y[2][k & 1] = (s0 - a) * kCodeUp;
            y[3][k & 1] = z0 - b;
            if (k & 1) {
                sh[k >> 1] = pack_h2(y[0][0], y[0][1]);
                zh[k >> 1] = pack_h2(y[1][0], y[1][1]);
                sl[k >> 1] = pack_h2(y[2][0], y[2][1]);
                zl[k >> 1] = pack_h2(y[3][0], y[3][1]);
            }
        }
        const int plane = lane / kPer * 4 * B * 2 + 2 * at;
        *reinterpret_cast<uint4*>(hb + off_s(B, BITS) + 2 * at) = make_uint4(sh[0], sh[1], sh[2], sh[3]);
        *reinterpret_cast<uint4*>(hb + off_z(B, BITS) + 2 * at) = make_uint4(zh[0], zh[1], zh[2], zh[3]);
        *reinterpret_cast<uint4*>(rest + plane) = make_uint4(sl[0], sl[1], sl[2], sl[3]);
        *reinterpret_cast<uint4*>(rest + kRest + plane) = make_uint4(zl[0], zl[1], zl[2], zl[3]);
    }
    return v_exp + c_exp;
}

// A pair of values as two fp16 halves.
__device__ __forceinline__ void build_pair(uint32_t code, __half2 sh, __half2 zh, __half2 sl, __half2 zl, __half2 c, uint32_t& hi, uint32_t& lo) {
    const __half2 f = u32_as_h2(code);
    const __half2 top = __hfma2(f, sh, zh), rest = __hfma2(f, sl, zl);
    const __half2 h = __hmul2(top, c);
    hi = h2_as_u32(h);
    lo = h2_as_u32(__hfma2(rest, c, __hfma2(top, c, __hneg2(h))));
}
__device__ __forceinline__ __half2 scaled_channels(uint32_t c, float up) {
    const float2 f = __half22float2(u32_as_h2(c));
    return __floats2half2_rn(f.x * up, f.y * up);
}
// Both halves of a register one of them.
__device__ __forceinline__ __half2 both(uint32_t x, int high) { return u32_as_h2(__byte_perm(x, x, high ? 0x3232 : 0x1010)); }

// K' of group g of the 32 records of half sb of a tile, a record a lane: tokens 4 (lane / 4) + k,
// channels 32 g + 8 (lane % 4) .. + 7. hb: the half's K head-block, rest: its rests; up:
// 2^-(C's exponent); ready(): waits until dst (hi, then lo) may be written (false: gave up).
template <int B, int BITS, typename Ready>
__device__ __forceinline__ bool tree_keys(const uint8_t* hb, const uint8_t* rest, int g, int sb, int lane, float up, uint8_t* dst, Ready&& ready) {
    const int ra = lane >> 2, rb = lane & 3;
    const int half0 = B == 64 ? 32 * sb : 0;             // the half's first token within its block
    const uint8_t* codes = hb + (half0 + lane) * 16 * BITS;
    uint32_t w[4], hw[4];              // token k's word with this group's fields at its low end
    const uint4* src = reinterpret_cast<const uint4*>(codes);
    if constexpr (BITS == 4) {         // word 4 k + g
        // (records are 16 words apart, two banks for all lanes: in load j a lane takes k = j + lane / 2,
        // 8 banks, and turns the words back in registers)
        const int turn = lane >> 1 & 3;
        uint32_t x[4], y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = reinterpret_cast<const uint32_t*>(codes)[4 * (j + turn & 3) + g];
#pragma unroll
        for (int k = 0; k < 4; ++k) y[k] = turn & 1 ? x[k + 3 & 3] : x[k];
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = turn & 2 ? y[k + 2 & 3] : y[k];
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
    const int at = 2 * (g * B + half0 + 4 * ra), block = B == 64 ? 0 : sb * 4 * B * 2;
    const uint2 sh = *reinterpret_cast<const uint2*>(hb + off_s(B, BITS) + at);
    const uint2 zh = *reinterpret_cast<const uint2*>(hb + off_z(B, BITS) + at);
    const uint2 sl = *reinterpret_cast<const uint2*>(rest + block + at);
    const uint2 zl = *reinterpret_cast<const uint2*>(rest + kRest + block + at);
    const uint4 cu = *reinterpret_cast<const uint4*>(hb + off_C(B, BITS) + 2 * (32 * g + 8 * rb));
    const __half2 c[4] = {scaled_channels(cu.x, up), scaled_channels(cu.y, up), scaled_channels(cu.z, up), scaled_channels(cu.w, up)};
    if (!ready()) return false;
    dst += (g >> 1) * (kPkK / 2);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const __half2 s1 = both(k < 2 ? sh.x : sh.y, k & 1), z1 = both(k < 2 ? zh.x : zh.y, k & 1);
        const __half2 s2 = both(k < 2 ? sl.x : sl.y, k & 1), z2 = both(k < 2 ? zl.x : zl.y, k & 1);
        const uint32_t w8 = w[k] >> 8;
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) build_pair(code_pair<BITS>(w[k], w8, hw[k], p, p), s1, z1, s2, z2, c[p], hi[p], lo[p]);
        const uint32_t to = swizzled(32 * sb + 4 * ra + k, 4 * (g & 1) + rb);
        // (an absent half's scores are masked, whatever its raw bytes were)
        *reinterpret_cast<uint4*>(dst + to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(dst + kPkK + to) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
    return true;
}

// V' likewise: channels 32 g + 4 (lane / 4) + k, tokens 8 (lane % 4) .. + 7 of the half. `there`: the
// half is (else, whatever its raw bytes are, its values are zeros).
template <int B, int BITS, typename Ready>
__device__ __forceinline__ bool tree_values(const uint8_t* vb, const uint8_t* rest, bool there, int g, int sb, int lane, float up, uint8_t* dst,
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
    const int at = 2 * (g * B + half0 + 8 * rb), block = B == 64 ? 0 : sb * 4 * B * 2;
    const uint4 sh = *reinterpret_cast<const uint4*>(vb + off_s(B, BITS) + at);
    const uint4 zh = *reinterpret_cast<const uint4*>(vb + off_z(B, BITS) + at);
    const uint4 sl = *reinterpret_cast<const uint4*>(rest + block + at);
    const uint4 zl = *reinterpret_cast<const uint4*>(rest + kRest + block + at);
    const uint32_t s1[4] = {sh.x, sh.y, sh.z, sh.w}, z1[4] = {zh.x, zh.y, zh.z, zh.w};
    const uint32_t s2[4] = {sl.x, sl.y, sl.z, sl.w}, z2[4] = {zl.x, zl.y, zl.z, zl.w};
    const uint2 cu = *reinterpret_cast<const uint2*>(vb + off_C(B, BITS) + 2 * (32 * g + 4 * ra));
    const uint32_t c[2] = {h2_as_u32(scaled_channels(cu.x, up)), h2_as_u32(scaled_channels(cu.y, up))};
    if (!ready()) return false;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t w8 = w[k] >> 8;
        const __half2 ck = both(c[k >> 1], k & 1);
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) {                 // tokens 2p, 2p + 1
            const int j = BITS == 4 ? p : 4 * (p >> 1) + 2 * (p & 1) + (k & 1);
            build_pair(code_pair<BITS>(w[k], w8, hw, j, 8 * (k >> 1) + j), u32_as_h2(s1[p]), u32_as_h2(z1[p]), u32_as_h2(s2[p]),
                       u32_as_h2(z2[p]), ck, hi[p], lo[p]);
            if (!there) hi[p] = lo[p] = 0u;
        }
        const uint32_t to = swizzled(32 * g + 4 * ra + k, 4 * sb + rb);
        *reinterpret_cast<uint4*>(dst + to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(dst + kPkV + to) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
    return true;
}

// ---------------------------------------------------------------- cached tokens
struct TreePackedSmem {
    // of raw tiles of keys and of values: ready: the levels are prepared; raw_empty: the operands are built
    uint64_t raw_full[2][kMaxRaw], ready[2][kMaxRaw], raw_empty[2][kMaxRaw];
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_ready[2], o_full[2], q_full, drained;
    uint32_t tmem;
    int stop;
    // the exponents of the last tiles [K, V], and of their C: the warps that find them are at most kMaxRaw
    // tiles ahead of the operands that are built, and those at most three ahead of the softmax. The softmax of a
    // tile follows the keys by way of S but nothing of its values, so that exps has the tile's
    // number in its upper half, which the softmax waits for
    int exps[2][8], c_exps[2][8];
};

// A tile's number (its low 16 bits) and exponent; the exponent of tile g, waited for (the limit
// run out: raises stop, with which the call's result is void).
__device__ __forceinline__ int tile_exps(int g, int e) { return (int)((uint32_t)g << 16 | (uint32_t)e & 0xffffu); }
__device__ __forceinline__ int exponent_of(const int* at, int g, int* stop) {
    int x = *reinterpret_cast<const volatile int*>(at);
    if (((uint32_t)x >> 16) != ((uint32_t)g & 0xffffu)) {   // (seldom: its tile is on its way two tiles ahead)
#pragma unroll 1
        for (uint32_t n = 0; ((uint32_t)x >> 16) != ((uint32_t)g & 0xffffu); ++n) {
            if (n == kWaitLimit) *reinterpret_cast<volatile int*>(stop) = 1;
            if (*reinterpret_cast<volatile int*>(stop)) break;
            x = *reinterpret_cast<const volatile int*>(at);
        }
    }
    __syncwarp();
    return (int16_t)x;
}

template <int B, int BITS, int NT>
struct TreePackedLayout {
    static constexpr int kSoft = 4 * NT, kThreads = 32 * (kSoft + 3 + 2 * kTreeBuild);
    static constexpr int HB = head_block_bytes(B, BITS);
    static constexpr int kBlocks = kPkTok / B;                 // blocks per tile
    static constexpr int kTile = kBlocks * HB;                 // bytes of a raw tile of keys or of values: its blocks,
    static constexpr int kRaw = kTile + 2 * kRest;             // and the rests of its levels [S, Z]
    static constexpr int kHeader = 1024;
    static_assert(sizeof(TreePackedSmem) <= kHeader, "header");
    static constexpr int kQLowBytes = NT == 2 ? 2 * kPkQ : 0;  // (with one row tile in tensor memory)
    static constexpr int kFixed = 1024 + kHeader + kQLowBytes + 4 * kPkK + 4 * kPkV;
    static constexpr int kFit = (227 * 1024 - kFixed) / (2 * kRaw);
    static constexpr int kRawStages = kFit < kMaxRaw ? kFit : kMaxRaw;
    static_assert(kRawStages >= 2, "a raw tile in flight while another is built");
    static constexpr size_t bytes = kFixed + 2 * kRawStages * kRaw;
};

template <int B, int BITS, int NT>
__global__ void __launch_bounds__(TreePackedLayout<B, BITS, NT>::kThreads, 1) tree_packed_kernel(TreeArgs a) {
    // (it starts beside tree_rotate_kernel, which has waited for what came before; the softmax warps
    // wait for the turned queries, so that this grid ends behind that one)
    let_next_grid_start();   // the join
    using Lay = TreePackedLayout<B, BITS, NT>;
    constexpr int kSoft = Lay::kSoft, kRawStages = Lay::kRawStages, TOK = kPkTok;
    extern __shared__ uint8_t raw_smem[];
    uint8_t* base = raw_smem + ((1024 - (smem_addr(raw_smem) & 1023)) & 1023);
    TreePackedSmem& s = *reinterpret_cast<TreePackedSmem*>(base);
    uint8_t* q_lo = base + Lay::kHeader;          // [row tile]
    uint8_t* k_op = q_lo + Lay::kQLowBytes;       // [stage][hi, lo]
    uint8_t* v_op = k_op + 4 * kPkK;              // [stage][hi, lo]
    uint8_t* raw = v_op + 4 * kPkV;               // [K, V][raw stage]: blocks, rests
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rt = blockIdx.x % a.row_tiles;
    const int64_t range = blockIdx.x / a.row_tiles;

    TreeCursor c = {};
    const int64_t W = tree_locate<TOK, true>(a, -1, lane, c), n_ranges = tree_ranges(W, a.ranges);
    if (range >= n_ranges) {
        wait_prior_grids();
        return;
    }
    const int64_t x_beg = range * W / n_ranges;
    const int total = (int)((range + 1) * W / n_ranges - x_beg);   // tiles of this CTA
    tree_locate<TOK, true>(a, x_beg, lane, c);

    // softmax warps of row tile x that have rows (one at least): the others leave at once
    const auto alive = [&](int x) { return min(4, max(1, (a.drafts * a.G - (rt * NT + x) * kPRows + 31) / 32)); };
    if (tid == 0) {
        s.stop = 0;
        for (int i = 0; i < 8; ++i) s.exps[0][i] = s.exps[1][i] = -1;   // (no tile 65535 that is the first of its place)
        for (int i = 0; i < 2 * kRawStages; ++i) {
            mbar_init(&s.raw_full[i & 1][i >> 1], 1);
            mbar_init(&s.ready[i & 1][i >> 1], 1);
            mbar_init(&s.raw_empty[i & 1][i >> 1], kTreeBuild);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.k_full[i], kTreeBuild);
            mbar_init(&s.k_empty[i], 1);
            mbar_init(&s.v_full[i], kTreeBuild);
            mbar_init(&s.v_empty[i], 1);
            mbar_init(&s.s_full[i], 1);
            mbar_init(&s.p_ready[i], NT == 2 ? alive(i) : alive(0));
            mbar_init(&s.o_full[i], 1);
        }
        mbar_init(&s.q_full, NT == 2 ? alive(0) + alive(1) : alive(0));
        mbar_init(&s.drained, 1);
        fence_mbar_init();
    }
    if (warp == kSoft) tmem_alloc(&s.tmem, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // Q of row tile x at + 64 x; S (and P) at + 64 w, of tile g, w = g % 2 (NT 1), or of row
    // tile w (NT 2); O at + 128 x
    const uint32_t tm_q = __reduce_max_sync(kFull, s.tmem), tm_s = tm_q + 128, tm_o = tm_q + 256;   // (uniform to the compiler)
    int* stop = &s.stop;
    int fetched = 0;                              // raw tiles whose copies have been issued
    int g = 0;                                    // tiles of this CTA so far
    bool ok = true;

    if (warp == kSoft + 1 || warp == kSoft + 2) {
        // ---------------------------------------------------------- raw tiles and their levels: a warp for the keys, one for the values
        // (in rings of their own: a tile's values are built two tiles behind its keys)
        const int kind = warp - (kSoft + 1);
        uint8_t* ring = raw + kind * kRawStages * Lay::kRaw;
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
            const uint32_t bytes = __popc(__ballot_sync(kFull, page >= 0)) * Lay::HB;
            if (lane == 0) mbar_arrive_expect_tx(&s.raw_full[kind][st], bytes);
            __syncwarp();
            if (page >= 0)
                bulk_g2s(ring + st * Lay::kRaw + lane * Lay::HB, a.pool + page * a.block_bytes + (int64_t)(2 * f.h + kind) * Lay::HB,
                         Lay::HB, &s.raw_full[kind][st]);
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
                    ok = warp_wait_or_stop(&s.raw_empty[kind][fetched % kRawStages], (fetched / kRawStages - 1) & 1, stop, kWaitLimit);
                if (ok) fetch();
            }
            const int st = g % kRawStages;
            ok = ok && warp_wait_or_stop(&s.raw_full[kind][st], (g / kRawStages) & 1, stop, kWaitLimit);
            if (!ok) break;
            const int x = lane / (32 / Lay::kBlocks);              // this lane's block
            const bool there = c.t * Lay::kBlocks + x < c.tokens / B;
            uint8_t* tile = ring + st * Lay::kRaw;
            int c_exp;
            const int e = prepare_levels<B, BITS>(tile + x * Lay::HB, there, lane, tile + Lay::kTile, c_exp);
            fence_async_smem();                   // (before the stage's next copy writes over it)
            if (lane == 0) {
                *reinterpret_cast<volatile int*>(&s.exps[kind][g & 7]) = tile_exps(g, e);
                s.c_exps[kind][g & 7] = c_exp;
            }
            warp_arrive(&s.ready[kind][st]);
            if (++c.t == c.tiles && g + 1 < total) tree_next<TOK, true>(a, c);
        }
    } else if (warp > kSoft) {
        // ---------------------------------------------------------- operands from codes
        // kTreeBuild warps the keys, as many the values; a warp has group grp of the 32 records of
        // one half of the tile, or of both, a record a lane
        const int kind = (warp - (kSoft + 3)) / kTreeBuild, bw = (warp - (kSoft + 3)) % kTreeBuild, grp = bw & 3;
        for (; g < total && ok; ++g) {
            const int st = g % kRawStages, par = g & 1;
            // (the copies' barrier has been waited for by the warp that prepared the levels)
            ok = warp_wait_or_stop(&s.ready[kind][st], (g / kRawStages) & 1, stop, kWaitLimit);
            if (!ok) break;
            const uint8_t* tile = raw + (kind * kRawStages + st) * Lay::kRaw;
            const float up = exp2i(-*reinterpret_cast<volatile int*>(&s.c_exps[kind][g & 7]));
#pragma unroll 1
            for (int sb = bw >> 2; sb < 2 && ok; sb += kTreeBuild / 4) {
                const uint8_t* hb = tile + (B == 64 ? 0 : sb) * Lay::HB;
                const bool wait = g >= 2 && sb == bw >> 2;
                if (kind == 0) {
                    ok = tree_keys<B, BITS>(hb, tile + Lay::kTile, grp, sb, lane, up, k_op + par * 2 * kPkK, [&] {
                        return !wait || warp_wait_or_stop(&s.k_empty[par], ((g >> 1) - 1) & 1, stop, kWaitLimit);
                    });
                } else {
                    const bool there = B == 64 || c.t * Lay::kBlocks + sb < c.tokens / B;   // else its values are zero
                    ok = tree_values<B, BITS>(hb, tile + Lay::kTile, there, grp, sb, lane, up, v_op + par * 2 * kPkV, [&] {
                        return !wait || warp_wait_or_stop(&s.v_empty[par], ((g >> 1) - 1) & 1, stop, kWaitLimit);
                    });
                }
            }
            if (!ok) break;
            fence_async_smem();
            warp_arrive(kind ? &s.v_full[par] : &s.k_full[par]);
            warp_arrive(&s.raw_empty[kind][st]);
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
                    const uint32_t vd = v_desc + (tj & 1) * (2 * kPkV >> 4);
                    run_pv_packed(tm_o + 128 * x, tm_s + 64 * w, vd, vd + (kPkV >> 4), kPv, j >= NT);
                    if (trail) mma_commit(&s.v_empty[tj & 1]);
                    if (tj == g + n - 1) mma_commit(&s.o_full[x]);
                }
                // (the keys' wait comes behind the products that do not need them)
                if (i < NT * n && lead) ok = warp_wait_or_stop(&s.k_full[ti & 1], (ti >> 1) & 1, stop, kWaitLimit);
                if (!ok) break;
                tc_fence_after();
                if (i < NT * n) {
                    const uint32_t kd = k_desc + (ti & 1) * (2 * kPkK >> 4);
                    if (NT == 1) run_qk_packed(tm_s + 64 * w, tm_q, tm_q + kQLow, kd, kd + (kPkK >> 4), kQk);
                    else run_qk_packed_low(tm_s + 64 * w, tm_q + 64 * x, q_desc + x * (kPkQ >> 4), kd, kd + (kPkK >> 4), kQk);
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
        wait_prior_grids();
        const int x = warp >> 2;                                  // row tile of the CTA
        const int r = rt * NT * kPRows + tid;                     // this thread's query row of a unit
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t my_o = tm_o + 128 * x + lanes;
        int units = 0;
        if ((warp & 3) >= alive(x)) g = total;
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
                    if (NT == 2) *reinterpret_cast<uint4*>(q_lo + x * kPkQ + (at >> 3) * (kPkQ / 2) + swizzled((warp & 3) * 32 + lane, at & 7)) = lo[i];
                }
                tmem_st16(tm_q + 64 * x + 16 * k + lanes, y);
                if (NT == 1) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) y[4 * i] = lo[i].x, y[4 * i + 1] = lo[i].y, y[4 * i + 2] = lo[i].z, y[4 * i + 3] = lo[i].w;
                    tmem_st16(tm_q + kQLow + 16 * k + lanes, y);
                }
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
                const int e = exponent_of(&s.exps[1][g & 7], g, stop);
                // (finite and not 0, so that what is masked stays masked)
                const float here = fminf(fmaxf(scale * exp2i((int16_t)*reinterpret_cast<volatile int*>(&s.exps[0][g & 7])), 0x1p-126f), 0x1p127f);
                ok = softmax_rolled<TOK, true>(tm_s + 64 * w + lanes, my_o, len - (c.t + i) * TOK, here, (float)e, exp2i(-e),
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
        if (warp == kSoft + 1 || warp == kSoft + 2)
            for (int i = max(0, fetched - kRawStages); i < fetched; ++i)
                mbar_wait_bounded(&s.raw_full[warp - (kSoft + 1)][i % kRawStages], (i / kRawStages) & 1, kWaitLimit);
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
