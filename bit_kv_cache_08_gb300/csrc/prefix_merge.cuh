// prefix_merge.cuh -- the merge behind a shared-prefix kernel: the partials of
// the prefix's token ranges and what the own tokens give, in the log-sum-exp
// sense; raw tail rows of the packed cache on the way. A CTA serves one
// (sequence, kv head): its warps share out the G query heads, several to a head.
#pragma once
#include "prefix.cuh"

namespace kvarn {

// Warps to a query head (G = 3: the CTA's last ones are left over).
__device__ __forceinline__ int merge_parts(int G, int warps) { return G == 1 ? warps : G == 2 ? warps / 2 : warps / 4; }

struct PrefixMerge {
    const float* partials;
    const int32_t* lens;
    int max_len;
    int splits;
    void* out;
    int out_bf16;
};

// LSE merge of the partials first .. last - 1 of a row's list (np own ones at
// p0, pstride apart, then the prefix's at s0, sstride apart), NB in flight at a
// time with a running rescale; m, l and acc start at -inf, 0 and 0.
template <int NB>
__device__ __forceinline__ void lse_list(const float* p0, int np, int64_t pstride, const float* s0, int64_t sstride, int first,
                                         int last, int lane, float& m, float& l, float (&acc)[4]) {
    auto at = [&](int i) { return i < np ? p0 + i * pstride : s0 + (i - np) * sstride; };
    for (int i0 = first; i0 < last; i0 += NB) {
        const int cnt = min(NB, last - i0);
        float2 ml = make_float2(-INFINITY, 0.f);
        if (lane < cnt) ml = __ldcg(reinterpret_cast<const float2*>(at(i0 + lane)));
        float4 pa[NB];
#pragma unroll
        for (int i = 0; i < NB; ++i)
            if (i < cnt) pa[i] = __ldcg(reinterpret_cast<const float4*>(at(i0 + i) + 4) + lane);
        const float bm = warp_max(ml.x);
        if (bm == -INFINITY) continue;
        const float mn = fmaxf(m, bm);
        const float fa = m == -INFINITY ? 0.f : exp2f(m - mn);
        const float wl = ml.x == -INFINITY ? 0.f : exp2f(ml.x - mn);
        l = l * fa + warp_sum(ml.y * wl);
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[k] *= fa;
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            if (i < cnt) {
                const float wgt = __shfl_sync(kFull, wl, i);
                acc[0] = fmaf(wgt, pa[i].x, acc[0]);
                acc[1] = fmaf(wgt, pa[i].y, acc[1]);
                acc[2] = fmaf(wgt, pa[i].z, acc[2]);
                acc[3] = fmaf(wgt, pa[i].w, acc[3]);
            }
        }
        m = mn;
    }
}

// (m, l, acc) += (ms, ls, as) in the log-sum-exp sense.
__device__ __forceinline__ void add_slice(float& m, float& l, float (&acc)[4], float ms, float ls, const float (&as)[4]) {
    if (ms == -INFINITY) return;
    const float mn = fmaxf(m, ms);
    const float fa = m == -INFINITY ? 0.f : exp2f(m - mn), fs = exp2f(ms - mn);
    l = l * fa + ls * fs;
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[k] = acc[k] * fa + as[k] * fs;
    m = mn;
}

__device__ __forceinline__ void store_out(const PrefixMerge& pm, int64_t row, int lane, float l, float (&acc)[4]) {
    const float inv = l > 0.f ? 1.f / l : l;   // (0 for no token at all; NaN stays)
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[k] *= inv;
    if (pm.out_bf16) {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(acc[0], acc[1]), hi = __floats2bfloat162_rn(acc[2], acc[3]);
        reinterpret_cast<uint2*>(static_cast<uint16_t*>(pm.out) + row * kD)[lane] =
            make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    } else {
        reinterpret_cast<float4*>(static_cast<float*>(pm.out) + row * kD)[lane] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    }
}

// A sequence with a length outside its range: NaN and the error word.
__device__ __forceinline__ void refuse_row(const AttnArgs& a, const PrefixMerge& pm, int b, int h) {
    if (threadIdx.x == 0) raise_error(a.err, KVARN_DEVERR_POSITION);
    for (int i = threadIdx.x; i < a.G * kD; i += blockDim.x) {
        const int64_t at = ((int64_t)b * a.n_q + h * a.G) * kD + i;
        if (pm.out_bf16) static_cast<uint16_t*>(pm.out)[at] = 0x7fc0;
        else static_cast<float*>(pm.out)[at] = NAN;
    }
}

template <int B>
__device__ __forceinline__ bool lengths_ok(const AttnArgs& a, const PrefixMerge& pm, int L, int PL) {
    return L >= 0 && L <= a.max_blocks * B && PL >= 0 && PL <= pm.max_len;
}

__device__ __forceinline__ void put_slice(float* s, int lane, float m, float l, const float (&acc)[4]) {
    if (lane == 0) {
        s[0] = m;
        s[1] = l;
    }
    *reinterpret_cast<float4*>(s + 4 + 4 * lane) = make_float4(acc[0], acc[1], acc[2], acc[3]);
}

// A warp's share of the prefix's partials of (sequence b, query head g of kv
// head h) as a slice.
__device__ __forceinline__ void prefix_slice(const AttnArgs& a, const PrefixMerge& pm, int b, int h, int g, int part, int parts,
                                             int PL, int lane, float* slice) {
    float m = -INFINITY, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
    const int n = PL > 0 ? pm.splits : 0;
    const int64_t R = (int64_t)a.batch * a.G;
    lse_list<16>(nullptr, 0, 0, pm.partials + partial_row(0, a.n_kv, h, R, (int64_t)b * a.G + g),
                 partial_row(1, a.n_kv, 0, R, 0), n * part / parts, n * (part + 1) / parts, lane, m, l, acc);
    put_slice(slice, lane, m, l, acc);
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t bf16_pair(float v0, float v1, bool low) {   // RN(v), or RN(v - RN(v))
    const __nv_bfloat162 h = __floats2bfloat162_rn(v0, v1);
    if (!low) return *reinterpret_cast<const uint32_t*>(&h);
    const float2 f = __bfloat1622float2(h);
    const __nv_bfloat162 r = __floats2bfloat162_rn(v0 - f.x, v1 - f.y);
    return *reinterpret_cast<const uint32_t*>(&r);
}

struct ChunkRows {
    int64_t at;   // bytes from the base to K's rows (128 channels, 256 bytes apart); V's are B rows behind
    int rows;     // that there are (16 and more: all)
};
// n chunks of 16 bf16 tokens (chunk(i): the whole warp calls it) against the G
// queries of (sequence b, kv head h), a slice for each in own[head][wp]. Both
// products run on mma.sync with the columns (head, high | low half of q or of
// p), as in attention_bf16.cu. The fragments are loaded straight from memory:
// the order of the channels in S and of the output rows in O is free, so a
// lane's 16-byte loads of K (token gq, channels 32 j + 8 tq ..) and V (channels
// 64 j + 8 gq .. of the four tokens its A fragment holds) are whole fragments,
// and nothing passes through shared memory but q. K, V and O take 96 registers
// a lane: with a chunk's loads at the end of the one before, 128 did not hold
// them (112 instead of 106 us for 128 x 384 own tokens behind 32 768).
template <int B, int W, int SLICES, typename At>
__device__ __forceinline__ void bf16_slice(const AttnArgs& a, int b, int h, int n, const uint8_t* base, const At& chunk, int wp, int lane,
                                           uint2 (*qf)[32], float (*own)[SLICES][kPartialStride]) {
    const int gq = lane >> 2, tq = lane & 3;
    const int head = gq >> 1;          // this lane's column of the products: (head, high | low half)
    const bool low = gq & 1;
    const uint8_t* lane_k = base + gq * (kD * 2) + tq * 16;
    const uint8_t* lane_v = base + B * kD * 2 + 2 * tq * (kD * 2) + gq * 16;
    uint4 k[2][4], v[4][2];
    auto load_k = [&](const ChunkRows& c) {
        const uint8_t* p = lane_k + c.at;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                k[t][j] = 8 * t + gq < c.rows ? __ldcg(reinterpret_cast<const uint4*>(p + 8 * t * (kD * 2) + 64 * j))
                                            : make_uint4(0u, 0u, 0u, 0u);
    };
    auto load_v = [&](const ChunkRows& c) {
        const uint8_t* p = lane_v + c.at;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int row = (t & 1) + 8 * (t >> 1);
#pragma unroll
            for (int j = 0; j < 2; ++j)
                v[t][j] = 2 * tq + row < c.rows ? __ldcg(reinterpret_cast<const uint4*>(p + row * (kD * 2) + 128 * j))
                                              : make_uint4(0u, 0u, 0u, 0u);
        }
    };
    ChunkRows now{0, 0};
    if (n > 0) {   // (the first one's loads go ahead of the query's)
        now = chunk(0);
        load_k(now);
        load_v(now);
    }
    for (int ks = wp; ks < 8; ks += W) {   // the query as the B operand of each k-step, a column for each (head, high | low half)
        const int c = 32 * (ks >> 1) + 8 * tq + 4 * (ks & 1);
        const int64_t at_q = ((int64_t)b * a.n_q + h * a.G + min(head, a.G - 1)) * kD + c;
        float x[4];
        if (a.q_dtype == KVARN_FP32) {
            *reinterpret_cast<float4*>(x) = *reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + at_q);
        } else {
            const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.q) + at_q);
            x[0] = __uint_as_float(u.x << 16);
            x[1] = __uint_as_float(u.x & 0xffff0000u);
            x[2] = __uint_as_float(u.y << 16);
            x[3] = __uint_as_float(u.y & 0xffff0000u);
        }
        qf[ks][lane] = make_uint2(bf16_pair(x[0], x[1], low), bf16_pair(x[2], x[3], low));
    }
    __syncthreads();
    float o[8][4], m = -INFINITY, l = 0.f;   // o[4 i + e]: channels 64 i + 8 gq + 2 e (+ 1), head tq high | low
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    const float qs = a.sm_scale * kLog2e;
    for (int i = 0; i < n; ++i) {
        if (i > 0) {
            now = chunk(i);
            load_k(now);
            load_v(now);
        }
        float s[4] = {0.f, 0.f, 0.f, 0.f};   // tokens gq and gq + 8, head tq high | low
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint2 q0 = qf[2 * j][lane], q1 = qf[2 * j + 1][lane];
            mma_bf16(s, k[0][j].x, k[1][j].x, k[0][j].y, k[1][j].y, q0.x, q0.y);
            mma_bf16(s, k[0][j].z, k[1][j].z, k[0][j].w, k[1][j].w, q1.x, q1.y);
        }
        const int here = now.rows;
        const float s0 = gq < here ? (s[0] + s[1]) * qs : -INFINITY, s1 = gq + 8 < here ? (s[2] + s[3]) * qs : -INFINITY;
        float bm = fmaxf(s0, s1);
        bm = fmaxf(bm, __shfl_xor_sync(kFull, bm, 4));
        bm = fmaxf(bm, __shfl_xor_sync(kFull, bm, 8));
        bm = fmaxf(bm, __shfl_xor_sync(kFull, bm, 16));
        const float mn = fmaxf(m, bm), off = mn == -INFINITY ? 0.f : mn;
        const float f = mn == -INFINITY ? 1.f : exp2f(m - mn), p0 = exp2f(s0 - off), p1 = exp2f(s1 - off);
        m = mn;
        l = l * f + (p0 + p1);
        if (__any_sync(kFull, f != 1.f)) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                o[e][0] *= f;
                o[e][1] *= f;
                o[e][2] *= f;
                o[e][3] *= f;
            }
        }
        // weights of tokens 2 tq, 2 tq + 1 and 2 tq + 8, 2 tq + 9 for this lane's column
        const int from = 8 * tq + head;
        const uint32_t b0 = bf16_pair(__shfl_sync(kFull, p0, from), __shfl_sync(kFull, p0, from + 4), low);
        const uint32_t b1 = bf16_pair(__shfl_sync(kFull, p1, from), __shfl_sync(kFull, p1, from + 4), low);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t* r0 = &v[0][j].x;
            const uint32_t* r1 = &v[1][j].x;
            const uint32_t* r2 = &v[2][j].x;
            const uint32_t* r3 = &v[3][j].x;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                mma_bf16(o[4 * j + e], __byte_perm(r0[e], r1[e], 0x5410), __byte_perm(r0[e], r1[e], 0x7632),
                         __byte_perm(r2[e], r3[e], 0x5410), __byte_perm(r2[e], r3[e], 0x7632), b0, b1);
        }
    }
    l += __shfl_xor_sync(kFull, l, 4);
    l += __shfl_xor_sync(kFull, l, 8);
    l += __shfl_xor_sync(kFull, l, 16);
    if (tq < a.G && (SLICES == W || wp < SLICES)) {
        float* sl = own[tq][wp];
        if (gq == 0) {
            sl[0] = m;
            sl[1] = l;
        }
#pragma unroll
        for (int e = 0; e < 8; e += 2)
            *reinterpret_cast<float4*>(sl + 4 + 64 * (e >> 2) + 8 * gq + 2 * (e & 3)) =
                make_float4(o[e][0] + o[e][1], o[e][2] + o[e][3], o[e + 1][0] + o[e + 1][1], o[e + 1][2] + o[e + 1][3]);
    }
}

// The first ntail raw rows of a unit's staging buffer, one chunk to a warp
// (the first four have them all), as slices of the unrotated query.
template <int B, int W>
__device__ __forceinline__ void tail_slice16(const AttnArgs& a, int b, int h, int ntail, int wp, int lane, uint2 (*qf)[32],
                                             float (*tails)[4][kPartialStride]) {
    const uint8_t* st = reinterpret_cast<const uint8_t*>(a.staging) + ((int64_t)b * a.n_kv + h) * 2 * B * kD * 2;
    const int rows = ntail - wp * kChunk;
    bf16_slice<B, W, 4>(a, b, h, rows > 0 ? 1 : 0, st, [&](int) { return ChunkRows{wp * kChunk * kD * 2, rows}; }, wp, lane, qf,
                        tails);
}

// A row's merged result (own and prefix tokens) rotated back (ROT), joined
// with its four tail slices (nullptr: no tail)
// and stored. Maxima drop NaN, so a row of tokens (any) without a score above
// -inf is one whose scores are NaN, or all -inf: its softmax is NaN.
template <bool ROT>
__device__ __forceinline__ void finish_row(const AttnArgs& a, const PrefixMerge& pm, int64_t row, bool any, const float* tails,
                                           int lane, float m, float l, float (&acc)[4]) {
    if (ROT && !(a.flags & KVARN_FLAG_NO_ROTATION)) {
        fwht128(acc, lane);
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[k] *= kInvSqrtD * sign_of4(a.sb[0], a.sb[1], a.sb[2], a.sb[3], 4 * lane + k);
    }
    if (tails) {
        float mt = -INFINITY, lt = 0.f, at[4] = {0.f, 0.f, 0.f, 0.f};
        combine_slices(tails, 4, lane, mt, lt, at);
        add_slice(m, l, acc, mt, lt, at);
    }
    if (any && m == -INFINITY) l = NAN;
    store_out(pm, row, lane, l, acc);
}

}  // namespace kvarn
