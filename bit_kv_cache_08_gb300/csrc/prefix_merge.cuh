// prefix_merge.cuh -- the merge behind a shared-prefix kernel: the partials of
// the prefix's token ranges and what the own tokens give, in the log-sum-exp
// sense; raw tail rows of the packed cache on the way. A CTA serves one
// (sequence, kv head): its warps share out the G query heads, several to a head.
#pragma once
#include "prefix.cuh"

namespace kvarn {

constexpr int kMergeWarps = 8;
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
// p0, pstride apart, then the prefix's at s0, sstride apart), 8 in flight at a
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

__device__ __forceinline__ void async_copy16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void async_copy_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

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
    const float inv = l > 0.f ? 1.f / l : 0.f;
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

// The raw tail rows in shared memory, PER of them in every REGION bytes: K,
// then V 272 bytes on; rows 528 bytes apart, so that lanes that score a row
// each read different banks.
template <int PER, int REGION>
struct TailRows {
    static constexpr int kPitch = 2 * kD * 2 + 16, kBytes = PER * kPitch;
    uint8_t* base;
    __device__ __forceinline__ uint8_t* k(int i) const { return base + i / PER * REGION + i % PER * kPitch; }
    __device__ __forceinline__ uint8_t* v(int i) const { return k(i) + kD * 2 + 16; }
};

// The whole CTA starts the copies of the first ntail staging rows.
template <int B, typename Rows>
__device__ __forceinline__ void copy_tail(const AttnArgs& a, const Rows& rows, int b, int h, int ntail) {
    const uint16_t* st = a.staging + ((int64_t)b * a.n_kv + h) * 2 * B * kD;
    for (int i = threadIdx.x; i < ntail * 16; i += 32 * kMergeWarps) {
        async_copy16(rows.k(i >> 4) + (i & 15) * 16, st + i * 8);
        async_copy16(rows.v(i >> 4) + (i & 15) * 16, st + B * kD + i * 8);
    }
}

// A warp's share (at most 32) of the tail rows against query row `row` as a
// slice, unrotated: a lane scores a row.
template <typename Rows>
__device__ __forceinline__ void tail_share(const AttnArgs& a, const Rows& rows, int ntail, int part, int parts, int64_t row,
                                           int lane, float* tail) {
    const int c0 = ntail * part / parts, cnt = ntail * (part + 1) / parts - c0;
    float qv[4];
    load_q4(a.q, a.q_dtype, row, lane, qv);
    const float qs = a.sm_scale * kLog2e;
    *reinterpret_cast<float4*>(&tail[4 * lane]) = make_float4(qv[0] * qs, qv[1] * qs, qv[2] * qs, qv[3] * qs);
    __syncwarp();
    float s = -INFINITY;
    if (lane < cnt) {
        const uint4* kr = reinterpret_cast<const uint4*>(rows.k(c0 + lane));
        s = 0.f;
#pragma unroll 4
        for (int c = 0; c < 16; ++c) {
            const uint4 k = kr[c];
            const float4 qa = *reinterpret_cast<const float4*>(&tail[8 * c]);
            const float4 qb = *reinterpret_cast<const float4*>(&tail[8 * c + 4]);
            s = fmaf(qa.x, __uint_as_float(k.x << 16), s);
            s = fmaf(qa.y, __uint_as_float(k.x & 0xffff0000u), s);
            s = fmaf(qa.z, __uint_as_float(k.y << 16), s);
            s = fmaf(qa.w, __uint_as_float(k.y & 0xffff0000u), s);
            s = fmaf(qb.x, __uint_as_float(k.z << 16), s);
            s = fmaf(qb.y, __uint_as_float(k.z & 0xffff0000u), s);
            s = fmaf(qb.z, __uint_as_float(k.w << 16), s);
            s = fmaf(qb.w, __uint_as_float(k.w & 0xffff0000u), s);
        }
    }
    const float tm = warp_max(s);
    const float p = s == -INFINITY ? 0.f : exp2f(s - tm);
    const float tl = warp_sum(p);
    float tacc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int i = 0; i < cnt; ++i) {
        const float w = __shfl_sync(kFull, p, i);
        const uint2 v = reinterpret_cast<const uint2*>(rows.v(c0 + i))[lane];
        tacc[0] = fmaf(w, __uint_as_float(v.x << 16), tacc[0]);
        tacc[1] = fmaf(w, __uint_as_float(v.x & 0xffff0000u), tacc[1]);
        tacc[2] = fmaf(w, __uint_as_float(v.y << 16), tacc[2]);
        tacc[3] = fmaf(w, __uint_as_float(v.y & 0xffff0000u), tacc[3]);
    }
    __syncwarp();   // (the query has been read)
    if (lane == 0) {
        tail[0] = tm;
        tail[1] = tl;
    }
    *reinterpret_cast<float4*>(&tail[4 + 4 * lane]) = make_float4(tacc[0], tacc[1], tacc[2], tacc[3]);
}

// A row's merged result (own and prefix tokens) rotated back (ROT), joined
// with its tail slices (tails, one for each of `parts` warps; nullptr: no tail)
// and stored.
template <bool ROT>
__device__ __forceinline__ void finish_row(const AttnArgs& a, const PrefixMerge& pm, int64_t row, const float* tails, int parts,
                                           int lane, float m, float l, float (&acc)[4]) {
    if (ROT && !(a.flags & KVARN_FLAG_NO_ROTATION)) {
        fwht128(acc, lane);
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[k] *= kInvSqrtD * sign_of4(a.sb[0], a.sb[1], a.sb[2], a.sb[3], 4 * lane + k);
    }
    if (tails) {
        float mt = -INFINITY, lt = 0.f, at[4] = {0.f, 0.f, 0.f, 0.f};
        combine_slices(tails, parts, lane, mt, lt, at);
        add_slice(m, l, acc, mt, lt, at);
    }
    store_out(pm, row, lane, l, acc);
}

}  // namespace kvarn
