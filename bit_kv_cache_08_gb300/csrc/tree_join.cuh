// tree_join.cuh -- the end of the attention for a tree of drafted tokens: the
// partials of the cached tokens' ranges, the raw tail rows of the packed cache, and
// the drafts themselves.
//
// A warp takes 16 query rows of a (sequence, kv head) and holds O (16 x 128) as the
// accumulators of mma.sync m16n8k16: it joins the partials in the log-sum-exp sense, m = max m_i,
// l = sum l_i 2^(m_i - m), O = sum O_i 2^(m_i - m), turns O back (packed cache), and goes
// on as an online softmax over the raw bf16 rows, 16 tokens a step:
//   S = Q K^T   A = 16 query rows, B = 8 tokens; the order of the channels in the sum is
//               free, so a lane's 16-byte loads of Q and K are whole fragments
//   P           the accumulators of S are the A fragments of
//   O += P V    B = 8 channels; a lane's 16-byte loads of V's rows hold 8 channels, one for each
//               of 8 products, in which the lane's column stands for the channel
// P and an fp32 query enter as two bf16 halves (2^-16). The mask of a row is 16 bits of
// its words a step; a step that no row of the warp sees is left out. Where there
// are few rows, several warps share them: each takes its part of the partials and of the
// steps, and their states are joined through shared memory. Its time is a chain of loads (13 us alone and cold
// for 128 units of 64 rows, 24 for 256 of 132, of which a call sees about half); 16 or 24 warps an SM instead of
// 8 spill and lose (32 x 33 drafts over 8192 tokens 192 -> 197, 205 us).
#pragma once
#include "prefix_merge.cuh"
#include "tree.cuh"

namespace kvarn {

constexpr int kJoinRows = 16;

// Channel of accumulator x (0, 1: the lane's columns 2 tq, 2 tq + 1) of product (j, e):
// 64 j + 16 tq + 8 x + e. The Hadamard transform over channels, for rows gq (d = 0) and gq + 8
// (d = 2): all bits but those of tq lie within a lane.
__device__ __forceinline__ void fwht_fragment(float (&o)[2][8][4], int tq) {
#pragma unroll
    for (int m = 1; m <= 4; m <<= 1)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (!(e & m))
#pragma unroll
                    for (int d = 0; d < 4; ++d) {
                        const float x = o[j][e][d], y = o[j][e | m][d];
                        o[j][e][d] = x + y;
                        o[j][e | m][d] = x - y;
                    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e)
#pragma unroll
            for (int d = 0; d < 4; d += 2) {
                const float x = o[j][e][d], y = o[j][e][d + 1];
                o[j][e][d] = x + y;
                o[j][e][d + 1] = x - y;
            }
#pragma unroll
    for (int e = 0; e < 8; ++e)
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const float x = o[0][e][d], y = o[1][e][d];
            o[0][e][d] = x + y;
            o[1][e][d] = x - y;
        }
#pragma unroll
    for (int m = 1; m <= 2; m <<= 1) {
        const float sgn = (tq & m) ? -1.f : 1.f;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e)
#pragma unroll
                for (int d = 0; d < 4; ++d) o[j][e][d] = fmaf(sgn, o[j][e][d], __shfl_xor_sync(kFull, o[j][e][d], m));
    }
}

// The state of a warp's 16 rows: x = 0 is row gq, x = 1 row gq + 8. l is a sum over the
// lane's own columns, to be added over the four lanes of a row.
template <bool Q32>
struct JoinRows {
    uint32_t q[Q32 ? 2 : 1][8][4];   // A fragments [half][k-step]
    float o[2][8][4], m[2], l[2];
};

// 16 raw tokens at k and v (rows ks / vs elements apart), of which the first `there` exist;
// bit i of seen[x]: token i is shown to row x. APART: not every row sees every token, and a
// value that is not finite must not reach the rows that do not see it (0 times it is NaN):
// its row of V is taken as zeros, and wrong[x] says that the row has seen one.
template <bool Q32, bool APART>
__device__ __forceinline__ void join_step(JoinRows<Q32>& s, const uint16_t* k, const uint16_t* v, int64_t ks, int64_t vs, int there,
                                          const uint32_t (&seen)[2], float scale, int lane, bool (&wrong)[2]) {
    const int gq = lane >> 2, tq = lane & 3;
    uint4 kk[2][4], vv[4][2];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            kk[t][j] = 8 * t + gq < there ? *reinterpret_cast<const uint4*>(k + (8 * t + gq) * ks + 32 * j + 8 * tq) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const int row = 2 * tq + (t & 1) + 8 * (t >> 1);
#pragma unroll
        for (int j = 0; j < 2; ++j)
            vv[t][j] = row < there ? *reinterpret_cast<const uint4*>(v + row * vs + 64 * j + 8 * gq) : make_uint4(0, 0, 0, 0);
    }
    float sc[2][4];   // [8 tokens][row gq: tokens 2 tq, 2 tq + 1; row gq + 8]
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        sc[t][0] = sc[t][1] = sc[t][2] = sc[t][3] = 0.f;
#pragma unroll
        for (int p = 0; p < (Q32 ? 2 : 1); ++p)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                mma_bf16(sc[t], s.q[p][2 * j][0], s.q[p][2 * j][1], s.q[p][2 * j][2], s.q[p][2 * j][3], kk[t][j].x, kk[t][j].y);
                mma_bf16(sc[t], s.q[p][2 * j + 1][0], s.q[p][2 * j + 1][1], s.q[p][2 * j + 1][2], s.q[p][2 * j + 1][3], kk[t][j].z, kk[t][j].w);
            }
    }
    if constexpr (APART) {
        // values that are not finite: 0 times one is NaN, 0 times any other 0
        const __nv_bfloat162 zero = __floats2bfloat162_rn(0.f, 0.f);
        uint32_t bad = 0;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            __nv_bfloat162 n = zero;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t w[4] = {vv[t][j].x, vv[t][j].y, vv[t][j].z, vv[t][j].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) n = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&w[e]), zero, n);
            }
            const uint32_t bits = *reinterpret_cast<const uint32_t*>(&n);
            // lanes of the same tq hold the token's other channels
            const uint32_t lanes = __ballot_sync(kFull, (bits & 0x7fff7fffu) != 0);
#pragma unroll
            for (int x = 0; x < 4; ++x)
                if (lanes & 0x11111111u << x) bad |= 1u << (2 * x + (t & 1) + 8 * (t >> 1));
        }
        if (bad) {
#pragma unroll
            for (int t = 0; t < 4; ++t)
                if (bad >> (2 * tq + (t & 1) + 8 * (t >> 1)) & 1) vv[t][0] = vv[t][1] = make_uint4(0, 0, 0, 0);
            wrong[0] = wrong[0] || (bad & seen[0]);
            wrong[1] = wrong[1] || (bad & seen[1]);
        }
    }
    float p[2][4], f[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        float top = -INFINITY;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float& z = sc[t][2 * x + i];
                z = seen[x] >> (8 * t + 2 * tq + i) & 1 ? z * scale : -INFINITY;
                top = fmaxf(top, z);
            }
        top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
        top = fmaxf(top, __shfl_xor_sync(kFull, top, 2));
        const float mn = fmaxf(s.m[x], top), off = mn == -INFINITY ? 0.f : mn;
        f[x] = mn == -INFINITY ? 1.f : exp2f(s.m[x] - mn);
        s.m[x] = mn;
        float sum = 0.f;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i) sum += p[t][2 * x + i] = exp2f(sc[t][2 * x + i] - off);
        s.l[x] = s.l[x] * f[x] + sum;
    }
    if (__any_sync(kFull, f[0] != 1.f || f[1] != 1.f))
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                s.o[j][e][0] *= f[0];
                s.o[j][e][1] *= f[0];
                s.o[j][e][2] *= f[1];
                s.o[j][e][3] *= f[1];
            }
    uint32_t hi[4], lo[4];
    split_pair<false>(p[0][0], p[0][1], hi[0], lo[0]);
    split_pair<false>(p[0][2], p[0][3], hi[1], lo[1]);
    split_pair<false>(p[1][0], p[1][1], hi[2], lo[2]);
    split_pair<false>(p[1][2], p[1][3], hi[3], lo[3]);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const uint32_t* r0 = &vv[0][j].x;
        const uint32_t* r1 = &vv[1][j].x;
        const uint32_t* r2 = &vv[2][j].x;
        const uint32_t* r3 = &vv[3][j].x;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t pick = e & 1 ? 0x7632u : 0x5410u;
            const uint32_t b0 = __byte_perm(r0[e >> 1], r1[e >> 1], pick), b1 = __byte_perm(r2[e >> 1], r3[e >> 1], pick);
            mma_bf16(s.o[j][e], hi[0], hi[1], hi[2], hi[3], b0, b1);
            mma_bf16(s.o[j][e], lo[0], lo[1], lo[2], lo[3], b0, b1);
        }
    }
}

// Warps that share a group of 16 rows (WARPS > 1: a CTA), or 4 groups to a CTA.
template <int WARPS>
constexpr int tree_join_threads() { return WARPS == 1 ? 128 : 32 * WARPS; }
template <int WARPS>
constexpr size_t tree_join_smem() { return WARPS == 1 ? 0 : (size_t)WARPS * (16 * 32 * sizeof(float4) + kJoinRows * sizeof(float4)); }

template <bool PACKED, bool Q32, int WARPS>
__global__ void __launch_bounds__(tree_join_threads<WARPS>()) tree_join_kernel(TreeArgs a) {
    if (!a.late) wait_prior_grids();   // (no kernel of this call before it, which would have waited)
    extern __shared__ __align__(16) float4 shared[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gq = lane >> 2, tq = lane & 3;
    const int R = a.drafts * a.G, groups = (R + kJoinRows - 1) / kJoinRows;
    const int64_t gw = WARPS == 1 ? (int64_t)blockIdx.x * 4 + warp : blockIdx.x, u = gw / groups;
    const int part = WARPS == 1 ? 0 : warp;
    if (u >= (int64_t)a.batch * a.n_kv) {
        wait_prior_grids();
        return;
    }
    const int row0 = (int)(gw % groups) * kJoinRows, b = (int)(u / a.n_kv), h = (int)(u % a.n_kv);
    const int L = a.lens[b], T = tree_rows(a, b);
    const bool bad = L < 0 || (int64_t)L > (int64_t)a.max_blocks * a.B || T < 0;
    if (bad && lane == 0) raise_error(a.err, KVARN_DEVERR_POSITION);
    // rows of padding are left alone; those of a bad length are all NaN
    const int rows = bad ? R : T * a.G;
    const int mine[2] = {row0 + gq, row0 + gq + 8};
    if (row0 >= rows) {
        wait_prior_grids();
        return;
    }
    JoinRows<Q32> s;
    bool wrong[2] = {bad, bad}, any[2] = {L > 0, L > 0};
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        s.m[x] = -INFINITY;
        s.l[x] = 0.f;
        const int64_t at = (((int64_t)b * a.drafts + mine[x] / a.G) * a.n_q + h * a.G + mine[x] % a.G) * kD + 8 * tq;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (Q32) {
                uint4 y0 = make_uint4(0, 0, 0, 0), y1 = y0;
                if (mine[x] < rows) {
                    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const float*>(a.q) + at + 32 * j);
                    y0 = src[0];
                    y1 = src[1];
                }
                const uint32_t y[8] = {y0.x, y0.y, y0.z, y0.w, y1.x, y1.y, y1.z, y1.w};
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    split_pair<false>(__uint_as_float(y[2 * k]), __uint_as_float(y[2 * k + 1]), s.q[0][2 * j + (k >> 1)][x + 2 * (k & 1)],
                                      s.q[Q32 ? 1 : 0][2 * j + (k >> 1)][x + 2 * (k & 1)]);
            } else {
                const uint4 y = mine[x] < rows ? *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + at + 32 * j)
                                               : make_uint4(0, 0, 0, 0);
                s.q[0][2 * j][x] = y.x;
                s.q[0][2 * j][x + 2] = y.y;
                s.q[0][2 * j + 1][x] = y.z;
                s.q[0][2 * j + 1][x + 2] = y.w;
            }
        }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) s.o[j][e][0] = s.o[j][e][1] = s.o[j][e][2] = s.o[j][e][3] = 0.f;

    // the drafts' steps, 16 tokens each; this warp's are those whose number it has
    const float scale = a.sm_scale * kLog2e;
    auto drafts = [&] {
        for (int t = 0; t < T; t += 16) {     // (T: -1 for a bad length)
            const uint32_t all = T - t >= 16 ? 0xffffu : (1u << (T - t)) - 1;
            uint32_t seen[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                seen[x] = 0;
                if (mine[x] < rows) seen[x] = a.mask[((int64_t)b * a.drafts + mine[x] / a.G) * a.words + t / 32] >> (t % 32) & all;
                any[x] = any[x] || seen[x];
            }
            if ((WARPS > 1 && t / 16 % WARPS != part) || !__any_sync(kFull, seen[0] | seen[1])) continue;
            const int64_t at = (int64_t)b * a.drafts + t;
            join_step<Q32, true>(s, a.k + at * a.k_stride + h * kD, a.v + at * a.v_stride + h * kD, a.k_stride, a.v_stride, T - t, seen, scale,
                           lane, wrong);
        }
    };
    if (!PACKED) drafts();   // (they wait for nothing; O is in their space)
    wait_prior_grids();      // the cached tokens' kernel, beside which this one may have started
    if (!bad && tree_tokens<PACKED>(a, b) > 0) {
        int first = 0, last = a.few - 1;
        const float4* row_at[2];
        int64_t slot_stride, quad_stride;
        if (a.few > 0) {
            slot_stride = (int64_t)a.G * 33;
            quad_stride = 1;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int row = min(mine[x], rows - 1);
                row_at[x] = a.partials + ((((int64_t)b * a.drafts + row / a.G) * a.n_kv + h) * a.few * a.G + row % a.G) * 33;
            }
        } else {
            // (a range outside the grid, left by a CTA that gave up, is none)
            const int2 um = __ldcg(reinterpret_cast<const int2*>(a.unit_map) + u);
            first = um.x, last = um.x >= 0 && um.y >= um.x && um.y < a.ranges ? um.y : um.x - 1;
            slot_stride = (int64_t)33 * a.rows_pad;
            quad_stride = a.rows_pad;
#pragma unroll
            for (int x = 0; x < 2; ++x) row_at[x] = tree_partial(a, u, 0, min(mine[x], a.rows_pad - 1));
        }
        const int each = !PACKED && a.extra && row0 >= kPRows ? 2 : 1;
        for (int i = part; i < (last - first + 1) * each; i += WARPS) {
            if (PACKED && a.few > 0) {   // (a split without blocks)
                const int n = L / a.B;
                if ((int64_t)(i + 1) * n / a.few == (int64_t)i * n / a.few) continue;
            }
            float4 y[2][2][4], ml[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const float4* p = row_at[x] + (first + i / each) * slot_stride + i % each * kExtraRows;
                ml[x] = __ldcg(p);
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int k = 0; k < 4; ++k) y[x][j][k] = __ldcg(p + (1 + 16 * j + 4 * tq + k) * quad_stride);
            }
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                if (mine[x] >= rows) continue;   // (not written)
                const float mn = fmaxf(s.m[x], ml[x].x);
                const float f = s.m[x] == -INFINITY ? 0.f : exp2f(s.m[x] - mn);
                // (a range without a score above -inf: its sum is 0, or NaN, which stays)
                const float w = ml[x].x == -INFINITY ? 0.f : exp2f(ml[x].x - mn);
                s.m[x] = mn;
                s.l[x] = s.l[x] * f + (tq == 0 ? ml[x].y * w : 0.f);
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float z[4] = {y[x][j][k].x, y[x][j][k].y, y[x][j][k].z, y[x][j][k].w};
#pragma unroll
                        for (int i4 = 0; i4 < 4; ++i4) {
                            float& o = s.o[j][4 * (k & 1) + i4][2 * x + (k >> 1)];
                            o = fmaf(o, f, z[i4] * w);
                        }
                    }
            }
        }
        if (PACKED && first + part <= last && !(a.flags & KVARN_FLAG_NO_ROTATION)) {
            fwht_fragment(s.o, tq);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t word = j == 0 ? (tq < 2 ? a.sb[0] : a.sb[1]) : (tq < 2 ? a.sb[2] : a.sb[3]);
                const uint32_t bits = word >> (16 * (tq & 1));
#pragma unroll
                for (int e = 0; e < 8; ++e)
#pragma unroll
                    for (int d = 0; d < 4; ++d) s.o[j][e][d] *= bits >> (8 * (d & 1) + e) & 1 ? -kInvSqrtD : kInvSqrtD;
            }
        }
    }
    if (PACKED) {
        const int tail = bad ? 0 : L % a.B;
        const uint16_t* st = a.staging + ((int64_t)b * a.n_kv + h) * 2 * a.B * kD;
        for (int t = 0; t < tail; t += 16) {
            if (WARPS > 1 && (WARPS - 1 - t / 16 % WARPS) != part) continue;   // (from the last warp on)
            const int there = tail - t;
            const uint32_t all = there >= 16 ? 0xffffu : (1u << there) - 1;
            const uint32_t seen[2] = {all, all};
            join_step<Q32, false>(s, st + t * kD, st + (a.B + t) * kD, kD, kD, there, seen, scale, lane, wrong);
        }
        drafts();
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        s.l[x] += __shfl_xor_sync(kFull, s.l[x], 1);
        s.l[x] += __shfl_xor_sync(kFull, s.l[x], 2);
    }
    if constexpr (WARPS > 1) {
        // the warps' states: rows (m, l, wrong) behind the fragments; this warp then
        // has products WARPS apart
        float4* rows_of = shared + WARPS * 16 * 32;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                shared[(warp * 16 + 8 * j + e) * 32 + lane] = make_float4(s.o[j][e][0], s.o[j][e][1], s.o[j][e][2], s.o[j][e][3]);
        if (tq == 0) {
            rows_of[warp * kJoinRows + gq] = make_float4(s.m[0], s.l[0], wrong[0] ? 1.f : 0.f, 0.f);
            rows_of[warp * kJoinRows + gq + 8] = make_float4(s.m[1], s.l[1], wrong[1] ? 1.f : 0.f, 0.f);
        }
        __syncthreads();
        float w[2][WARPS];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            float m = -INFINITY, l = 0.f;
            bool off = false;
#pragma unroll
            for (int k = 0; k < WARPS; ++k) m = fmaxf(m, rows_of[k * kJoinRows + gq + 8 * x].x);
#pragma unroll
            for (int k = 0; k < WARPS; ++k) {
                const float4 r = rows_of[k * kJoinRows + gq + 8 * x];
                w[x][k] = r.x == -INFINITY ? 0.f : exp2f(r.x - m);
                l = fmaf(r.y, w[x][k], l);
                off = off || r.z != 0.f;
            }
            s.m[x] = m;
            s.l[x] = l;
            wrong[x] = off;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if ((8 * j + e) / (16 / WARPS) != part) continue;
                float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int k = 0; k < WARPS; ++k) {
                    const float4 y = shared[(k * 16 + 8 * j + e) * 32 + lane];
                    o[0] = fmaf(y.x, w[0][k], o[0]);
                    o[1] = fmaf(y.y, w[0][k], o[1]);
                    o[2] = fmaf(y.z, w[1][k], o[2]);
                    o[3] = fmaf(y.w, w[1][k], o[3]);
                }
#pragma unroll
                for (int d = 0; d < 4; ++d) s.o[j][e][d] = o[d];
            }
    }
    constexpr int kRun = WARPS == 1 ? 8 : 16 / WARPS > 8 ? 8 : 16 / WARPS;   // channels next to one another that this warp has
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        // Maxima drop NaN: tokens without a score above -inf have scores of NaN, or all -inf
        float l = s.l[x];
        if (wrong[x] || (any[x] && s.m[x] == -INFINITY)) l = NAN;
        if (mine[x] >= rows) continue;
        const float inv = l > 0.f ? 1.f / l : l;   // (0 for nothing seen; NaN stays)
        const int64_t at = (((int64_t)b * a.drafts + mine[x] / a.G) * a.n_q + h * a.G + mine[x] % a.G) * kD + 16 * tq;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int e0 = 0; e0 < 8; e0 += kRun) {
                    if (WARPS > 1 && (8 * j + e0) / (16 / WARPS) != part) continue;
                    float z[kRun];
#pragma unroll
                    for (int e = 0; e < kRun; ++e) z[e] = s.o[j][e0 + e][2 * x + c] * inv;
                    const int64_t to = at + 64 * j + 8 * c + e0;
                    if (a.out_bf16) {
                        uint32_t y[kRun / 2];
#pragma unroll
                        for (int k = 0; k < kRun / 2; ++k) {
                            const __nv_bfloat162 p = __floats2bfloat162_rn(z[2 * k], z[2 * k + 1]);
                            y[k] = *reinterpret_cast<const uint32_t*>(&p);
                        }
                        uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + to);
                        if constexpr (kRun == 8) *reinterpret_cast<uint4*>(dst) = make_uint4(y[0], y[1], y[2], y[3]);
                        else if constexpr (kRun == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(y[0], y[1]);
                        else *dst = y[0];
                    } else {
                        float* dst = static_cast<float*>(a.out) + to;
                        if constexpr (kRun == 2) {
                            *reinterpret_cast<float2*>(dst) = make_float2(z[0], z[1]);
                        } else {
#pragma unroll
                            for (int k = 0; k < kRun; k += 4) *reinterpret_cast<float4*>(dst + k) = make_float4(z[k], z[k + 1], z[k + 2], z[k + 3]);
                        }
                    }
                }
    }
}

// As many warps to a group of rows as leave 8 an SM (which holds that many).
template <bool PACKED, int WARPS>
cudaError_t launch_tree_join_as(const TreeArgs& a, int64_t groups, cudaStream_t st) {
    const auto fn = a.q_dtype == KVARN_FP32 ? tree_join_kernel<PACKED, true, WARPS> : tree_join_kernel<PACKED, false, WARPS>;
    constexpr size_t smem = tree_join_smem<WARPS>();
    if (smem > 48 * 1024) {
        static bool ready[2][64];
        int d = 0;
        cudaError_t e = cudaGetDevice(&d);
        if (e != cudaSuccess) return e;
        if (d < 0 || d >= 64) return cudaErrorInvalidDevice;
        bool& done = ready[a.q_dtype == KVARN_FP32][d];
        if (!done) {
            e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
            if (e != cudaSuccess) return e;
            done = true;
        }
    }
    const unsigned ctas = (unsigned)(WARPS == 1 ? (groups + 3) / 4 : groups);
    return launch_pdl(fn, ctas, tree_join_threads<WARPS>(), smem, st, a);
}
template <bool PACKED>
cudaError_t launch_tree_join(const TreeArgs& a, cudaStream_t st) {
    const int64_t groups = (int64_t)a.batch * a.n_kv * ((a.drafts * a.G + kJoinRows - 1) / kJoinRows), sms = current_device_sms();
    return groups <= sms       ? launch_tree_join_as<PACKED, 8>(a, groups, st)
           : groups <= 2 * sms ? launch_tree_join_as<PACKED, 4>(a, groups, st)
           : groups <= 4 * sms ? launch_tree_join_as<PACKED, 2>(a, groups, st)
                               : launch_tree_join_as<PACKED, 1>(a, groups, st);
}

}  // namespace kvarn
