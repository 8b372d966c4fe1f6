// rope.cuh -- RMS norm and rotary position rotation of one head's 128
// channels held by a warp (lane l: channels 4l .. 4l + 3, fp32).
//
// The rotation turns channel pair i by the angle position * inv_freq[i]. In
// 32 bits that product loses the angle of far positions (a position of 10^6
// leaves an error of 0.06 rad), so a rate is kept as the fraction of a turn
// per position in units of 2^-64: an integer product then wraps at whole
// turns by itself and its top 32 bits are the angle to 2^-32 of a turn,
// whatever the position. The error of the angle is |position| * 2^-54 turns
// from the rate's own rounding plus 2^-25 turns from the conversion to fp32
// (at half a turn; relative below), below sincospif's own.
#pragma once
#include "common.cuh"

namespace kvarn {

// This lane's share of a head at one position. HALF layout: channels c and
// c + rotary_dim / 2 are pair c, and the partner of a lane's four channels
// are the four of one other lane (rotary_dim is a multiple of 16).
// INTERLEAVED: channels 2i and 2i + 1 are pair i, both in this lane.
struct RopeLane {
    float c[4], s[4];   // cos and +-sin for this lane's channels (the sign of the partner's share in s)
    int partner;        // lane that holds the partner channels (HALF)
    bool interleaved;
};

__device__ __forceinline__ void turn_cossin(uint64_t rate, int64_t pos, float scale, float& c, float& s) {
    const uint64_t phase = rate * (uint64_t)pos;                        // turns mod 1, in 2^-64
    const float half_turns = (float)(int32_t)(uint32_t)(phase >> 32) * 0x1p-31f;   // [-1, 1]
    sincospif(half_turns, &s, &c);
    c *= scale;
    s *= scale;
}

__device__ __forceinline__ RopeLane rope_lane(const kvarn_rope& r, int64_t pos, int lane) {
    RopeLane p;
    p.interleaved = r.layout == KVARN_ROPE_INTERLEAVED;
    p.partner = lane;
#pragma unroll
    for (int k = 0; k < 4; ++k) { p.c[k] = 1.f; p.s[k] = 0.f; }
    if (4 * lane >= r.rotary_dim) return p;
    if (p.interleaved) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float c, s;
            turn_cossin(r.turns[2 * lane + k], pos, r.scale, c, s);
            p.c[2 * k] = p.c[2 * k + 1] = c;
            p.s[2 * k] = -s;
            p.s[2 * k + 1] = s;
        }
    } else {
        const int half = r.rotary_dim / 8;   // lanes of the first half
        const bool second = lane >= half;
        p.partner = second ? lane - half : lane + half;
        const int i0 = 4 * (second ? lane - half : lane);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float c, s;
            turn_cossin(r.turns[i0 + k], pos, r.scale, c, s);
            p.c[k] = c;
            p.s[k] = second ? s : -s;
        }
    }
    return p;
}

// x' = x cos + partner (+-sin); the whole warp calls it.
__device__ __forceinline__ void rope_apply(const RopeLane& p, float (&x)[4]) {
    float o[4];
    if (p.interleaved) {
        o[0] = x[1]; o[1] = x[0]; o[2] = x[3]; o[3] = x[2];
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] = __shfl_sync(kFull, x[k], p.partner);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = fmaf(x[k], p.c[k], __fmul_rn(o[k], p.s[k]));
}

// x' = x w / sqrt(mean(x^2) + eps) over the head; the whole warp calls it.
__device__ __forceinline__ void head_norm(float (&x)[4], const float (&w)[4], float eps) {
    const float ss = warp_sum(fmaf(x[0], x[0], fmaf(x[1], x[1], fmaf(x[2], x[2], __fmul_rn(x[3], x[3])))));
    const float r = rsqrtf(fmaf(ss, 1.0f / kD, eps));
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = __fmul_rn(x[k], __fmul_rn(r, w[k]));
}

// Four bf16 values of a row as floats, and four floats rounded to bf16.
__device__ __forceinline__ void unpack_bf4(uint2 u, float (&v)[4]) {
    v[0] = __uint_as_float(u.x << 16);
    v[1] = __uint_as_float(u.x & 0xffff0000u);
    v[2] = __uint_as_float(u.y << 16);
    v[3] = __uint_as_float(u.y & 0xffff0000u);
}
__device__ __forceinline__ uint2 pack_bf4(const float (&v)[4]) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

}  // namespace kvarn
