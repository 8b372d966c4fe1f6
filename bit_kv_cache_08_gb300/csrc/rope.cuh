// rope.cuh -- RMS norm and rotary position rotation of one head's 128
// channels held by half a warp, 8 channels a lane in fp32. A lane's two
// groups of 4 channels are chosen so that both channels of a pair are its
// own, whatever the layout and the part of the head that is rotated: no
// shuffle but the norm's, and two rows an instruction (with a row per warp and
// partners fetched by shuffles, the 32 760-token append took 216 us, now 128).
//
// The rotation turns channel pair i by the angle position * inv_freq[i]. In
// 32 bits that product loses the angle of far positions (a position of 10^6
// leaves an error of 0.06 rad), so a rate is kept as the fraction of a turn
// per position in units of 2^-64: an integer product then wraps at whole
// turns by itself and its top 32 bits are the angle to 2^-32 of a turn,
// whatever the position. The rate is exact to half a unit whatever its size, so
// the error of the angle is |position| * 2^-65 turns (2^-34 at the ends of 32
// bits), 2^-32 from the cut, and 2^-25 from the conversion to fp32 (at half a
// turn; relative below), which is below sincospif's own.
#pragma once
#include "common.cuh"

namespace kvarn {

// Half-lane l's (0..15) channels at one position: groups c0 .. c0 + 3 and
// c1 .. c1 + 3. HALF layout: channels c and c + rotary_dim / 2 are a pair, so
// lanes below rotary_dim / 8 take 4l and rotary_dim / 2 + 4l; the 128 -
// rotary_dim channels that pass are 8 for each lane that is left
// (rotary_dim is a multiple of 16). INTERLEAVED: 8l and 8l + 4.
struct RopeLane {
    float c[4], s[4];   // of the lane's 4 pairs
    int c0, c1;
    bool interleaved;
};

__device__ __forceinline__ void turn_cossin(uint64_t rate, int64_t pos, float scale, float& c, float& s) {
    const uint64_t phase = rate * (uint64_t)pos;                        // turns mod 1, in 2^-64
    const float half_turns = (float)(int32_t)(uint32_t)(phase >> 32) * 0x1p-31f;   // [-1, 1]
    sincospif(half_turns, &s, &c);
    c *= scale;
    s *= scale;
}

// turns: r.turns in shared memory (indexed as a kernel parameter, the lanes'
// rates would come from the constant bank one after the other, for each row).
__device__ __forceinline__ void copy_turns(const kvarn_rope& r, uint64_t* turns) {
    if (threadIdx.x < 64) turns[threadIdx.x] = r.turns[threadIdx.x];
}
__device__ __forceinline__ RopeLane rope_lane(const kvarn_rope& r, const uint64_t* turns, int64_t pos, int l) {
    RopeLane p;
    p.interleaved = r.layout == KVARN_ROPE_INTERLEAVED;
    const int turned = r.rotary_dim / 8;   // lanes whose channels are rotated
    if (p.interleaved) {
        p.c0 = 8 * l;
        p.c1 = 8 * l + 4;
    } else {
        p.c0 = l < turned ? 4 * l : 8 * l;
        p.c1 = l < turned ? r.rotary_dim / 2 + 4 * l : 8 * l + 4;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) { p.c[k] = 1.f; p.s[k] = 0.f; }
    if (l < turned) {
#pragma unroll
        for (int k = 0; k < 4; ++k) turn_cossin(turns[4 * l + k], pos, r.scale, p.c[k], p.s[k]);
    }
    return p;
}

// A row's 8 values of this lane: x[0..3] from channel c0, x[4..7] from c1.
__device__ __forceinline__ void load_row(const uint16_t* row, const RopeLane& p, uint2 (&u)[2]) {
    u[0] = *reinterpret_cast<const uint2*>(row + p.c0);
    u[1] = *reinterpret_cast<const uint2*>(row + p.c1);
}

// (a, b) -> (a cos - b sin, b cos + a sin) for the lane's 4 pairs
__device__ __forceinline__ void rope_apply(const RopeLane& p, float (&x)[8]) {
    if (p.interleaved) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float a = x[2 * k], b = x[2 * k + 1];
            x[2 * k] = fmaf(a, p.c[k], __fmul_rn(b, -p.s[k]));
            x[2 * k + 1] = fmaf(b, p.c[k], __fmul_rn(a, p.s[k]));
        }
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float a = x[k], b = x[k + 4];
            x[k] = fmaf(a, p.c[k], __fmul_rn(b, -p.s[k]));
            x[k + 4] = fmaf(b, p.c[k], __fmul_rn(a, p.s[k]));
        }
    }
}

// x' = x w / sqrt(mean(x^2) + eps) over the head; the whole warp calls it, a
// row per half.
__device__ __forceinline__ void head_norm(float (&x)[8], const float (&w)[8], float eps) {
    float ss = __fmul_rn(x[0], x[0]);
#pragma unroll
    for (int k = 1; k < 8; ++k) ss = fmaf(x[k], x[k], ss);
#pragma unroll
    for (int m = 8; m >= 1; m >>= 1) ss += __shfl_xor_sync(kFull, ss, m);
    const float r = rsqrtf(fmaf(ss, 1.0f / kD, eps));
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = __fmul_rn(x[k], __fmul_rn(r, w[k]));
}

// Four bf16 values as floats, and four floats rounded to bf16.
__device__ __forceinline__ void unpack_bf4(uint2 u, float* v) {
    v[0] = __uint_as_float(u.x << 16);
    v[1] = __uint_as_float(u.x & 0xffff0000u);
    v[2] = __uint_as_float(u.y << 16);
    v[3] = __uint_as_float(u.y & 0xffff0000u);
}
__device__ __forceinline__ uint2 pack_bf4(const float* v) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

}  // namespace kvarn
