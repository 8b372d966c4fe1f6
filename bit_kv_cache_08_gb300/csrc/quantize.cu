// quantize.cu -- KVarN quantise-on-write (bulk and fused into the decode-step
// KV append) and dequantisation, hand-written for sm_103a.
//
// Method: abstract of "KVarN: cuantizacion de KV-Cache normalizada por
// varianza mitiga la acumulacion de errores en tareas de razonamiento"
// (Hadamard rotation, then dual-scaling variance normalisation over both axes
// of K and V, 2-bit) and "KVarN：方差归一化让 2-bit KV 缓存扛住长链推理"
// section 三 3.1 (randomised Hadamard) and 3.2 (token axis then channel axis
// to variance 1, repeated; grouped scales kept for dequantisation; computed
// at decode time inside the KV write kernel).
//
// One CTA of 8B threads (B/4 warps) owns one head-block of B tokens x 128
// channels. Warp w holds tokens 4w .. 4w+3, lane l channels 4l..4l+3, all in
// registers:
//   rotation   sign flip + FWHT-128 (2 in-register + 5 shuffle stages), *1/sqrt(128)
//   VarN       each pass sets a factor from the rotated tile directly: scaling a
//              row by a constant scales its spread by the same constant, so after
//              a token pass R_t = std_c(x_rot[t][c] / C_c) and after a channel
//              pass C_c = std_t(x_rot[t][c] / R_t) -- the values the pages'
//              divide-and-accumulate iteration reaches, without keeping the
//              normalised tile. Token pass: two-pass mean/variance by warp
//              reduction; channel pass: per-warp partial sums through shared memory
//   factors    sqrt(v) as v * rsqrt(v) (a few fp32 ulps; the factors only feed
//              statistics and an fp16 rounding), then fp16 round-to-nearest of
//              the clamped factors
//   quantise   y = x_rot * (1/R16) * (1/C16) (correctly rounded reciprocals;
//              a few fp32 ulps from the quotient), per (token, 32-channel group):
//              z = fp16 round-down of the
//              minimum, s = least fp16 with z + L s >= maximum, L = 2^bits - 1
//              (directed-rounding candidate plus one exact check), code = nearest
//              level, ties even (3 compares at 2 bits, a 4-step binary search
//              over the 15 boundaries at 4 bits)
//   pack       codes OR-ed into the shared-memory image of the head-block in
//              the attention kernel's record order, then 16-byte stores.
#include "quantize.cuh"

namespace kvarn {

// ---------------------------------------------------------------- bulk quantise
template <int B, int BITS>
__global__ void __launch_bounds__(quant_threads<B>(), 3) quantize_blocks_kernel(
    const void* __restrict__ src, int dtype, int64_t block_stride, int64_t token_stride,
    uint8_t* __restrict__ dst_base, const int64_t* __restrict__ dst_offsets, QuantParams p,
    uint32_t* err) {
    wait_prior_grids();
    __shared__ QuantSmem<B, BITS> q;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t n = blockIdx.x;
    zero_code_words<B, BITS>(q, tid);
    float x[kRowsPerWarp][4];
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kRowsPerWarp; ++i) {
        const int t = warp * kRowsPerWarp + i;
        load4(src, dtype, n * block_stride + (int64_t)t * token_stride + 4 * lane, x[i]);
#pragma unroll
        for (int k = 0; k < 4; ++k) bad |= !isfinite(x[i][k]);
    }
    if (__syncthreads_or(bad) && tid == 0) raise_error(err, KVARN_DEVERR_NONFINITE);
    quantize_tile<B, BITS>(x, p, q, warp, lane);
    const int64_t off = dst_offsets ? dst_offsets[n] : n * (int64_t)head_block_bytes(B, BITS);
    store_image<B, BITS>(q, dst_base + off, tid);
}

// ---------------------------------------------------------------- fused append
// grid (batch, n_kv, 2): one CTA per (sequence, kv head, K|V).
template <int B, int BITS>
__global__ void __launch_bounds__(quant_threads<B>(), 3) append_kernel(
    uint8_t* __restrict__ pool, int64_t n_pool_blocks, int64_t block_bytes,
    uint16_t* __restrict__ staging, const int32_t* __restrict__ block_table, int max_blocks,
    const int32_t* __restrict__ pos_arr, const uint16_t* __restrict__ k_new,
    const uint16_t* __restrict__ v_new, int n_kv, QuantParams p, uint32_t* err) {
    wait_prior_grids();
    __shared__ QuantSmem<B, BITS> q;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int b = blockIdx.x, h = blockIdx.y, kv = blockIdx.z;
    const int pos = pos_arr[b];
    if (pos < 0 || pos >= max_blocks * B) {
        if (tid == 0 && h == 0 && kv == 0) raise_error(err, KVARN_DEVERR_POSITION);
        return;
    }
    const int row = pos % B;
    const uint16_t* newrow = (kv ? v_new : k_new) + ((int64_t)b * n_kv + h) * kD;
    uint16_t* stage = staging + (((int64_t)b * n_kv + h) * 2 + kv) * B * kD;
    if (tid < 16)   // 256 bytes, 16 per thread
        reinterpret_cast<uint4*>(stage + row * kD)[tid] = reinterpret_cast<const uint4*>(newrow)[tid];
    if (row != B - 1) return;

    const int64_t phys = block_table[(int64_t)b * max_blocks + pos / B];
    if (phys < 0 || phys >= n_pool_blocks) {
        if (tid == 0) raise_error(err, KVARN_DEVERR_BLOCK_ID);
        return;
    }
    p.kind = kv;
    zero_code_words<B, BITS>(q, tid);
    float x[kRowsPerWarp][4];
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kRowsPerWarp; ++i) {
        const int t = warp * kRowsPerWarp + i;
        const uint16_t* r = (t == B - 1) ? newrow : stage + t * kD;
        load4(r, KVARN_BF16, 4 * lane, x[i]);
#pragma unroll
        for (int k = 0; k < 4; ++k) bad |= !isfinite(x[i][k]);
    }
    if (__syncthreads_or(bad) && tid == 0) raise_error(err, KVARN_DEVERR_NONFINITE);
    quantize_tile<B, BITS>(x, p, q, warp, lane);
    store_image<B, BITS>(q, pool + phys * block_bytes + (int64_t)(2 * h + kv) * head_block_bytes(B, BITS), tid);
}

// ---------------------------------------------------------------- dequantise
template <int B, int BITS>
__global__ void __launch_bounds__(256) dequantize_kernel(
    const uint8_t* __restrict__ src_base, const int64_t* __restrict__ src_offsets, int kind,
    int rotated, QuantParams p, float* __restrict__ out) {
    wait_prior_grids();
    __shared__ alignas(16) uint8_t img[head_block_bytes(B, BITS)];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t n = blockIdx.x;
    const int64_t off = src_offsets ? src_offsets[n] : n * (int64_t)head_block_bytes(B, BITS);
    load_image<B, BITS>(img, src_base + off, tid);
    __syncthreads();
    for (int i = 0; i < B / 8; ++i) {
        const int t = warp * (B / 8) + i;
        float v[4];
        dequant_row4<B, BITS>(img, kind, t, lane, v);
        if (!rotated && !(p.flags & KVARN_FLAG_NO_ROTATION)) {
            fwht128(v, lane);
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] *= kInvSqrtD * sign_of(p.sb, 4 * lane + k);
        }
        *reinterpret_cast<float4*>(out + (n * B + t) * kD + 4 * lane) = make_float4(v[0], v[1], v[2], v[3]);
    }
}

// ---------------------------------------------------------------- error decomposition
// Per token: (|x|, |x^|, |E_M|, |E_D|) with E_M = (|x^| - |x|) x/|x| and
// E_D = |x^| (x^/|x^| - x/|x|), x the values before quantisation and x^ the
// dequantised ones. Norms and the angle do not change under the rotation, so
// both are taken in the rotated space (x rotated like the quantiser does).
template <int B, int BITS>
__global__ void __launch_bounds__(256) error_split_kernel(
    const void* __restrict__ src, int dtype, int64_t block_stride, int64_t token_stride,
    const uint8_t* __restrict__ packed_base, const int64_t* __restrict__ packed_offsets, int kind,
    QuantParams p, float* __restrict__ out) {
    wait_prior_grids();
    __shared__ alignas(16) uint8_t img[head_block_bytes(B, BITS)];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t n = blockIdx.x;
    const int64_t off = packed_offsets ? packed_offsets[n] : n * (int64_t)head_block_bytes(B, BITS);
    load_image<B, BITS>(img, packed_base + off, tid);
    __syncthreads();
    const uint32_t sw = p.sb[lane >> 3] >> (4 * (lane & 7));
    for (int i = 0; i < B / 8; ++i) {
        const int t = warp * (B / 8) + i;
        float x[4], xh[4];
        load4(src, dtype, n * block_stride + (int64_t)t * token_stride + 4 * lane, x);
        if (!(p.flags & KVARN_FLAG_NO_ROTATION)) {
#pragma unroll
            for (int k = 0; k < 4; ++k) x[k] = ((sw >> k) & 1u) ? -x[k] : x[k];
            fwht128(x, lane);
#pragma unroll
            for (int k = 0; k < 4; ++k) x[k] *= kInvSqrtD;
        }
        dequant_row4<B, BITS>(img, kind, t, lane, xh);
        const float nx = sqrtf(warp_sum(x[0] * x[0] + x[1] * x[1] + x[2] * x[2] + x[3] * x[3]));
        const float nh = sqrtf(warp_sum(xh[0] * xh[0] + xh[1] * xh[1] + xh[2] * xh[2] + xh[3] * xh[3]));
        float em, ed = 0.f;
        if (nx == 0.f) {
            em = nh;                 // direction undefined: all of the error is magnitude
        } else {
            em = fabsf(nh - nx);
            if (nh > 0.f) {
                const float ix = 1.0f / nx, ih = 1.0f / nh;
                float d = 0.f;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float u = xh[k] * ih - x[k] * ix;
                    d = fmaf(u, u, d);
                }
                ed = nh * sqrtf(warp_sum(d));
            }
        }
        if (lane == 0) *reinterpret_cast<float4*>(out + (n * B + t) * 4) = make_float4(nx, nh, em, ed);
    }
}

// ---------------------------------------------------------------- host launchers
cudaError_t launch_quantize_blocks(const kvarn_config& cfg, int kind, const void* src, int dtype,
                                   int64_t n, int64_t block_stride, int64_t token_stride,
                                   void* dst_base, const int64_t* dst_offsets, uint32_t* err,
                                   cudaStream_t st) {
    QuantParams p = make_params(cfg, kind);
    return dispatch(cfg, [&](auto b, auto w) {
        constexpr int B = decltype(b)::value, BITS = decltype(w)::value;
        return launch_pdl(quantize_blocks_kernel<B, BITS>, (unsigned)n, quant_threads<B>(), 0, st, src, dtype,
                          block_stride, token_stride, (uint8_t*)dst_base, dst_offsets, p, err);
    });
}

cudaError_t launch_append(const kvarn_config& cfg, void* pool, int64_t n_pool_blocks,
                          int64_t block_bytes, void* staging, const int32_t* block_table,
                          int max_blocks, const int32_t* pos, const void* k_new, const void* v_new,
                          int batch, uint32_t* err, cudaStream_t st) {
    QuantParams p = make_params(cfg, 0);
    const dim3 grid(batch, cfg.n_kv_heads, 2);
    return dispatch(cfg, [&](auto b, auto w) {
        constexpr int B = decltype(b)::value, BITS = decltype(w)::value;
        return launch_pdl(append_kernel<B, BITS>, grid, quant_threads<B>(), 0, st, (uint8_t*)pool, n_pool_blocks,
                          block_bytes, (uint16_t*)staging, block_table, max_blocks, pos, (const uint16_t*)k_new,
                          (const uint16_t*)v_new, cfg.n_kv_heads, p, err);
    });
}

cudaError_t launch_error_split(const kvarn_config& cfg, int kind, const void* src, int dtype, int64_t n,
                               int64_t block_stride, int64_t token_stride, const void* packed_base,
                               const int64_t* packed_offsets, float* out, cudaStream_t st) {
    QuantParams p = make_params(cfg, kind);
    return dispatch(cfg, [&](auto b, auto w) {
        constexpr int B = decltype(b)::value, BITS = decltype(w)::value;
        return launch_pdl(error_split_kernel<B, BITS>, (unsigned)n, 256, 0, st, src, dtype, block_stride,
                          token_stride, (const uint8_t*)packed_base, packed_offsets, kind, p, out);
    });
}

cudaError_t launch_dequantize(const kvarn_config& cfg, int kind, const void* src_base,
                              const int64_t* src_offsets, int64_t n, int rotated, float* out,
                              cudaStream_t st) {
    QuantParams p = make_params(cfg, kind);
    return dispatch(cfg, [&](auto b, auto w) {
        constexpr int B = decltype(b)::value, BITS = decltype(w)::value;
        return launch_pdl(dequantize_kernel<B, BITS>, (unsigned)n, 256, 0, st, (const uint8_t*)src_base,
                          src_offsets, kind, rotated, p, out);
    });
}

}  // namespace kvarn
