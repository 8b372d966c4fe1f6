// evict.cu -- cuts the sequences of a paged cache down to a budget: per
// (sequence, kv head) the last `recent` places and, of the others, those with
// the greatest accumulated attention weights, copied in order to new pages.
// A place is a token (bf16 pages) or a block (packed cache, by the sum of its
// tokens' weights).
//
// evict_select_kernel finds what is kept: a weight that is not negative orders
// as its bits, and three passes over 11, 11 and 10 of them from the top narrow
// down the key T of the last place that still fits; places above T are kept,
// and of those equal to it the first ones. evict_copy_kernel moves them.
#include "common.cuh"
#include "host_checks.h"

namespace kvarn {

struct EvictArgs {
    uint8_t* pool;
    const int32_t *table, *lens, *new_table;
    const float* weights;
    float* new_weights;
    int32_t *new_lens, *kept;
    uint32_t* err;
    int64_t n_pool_blocks, block_bytes, stride, new_stride, units;
    int n_kv, B, max_blocks, new_max_blocks;
    int unit;              // tokens of a place: 1 or B
    int budget, recent;    // in places
    int64_t head_bytes;    // of a kv head's K and V in a block
};

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kDigit = 2048;             // values of an 11-bit digit

// A weight as a key: its bits order as it does; what is not above 0 counts as 0.
__device__ __forceinline__ uint32_t weight_key(float w) { return w > 0.f ? __float_as_uint(w) : 0u; }

// (hi, lo) += w, exactly but for the last bits of lo: hi + lo keeps about 48
// bits, so that its rounding to 32 is that of the sum in 64 bits.
__device__ __forceinline__ void add_pair(float& hi, float& lo, float w) {
    const float s = hi + w, b = s - hi;
    lo += (hi - (s - b)) + (w - b);
    hi = s;
}

__device__ __forceinline__ float tidy(float w) { return w > 0.f ? w : 0.f; }

// The key of place i of a row of weights.
__device__ __forceinline__ uint32_t place_key(const float* w, int i, int unit) {
    if (unit == 1) return weight_key(w[i]);
    float hi = 0.f, lo = 0.f;
    const float4* x = reinterpret_cast<const float4*>(w + (int64_t)i * unit);
    for (int k = 0; k < unit / 4; ++k) {
        const float4 v = x[k];
        add_pair(hi, lo, tidy(v.x));
        add_pair(hi, lo, tidy(v.y));
        add_pair(hi, lo, tidy(v.z));
        add_pair(hi, lo, tidy(v.w));
    }
    return weight_key(isinf(hi) ? hi : hi + lo);
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(EvictArgs a) {
    wait_prior_grids();
    __shared__ uint32_t hist[kDigit];
    __shared__ int2 sums[kSelWarps];
    __shared__ int found_digit, found_above;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int64_t u = blockIdx.x; u < a.units; u += gridDim.x) {
        const int b = (int)(u / a.n_kv), h = (int)(u % a.n_kv);
        const int L = a.lens[b];
        int32_t* kept = a.kept + u * a.budget;
        const bool bad = L < 0 || (int64_t)L > (int64_t)a.max_blocks * a.B;
        const int have = bad ? 0 : L / a.unit, size = min(have, a.budget);
        if (h == 0 && tid == 0) {
            if (bad) raise_error(a.err, KVARN_DEVERR_POSITION);
            a.new_lens[b] = bad ? 0 : size * a.unit + L % a.unit;
        }
        const int fill = have > a.budget ? a.budget - a.recent : 0;   // to be chosen among the first n
        const int n = have > a.budget ? have - a.recent : 0;
        for (int i = tid; i < a.budget - fill; i += kSelThreads) {
            const int at = fill + i;
            kept[at] = at < size ? (have > a.budget ? n + i : at) : -1;
        }
        if (fill == 0) continue;
        const float* w = a.weights + u * a.stride;
        // T: the key of the fill-th greatest, digit by digit
        uint32_t T = 0;
        int need = fill;                  // of the places whose upper digits are T's
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, width = pass == 2 ? 10 : 11;
            for (int i = tid; i < kDigit; i += kSelThreads) hist[i] = 0;
            __syncthreads();
            for (int i = tid; i < n; i += kSelThreads) {
                const uint32_t key = place_key(w, i, a.unit);
                const int up = shift + width;
                if (pass == 0 || key >> up == T >> up) atomicAdd(&hist[key >> shift & (1u << width) - 1], 1u);
            }
            __syncthreads();
            if (warp == 0) {              // the digit at which the count from the top reaches need
                int above = 0;
                for (int d0 = kDigit - 32; d0 >= 0; d0 -= 32) {
                    const int c = hist[d0 + 31 - lane];   // lane 0: the greatest digit
                    int inc = c;
                    for (int m = 1; m < 32; m <<= 1) {
                        const int o = __shfl_up_sync(kFull, inc, m);
                        if (lane >= m) inc += o;
                    }
                    const uint32_t hit = __ballot_sync(kFull, above + inc >= need);
                    if (hit) {
                        const int first = __ffs(hit) - 1;
                        if (lane == first) {
                            found_digit = d0 + 31 - lane;
                            found_above = above + inc - c;
                        }
                        break;
                    }
                    above += __shfl_sync(kFull, inc, 31);
                }
            }
            __syncthreads();
            T |= (uint32_t)found_digit << shift;
            need -= found_above;
            __syncthreads();
        }
        // what is above T, and the first `need` that equal it, in order
        int2 base = make_int2(0, 0);      // (above, equal) so far
        for (int i0 = 0; i0 < n; i0 += kSelThreads) {
            const int i = i0 + tid;
            const uint32_t key = i < n ? place_key(w, i, a.unit) : 0u;
            const bool above = i < n && key > T, equal = i < n && key == T;
            const uint32_t ba = __ballot_sync(kFull, above), be = __ballot_sync(kFull, equal);
            if (lane == 0) sums[warp] = make_int2(__popc(ba), __popc(be));
            __syncthreads();
            int2 mine = base;
            for (int k = 0; k < kSelWarps; ++k) {
                const int2 s = sums[k];
                if (k < warp) mine = make_int2(mine.x + s.x, mine.y + s.y);
                base = make_int2(base.x + s.x, base.y + s.y);
            }
            const uint32_t below = (1u << lane) - 1;
            mine.x += __popc(ba & below);
            mine.y += __popc(be & below);
            if (above || (equal && mine.y < need)) kept[mine.x + min(mine.y, need)] = i;
            __syncthreads();
        }
    }
}

// Places one after the other, 16 bytes a thread; then the weights of the new columns.
constexpr int kCopyThreads = 256, kCopyPlaces = 64;
__global__ void __launch_bounds__(kCopyThreads) evict_copy_kernel(EvictArgs a) {
    wait_prior_grids();
    const int tid = threadIdx.x;
    const int i0 = blockIdx.x * (kCopyPlaces / a.unit), per = kCopyPlaces / a.unit;   // places of this CTA
    for (int64_t u = blockIdx.y; u < a.units; u += gridDim.y) {
        const int b = (int)(u / a.n_kv), h = (int)(u % a.n_kv);
        const int L = a.lens[b];
        const bool bad = L < 0 || (int64_t)L > (int64_t)a.max_blocks * a.B;
        const int have = bad ? 0 : L / a.unit, size = min(have, a.budget), tail = bad ? 0 : L % a.unit;
        const int32_t* kept = a.kept + u * a.budget;
        const int32_t* table = a.table + (int64_t)b * a.max_blocks;
        const int32_t* to = a.new_table + (int64_t)b * a.new_max_blocks;
        // 16-byte pieces: of a token's K and V row (2 x 16), or of a block's head
        const int pieces = a.unit == 1 ? 32 : (int)(a.head_bytes / 16);
        for (int x = tid; x < per * pieces; x += kCopyThreads) {
            const int i = i0 + x / pieces, p = x % pieces;
            if (i >= size) break;
            const int at = kept[i];
            const int64_t from_page = table[a.unit == 1 ? at / a.B : at], to_page = to[a.unit == 1 ? i / a.B : i];
            if (from_page < 0 || from_page >= a.n_pool_blocks || to_page < 0 || to_page >= a.n_pool_blocks) {
                raise_error(a.err, KVARN_DEVERR_BLOCK_ID);
                continue;
            }
            int64_t src = from_page * a.block_bytes + h * a.head_bytes, dst = to_page * a.block_bytes + h * a.head_bytes;
            if (a.unit == 1) {
                const int64_t kind = (int64_t)(p >> 4) * a.B * kD * 2 + 16 * (p & 15);
                src += kind + (int64_t)(at % a.B) * kD * 2;
                dst += kind + (int64_t)(i % a.B) * kD * 2;
            } else {
                src += 16 * p;
                dst += 16 * p;
            }
            *reinterpret_cast<uint4*>(a.pool + dst) = *reinterpret_cast<const uint4*>(a.pool + src);
        }
        const int64_t columns = (int64_t)a.new_max_blocks * a.B;
        const int64_t c = (int64_t)blockIdx.x * kCopyPlaces + tid;
        if (tid < kCopyPlaces && c < columns) {
            const float* w = a.weights + u * a.stride;
            const int64_t kept_tokens = (int64_t)size * a.unit;
            float v = 0.f;
            if (c < kept_tokens) v = w[(int64_t)kept[c / a.unit] * a.unit + c % a.unit];
            else if (c < kept_tokens + tail) v = w[(int64_t)have * a.unit + c - kept_tokens];
            a.new_weights[u * a.new_stride + c] = v;
        }
    }
}

namespace {

template <bool PACKED>
int evict(const kvarn_config* cfg, void* pool, int64_t n_pool_blocks, const int32_t* block_table, int32_t max_blocks,
          const int32_t* seq_lens, const float* weights, int64_t weights_stride, int32_t budget, int32_t recent,
          const int32_t* new_table, int32_t new_max_blocks, int32_t* new_lens, float* new_weights,
          int64_t new_weights_stride, int32_t* kept, int32_t batch, void* workspace, void* stream) {
    kvarn_config c;
    const int r = check_config(cfg, &c);
    if (r != KVARN_OK) return r;
    const int B = c.block_size;
    if (batch < 0 || max_blocks < 0 || new_max_blocks < 0 || n_pool_blocks < 1 || n_pool_blocks > 0x7fffffff)
        return KVARN_ERR_INVALID_ARG;
    if (budget < 1 || recent < 0 || recent > budget) return KVARN_ERR_INVALID_ARG;
    if (PACKED && (budget % B || recent % B)) return KVARN_ERR_INVALID_ARG;
    const int64_t columns = (int64_t)max_blocks * B, new_columns = (int64_t)new_max_blocks * B;
    if (columns > 0x7fffffff || new_columns > 0x7fffffff || new_columns < (int64_t)budget + (PACKED ? 1 : 0))
        return KVARN_ERR_INVALID_ARG;
    if (weights_stride < columns || new_weights_stride < new_columns || weights_stride % 4) return KVARN_ERR_INVALID_ARG;
    if (batch == 0) return KVARN_OK;
    if (!pool || !seq_lens || !new_table || !new_lens || !new_weights || !kept || !workspace) return KVARN_ERR_INVALID_ARG;
    if (max_blocks > 0 && (!block_table || !weights)) return KVARN_ERR_INVALID_ARG;
    if (!aligned(pool, 16) || !aligned(weights, 16) || !aligned(workspace, 16) || !aligned(block_table, 4) ||
        !aligned(seq_lens, 4) || !aligned(new_table, 4) || !aligned(new_lens, 4) || !aligned(new_weights, 4) || !aligned(kept, 4))
        return KVARN_ERR_INVALID_ARG;
    if (new_lens == seq_lens || new_weights == weights) return KVARN_ERR_INVALID_ARG;

    EvictArgs a = {};
    a.pool = (uint8_t*)pool;
    a.table = block_table;
    a.lens = seq_lens;
    a.new_table = new_table;
    a.weights = weights;
    a.new_weights = new_weights;
    a.new_lens = new_lens;
    a.kept = kept;
    a.err = (uint32_t*)workspace;
    a.n_pool_blocks = n_pool_blocks;
    a.head_bytes = PACKED ? 2 * head_block_bytes(B, c.bits) : 2 * B * kD * 2;
    a.block_bytes = c.n_kv_heads * a.head_bytes;
    a.stride = weights_stride;
    a.new_stride = new_weights_stride;
    a.units = (int64_t)batch * c.n_kv_heads;
    a.n_kv = c.n_kv_heads;
    a.B = B;
    a.max_blocks = max_blocks;
    a.new_max_blocks = new_max_blocks;
    a.unit = PACKED ? B : 1;
    a.budget = budget / a.unit;
    a.recent = recent / a.unit;
    const cudaStream_t st = (cudaStream_t)stream;
    const unsigned units = (unsigned)(a.units < 65535 ? a.units : 65535);
    cudaError_t e = launch_pdl(evict_select_kernel, units, kSelThreads, 0, st, a);
    if (e == cudaSuccess)
        e = launch_pdl(evict_copy_kernel, dim3((unsigned)((new_columns + kCopyPlaces - 1) / kCopyPlaces), units), kCopyThreads, 0, st, a);
    return e == cudaSuccess ? KVARN_OK : KVARN_ERR_CUDA;
}

}  // namespace
}  // namespace kvarn

using namespace kvarn;

extern "C" {

int kvarn_evict(const kvarn_config* cfg, void* pool, int64_t n_pool_blocks, const int32_t* block_table,
                int32_t max_blocks_per_seq, const int32_t* seq_lens, const float* weights, int64_t weights_stride,
                int32_t budget, int32_t recent, const int32_t* new_table, int32_t new_max_blocks, int32_t* new_lens,
                float* new_weights, int64_t new_weights_stride, int32_t* kept, int32_t batch, void* workspace, void* stream) {
    return evict<true>(cfg, pool, n_pool_blocks, block_table, max_blocks_per_seq, seq_lens, weights, weights_stride, budget,
                       recent, new_table, new_max_blocks, new_lens, new_weights, new_weights_stride, kept, batch, workspace,
                       stream);
}

int kvarn_evict_bf16(const kvarn_config* cfg, void* kv_pool, int64_t n_pool_blocks, const int32_t* block_table,
                     int32_t max_blocks_per_seq, const int32_t* seq_lens, const float* weights, int64_t weights_stride,
                     int32_t budget, int32_t recent, const int32_t* new_table, int32_t new_max_blocks, int32_t* new_lens,
                     float* new_weights, int64_t new_weights_stride, int32_t* kept, int32_t batch, void* workspace,
                     void* stream) {
    return evict<false>(cfg, kv_pool, n_pool_blocks, block_table, max_blocks_per_seq, seq_lens, weights, weights_stride,
                        budget, recent, new_table, new_max_blocks, new_lens, new_weights, new_weights_stride, kept, batch,
                        workspace, stream);
}

}  // extern "C"
