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
//
// The copies are HBM's: 32 sequences x 8192 bf16 tokens cut to 2048, 8 kv heads, 537 MB in
// 85 us (6.3 TB/s), 64 x 16384 2-bit tokens cut to 4096 453 MB in 70 us, with 8 16-byte
// loads a lane in flight (one: 132 and 160 us). The selection is a chain of short steps, a CTA a
// (sequence, kv head): 18 us there, 7 for 1000 tokens (with keys read again from memory in each
// pass and digits searched by one warp 42 to 68, and 27). Whole calls as graph nodes 106, 91 and 8 us.
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
    int budget, recent;    // in places
    int64_t head_bytes;    // of a kv head's K and V in a block
};

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kDigit = 2048;             // values of an 11-bit digit
constexpr int kBins = kDigit / kSelThreads;
constexpr int kSelKeys = 9728;           // keys held in shared memory (46 KB with the rest, the most without opting in; registers allow
                                         // 3 CTAs an SM of tokens, 2 of blocks)

// A weight as a key: its bits order as it does; what is not above 0 counts as 0.
__device__ __forceinline__ uint32_t weight_key(float w) { return w > 0.f ? __float_as_uint(w) : 0u; }

__device__ __forceinline__ float tidy(float w) { return w > 0.f ? w : 0.f; }
__device__ __forceinline__ float4 tidy(float4 w) { return make_float4(tidy(w.x), tidy(w.y), tidy(w.z), tidy(w.w)); }

// A sum in three floats, of falling size: hi + mid is exact but for what mid rounds off, which lo takes
// up. Together they keep about 72 bits, more than the 53 of a sum in 64 bits, in fp32 additions alone (64-bit
// ones run at 1/64 of their rate). Two floats keep 48: 1 + 2^-24 + 2^-50 lost its last term, and with it
// the rounding of the whole to 32 bits; they take as long (64 x 16384 2-bit tokens 92.0 us a call, 91.9 so; 5 x
// 1500 8.3, 9.3).
struct Sum3 {
    float hi, mid, lo;
};
// (s, e) = a + b exactly, s rounded to nearest.
__device__ __forceinline__ void two_sum(float a, float b, float& s, float& e) {
    s = __fadd_rn(a, b);
    const float y = __fsub_rn(s, a);
    e = __fadd_rn(__fsub_rn(a, __fsub_rn(s, y)), __fsub_rn(b, y));
}
__device__ __forceinline__ Sum3 sum_of(float4 w) {
    float a, b, c, d, e, f;
    two_sum(w.x, w.y, a, c);
    two_sum(w.z, w.w, b, d);
    Sum3 s;
    two_sum(a, b, s.hi, e);
    two_sum(c, d, s.mid, f);
    two_sum(s.mid, e, s.mid, s.lo);
    s.lo = __fadd_rn(s.lo, f);
    return s;
}
// (The same whichever of the two is added to the other: a two_sum's error is exact. Where weights are
// infinite hi is, and mid and lo count no more.)
__device__ __forceinline__ Sum3 sum_of(const Sum3& a, const Sum3& b) {
    Sum3 s;
    float e, f, g;
    two_sum(a.hi, b.hi, s.hi, e);
    two_sum(a.mid, b.mid, s.mid, f);
    two_sum(s.mid, e, s.mid, g);
    s.lo = __fadd_rn(__fadd_rn(a.lo, b.lo), __fadd_rn(f, g));
    return s;
}
// Rounded to 64 bits, then to 32 (past the largest float: infinity).
__device__ __forceinline__ float rounded(const Sum3& s) {
    return isinf(s.hi) ? s.hi : __double2float_rn((double)s.hi + ((double)s.mid + (double)s.lo));
}

// The key of place i0 + lane of a row of weights with n places (0 behind them). Of a
// place of 32 or 64 tokens 8 lanes add up a part each, 16 bytes a load, 4 places a warp at once.
template <int UNIT>
__device__ __forceinline__ uint32_t place_key(const float* w, uint32_t i0, uint32_t n, int lane) {
    if constexpr (UNIT == 1) return i0 + lane < n ? weight_key(w[i0 + lane]) : 0u;
    constexpr int kParts = UNIT >= 32 ? UNIT / 32 : 1, kBatch = 4;
    Sum3 mine = {0.f, 0.f, 0.f};            // of this lane's place
#pragma unroll
    for (int s0 = 0; s0 < 8; s0 += kBatch) {
        float4 v[kBatch][kParts];
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
#pragma unroll
            for (int p = 0; p < kParts; ++p) {
                const uint32_t i = i0 + 4 * (s0 + k) + (lane >> 3);
                v[k][p] = i < n ? tidy(__ldcg(reinterpret_cast<const float4*>(w + (int64_t)i * UNIT + 4 * (lane & 7) + 32 * p)))
                                : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            Sum3 sum = sum_of(v[k][0]);
#pragma unroll
            for (int p = 1; p < kParts; ++p) sum = sum_of(sum, sum_of(v[k][p]));
#pragma unroll
            for (int m = 1; m < 8; m <<= 1)
                sum = sum_of(sum, Sum3{__shfl_xor_sync(kFull, sum.hi, m), __shfl_xor_sync(kFull, sum.mid, m), __shfl_xor_sync(kFull, sum.lo, m)});
            const int from = 8 * (lane & 3);
            const Sum3 its = {__shfl_sync(kFull, sum.hi, from), __shfl_sync(kFull, sum.mid, from), __shfl_sync(kFull, sum.lo, from)};
            if (lane >> 2 == s0 + k) mine = its;
        }
    }
    return weight_key(rounded(mine));
}

template <int UNIT>
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(EvictArgs a) {
    wait_prior_grids();
    let_next_grid_start();               // the copies
    __shared__ uint32_t hist[kDigit], keys[kSelKeys];
    __shared__ int2 sums[kSelWarps];
    __shared__ int found_digit, found_above, found_count;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int i = tid; i < kDigit; i += kSelThreads) hist[i] = 0;   // (and so each pass leaves them)
    for (int64_t u = blockIdx.x; u < a.units; u += gridDim.x) {
        const int b = (int)(u / a.n_kv), h = (int)(u % a.n_kv);
        const int L = a.lens[b];
        int32_t* kept = a.kept + u * a.budget;
        const bool bad = L < 0 || (int64_t)L > (int64_t)a.max_blocks * a.B;
        const int have = bad ? 0 : L / UNIT, size = min(have, a.budget);
        if (h == 0 && tid == 0) {
            if (bad) raise_error(a.err, KVARN_DEVERR_POSITION);
            a.new_lens[b] = bad ? 0 : size * UNIT + L % UNIT;
        }
        const int fill = have > a.budget ? a.budget - a.recent : 0;   // to be chosen among the first n
        const uint32_t n = have > a.budget ? have - a.recent : 0;
        for (int i = tid; i < a.budget - fill; i += kSelThreads) {
            const int at = fill + i;
            kept[at] = at < size ? (have > a.budget ? (int)n + i : at) : -1;
        }
        if (fill == 0) continue;
        const float* w = a.weights + u * a.stride;
        __syncthreads();                  // (the unit before has read its keys)
        // T: the key of the fill-th greatest, digit by digit. Keys that shared memory does
        // not hold are made again from the weights (L2) in each pass.
        const bool held = n <= kSelKeys;
        uint32_t T = 0;
        int need = fill;                  // of the places whose upper digits are T's
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, width = pass == 2 ? 10 : 11, up = shift + width;
            if (pass == 0 || !held) {
                constexpr int kBatch = UNIT == 1 ? 8 : 1;
                for (uint32_t i0 = 32 * warp; i0 < n; i0 += kSelThreads * kBatch) {
                    uint32_t key[kBatch];
#pragma unroll
                    for (int k = 0; k < kBatch; ++k) key[k] = place_key<UNIT>(w, i0 + kSelThreads * k, n, lane);
#pragma unroll
                    for (int k = 0; k < kBatch; ++k) {
                        const uint32_t i = i0 + kSelThreads * k + lane;
                        if (i >= n) continue;
                        if (held) keys[i] = key[k];
                        if (pass == 0 || key[k] >> up == T >> up) atomicAdd(&hist[key[k] >> shift & (1u << width) - 1], 1u);
                    }
                }
            } else {
                for (uint32_t i = tid; i < n; i += kSelThreads)
                    if (keys[i] >> up == T >> up) atomicAdd(&hist[keys[i] >> shift & (1u << width) - 1], 1u);
            }
            __syncthreads();
            // the digit at which the count from the top reaches need; thread t has digits
            // kDigit - 1 - kBins t and those below
            int c[kBins], mine = 0;
#pragma unroll
            for (int k = 0; k < kBins; ++k) {
                uint32_t& bin = hist[kDigit - 1 - kBins * tid - k];
                mine += c[k] = (int)bin;
                bin = 0;
            }
            int inc = mine;
            for (int m = 1; m < 32; m <<= 1) {
                const int o = __shfl_up_sync(kFull, inc, m);
                if (lane >= m) inc += o;
            }
            if (lane == 31) sums[warp].x = inc;
            __syncthreads();
            int before = lane < kSelWarps ? sums[lane].x : 0;
            before = __reduce_add_sync(kFull, lane < warp ? before : 0);
            int above = before + inc - mine;
            if (above < need && above + mine >= need) {
#pragma unroll
                for (int k = 0; k < kBins; ++k) {
                    if (above < need && above + c[k] >= need) {
                        found_digit = kDigit - 1 - kBins * tid - k;
                        found_above = above;
                        found_count = c[k];
                    }
                    above += c[k];
                }
            }
            __syncthreads();
            T |= (uint32_t)found_digit << shift;
            need -= found_above;
            if (need == found_count) {    // all places of T's digits so far are kept: those of T and above
                --T;                      // (T > 0: some place is not kept)
                need = 0;
                break;
            }
            // (the next write of found_* and sums is two barriers away)
        }
        // what is above T, and the first `need` that equal it, in order: a warp takes
        // places next to one another, counts, and then writes
        const uint32_t run = ((n - 1) / (32 * kSelWarps) + 1) * 32, beg = min(n, warp * run), end = min(n, beg + run);
        auto key_of = [&](uint32_t i0) { return !held ? place_key<UNIT>(w, i0, end, lane) : i0 + lane < end ? keys[i0 + lane] : 0u; };
        int2 mine = make_int2(0, 0);      // (above, equal)
        for (uint32_t i0 = beg; i0 < end; i0 += 32) {
            const uint32_t key = key_of(i0);
            mine.x += i0 + lane < end && key > T;
            mine.y += i0 + lane < end && key == T;
        }
        mine.x = __reduce_add_sync(kFull, mine.x);
        mine.y = __reduce_add_sync(kFull, mine.y);
        if (lane == 0) sums[warp] = mine;
        __syncthreads();
        const int2 s = lane < warp ? sums[lane] : make_int2(0, 0);
        mine.x = __reduce_add_sync(kFull, s.x);
        mine.y = __reduce_add_sync(kFull, s.y);
        for (uint32_t i0 = beg; i0 < end; i0 += 32) {
            const uint32_t i = i0 + lane, key = key_of(i0);
            const bool above = i < end && key > T, equal = i < end && key == T;
            const uint32_t ba = __ballot_sync(kFull, above), be = __ballot_sync(kFull, equal), below = (1u << lane) - 1;
            const int x = mine.x + __popc(ba & below), y = mine.y + __popc(be & below);
            if (above || (equal && y < need)) kept[x + min(y, need)] = i;
            mine.x += __popc(ba);
            mine.y += __popc(be);
        }
    }
}

// A warp takes kRowsPerWarp tokens (a K and a V row of 256 bytes each, 16 bytes a
// lane), or one block's head, with as many loads in flight, and its weights' new columns.
constexpr int kCopyWarps = 4, kRowsPerWarp = 8;
template <bool PACKED>
__global__ void __launch_bounds__(32 * kCopyWarps) evict_copy_kernel(EvictArgs a) {
    wait_prior_grids();
    constexpr int kPlaces = PACKED ? 1 : kRowsPerWarp;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, unit = PACKED ? a.B : 1;
    const int64_t columns = (int64_t)a.new_max_blocks * a.B;
    const int64_t i0 = ((int64_t)blockIdx.x * kCopyWarps + warp) * kPlaces;
    if (i0 * unit >= columns) return;
    for (int64_t u = blockIdx.y; u < a.units; u += gridDim.y) {
        const int b = (int)(u / a.n_kv), h = (int)(u % a.n_kv);
        const int L = a.lens[b];
        const bool bad = L < 0 || (int64_t)L > (int64_t)a.max_blocks * a.B;
        const int have = bad ? 0 : L / unit, size = min(have, a.budget), tail = bad ? 0 : L % unit;
        const float* w = a.weights + u * a.stride;
        float* new_w = a.new_weights + u * a.new_stride;
        // lane x: place i0 + x (packed: i0)
        const int64_t i = i0 + (PACKED ? 0 : lane);
        int64_t src = -1, dst = 0;
        int at = -1;
        if (lane < kPlaces || PACKED) {
            if (i < size) {
                at = a.kept[u * a.budget + i];
                const int64_t from_page = a.table[(int64_t)b * a.max_blocks + (PACKED ? at : at / a.B)];
                const int64_t to_page = a.new_table[(int64_t)b * a.new_max_blocks + (PACKED ? i : i / a.B)];
                if (from_page < 0 || from_page >= a.n_pool_blocks || to_page < 0 || to_page >= a.n_pool_blocks) {
                    if (lane < kPlaces) raise_error(a.err, KVARN_DEVERR_BLOCK_ID);
                } else {
                    src = from_page * a.block_bytes + h * a.head_bytes + (PACKED ? 0 : (int64_t)(at % a.B) * kD * 2);
                    dst = to_page * a.block_bytes + h * a.head_bytes + (PACKED ? 0 : (int64_t)(i % a.B) * kD * 2);
                }
            }
        }
        if constexpr (PACKED) {
            for (int x = lane; x < a.B; x += 32) {
                const int64_t c = i * a.B + x, kept_tokens = (int64_t)size * a.B;
                float v = 0.f;
                if (at >= 0) v = w[(int64_t)at * a.B + x];
                else if (c < kept_tokens + tail) v = w[(int64_t)have * a.B + c - kept_tokens];
                new_w[c] = v;
            }
            if (src >= 0) {
                const uint4* from = reinterpret_cast<const uint4*>(a.pool + src);
                uint4* to = reinterpret_cast<uint4*>(a.pool + dst);
                const int pieces = (int)(a.head_bytes / 16);
                constexpr int kBatch = 8;
                for (int p0 = lane; p0 < pieces; p0 += 32 * kBatch) {
                    uint4 v[kBatch];
#pragma unroll
                    for (int k = 0; k < kBatch; ++k)
                        if (p0 + 32 * k < pieces) v[k] = __ldcs(from + p0 + 32 * k);
#pragma unroll
                    for (int k = 0; k < kBatch; ++k)
                        if (p0 + 32 * k < pieces) to[p0 + 32 * k] = v[k];
                }
            }
        } else {
            if (lane < kPlaces && i < columns) new_w[i] = at >= 0 ? w[at] : 0.f;
            const int64_t piece = (int64_t)(lane >> 4) * a.B * kD * 2 + 16 * (lane & 15);
            uint4 v[kPlaces];
            int64_t from[kPlaces];
#pragma unroll
            for (int k = 0; k < kPlaces; ++k) {
                from[k] = __shfl_sync(kFull, src, k);
                if (from[k] >= 0) v[k] = __ldcs(reinterpret_cast<const uint4*>(a.pool + from[k] + piece));
            }
#pragma unroll
            for (int k = 0; k < kPlaces; ++k) {
                const int64_t to = __shfl_sync(kFull, dst, k);
                if (from[k] >= 0) *reinterpret_cast<uint4*>(a.pool + to + piece) = v[k];
            }
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
    a.budget = PACKED ? budget / B : budget;
    a.recent = PACKED ? recent / B : recent;
    const cudaStream_t st = (cudaStream_t)stream;
    const unsigned units = (unsigned)(a.units < 65535 ? a.units : 65535);
    const auto select = !PACKED ? evict_select_kernel<1> : B == 32 ? evict_select_kernel<32> : evict_select_kernel<64>;
    cudaError_t e = launch_pdl(select, units, kSelThreads, 0, st, a);
    const int per = PACKED ? kCopyWarps * B : kCopyWarps * kRowsPerWarp;   // new columns of a CTA
    if (e == cudaSuccess)
        e = launch_pdl(evict_copy_kernel<PACKED>, dim3((unsigned)((new_columns + per - 1) / per), units), 32 * kCopyWarps, 0, st, a);
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
