// tcgen05.cuh -- the fifth-generation tensor core and tile-copy instructions
// the shared-prefix kernels use, as thin inline PTX (sm_103a).
#pragma once
#include "common.cuh"

namespace kvarn {

// ---------------------------------------------------------------- tensor memory
// One warp allocates and frees; the base address comes back through shared memory.
__device__ __forceinline__ void tmem_alloc(uint32_t* slot, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(slot)), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t base, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols));
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 columns of this warp's 32 lanes: thread's lane, r[i] = column i. A warp
// reaches lanes 32 (warp % 4) .. + 31, given in the address's upper half.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, "
        "[%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
        ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]),
        "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]),
        "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

// 16 columns, the same way.
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// ---------------------------------------------------------------- matrix products
// 128-byte-swizzled shared-memory operand: 16-byte units of a 128-byte row
// are XORed with the row's index mod 8, 8 rows to a 1024-byte atom.
//   K-major (contraction along the row): sbo = bytes from 8 rows to the next 8
//   MN-major (contraction across rows):  sbo the same, lbo = bytes from one
//   64-element column block to the next
// The descriptor's low word for an address (+ bytes / 16 steps through the
// operand) and its constant high word: the thread that issues products adds
// one immediate per product, since the tensor core takes one every 32-64 cycles.
__device__ __forceinline__ uint32_t smem_operand(uint32_t addr, uint32_t lbo) {
    return ((addr >> 4) & 0x3fff) | ((lbo >> 4) & 0x3fff) << 16;
}
constexpr uint32_t kOperandHigh = (1024u >> 4) | 1u << 14 | 2u << 29;   // sbo 1024, version 1, 128-byte swizzle

enum { kMmaF16 = 0, kMmaBf16 = 1 };
// kind::f16, fp32 accumulators, M = 128; b_mn: B is MN-major
__host__ __device__ constexpr uint32_t mma_shape(int type, int n, bool b_mn) {
    return 1u << 4 | (uint32_t)type << 7 | (uint32_t)type << 10 | (b_mn ? 1u << 16 : 0u) | (uint32_t)(n / 8) << 17 |
           (128u / 16) << 24;
}

// d (+)= A B, A and B in shared memory / A in tensor memory (two 16-bit
// values of the contraction axis per column). Called by a whole warp with the
// same arguments; one lane, always the same, issues. (Called from a branch of
// one lane instead, every operand takes a trip from a lane's register to a
// uniform one: about 80-110 cycles a product, which starves the tensor core.)
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t shape, bool acc) {
    asm volatile(
        "{\n .reg .pred p, e;\n .reg .b64 da, db;\n elect.sync _|e, 0xffffffff;\n setp.ne.u32 p, %4, 0;\n mov.b64 da, {%1, %5};\n mov.b64 db, {%2, %5};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n}\n" ::"r"(d),
        "r"(a), "r"(b), "r"(shape), "r"((uint32_t)acc), "r"(kOperandHigh)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t shape, bool acc) {
    asm volatile(
        "{\n .reg .pred p, e;\n .reg .b64 db;\n elect.sync _|e, 0xffffffff;\n setp.ne.u32 p, %4, 0;\n mov.b64 db, {%2, %5};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n}\n" ::"r"(d),
        "r"(a), "r"(b), "r"(shape), "r"((uint32_t)acc), "r"(kOperandHigh)
        : "memory");
}
// Arrives on the barrier once every product issued before has completed (a
// whole warp calls it, the same lane as above issues).
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
    asm volatile(
        "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
        " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_addr(bar))
        : "memory");
}

// ---------------------------------------------------------------- barriers and copies
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Bounded wait of a whole warp for a phase, which also gives up when another
// warp of the CTA has: true for all lanes or for none. Every lane polls (a
// lane polling for the others takes longer: the branch and the shuffle cost
// more than the 32 polls), in a loop of a few instructions: these kernels'
// hot loops overflow the instruction caches, where straight-line waits cost
// several hundred cycles.
__device__ __forceinline__ bool warp_wait_or_stop(uint64_t* bar, uint32_t parity, int* stop, uint32_t limit) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p, q;\n .reg .u32 n, s;\n"
        " mov.u32 n, %4;\n"
        "POLL:\n"
        " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        " @p bra MET;\n"
        " ld.volatile.shared.u32 s, [%3];\n"
        " sub.u32 n, n, 1;\n"
        " setp.ne.u32 q, s, 0;\n"
        " setp.eq.or.u32 q, n, 0, q;\n"
        " @!q bra POLL;\n"
        "MET:\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity), "r"(smem_addr(stop)), "r"(limit)
        : "memory");
    const bool all = __all_sync(kFull, ok);
    if (!all) *reinterpret_cast<volatile int*>(stop) = 1;
    return all;
}
// One arrival for a warp, behind all its lanes' earlier work.
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// Tile copy global -> shared of a 2-D tensor map, completion counted on a
// barrier; x (elements) times the element size is a multiple of 16 bytes.
__device__ __forceinline__ void tile_g2s(void* dst, const void* map, int x, int y, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            smem_addr(dst)),
        "l"(map), "r"(x), "r"(y), "r"(smem_addr(bar))
        : "memory");
}

// Bulk copy shared -> global (16-byte aligned, a multiple of 16 bytes), and
// the wait until the copies of this thread have been written.
__device__ __forceinline__ void bulk_s2g(void* dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_addr(src)), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void bulk_store_wait() {
    asm volatile("cp.async.bulk.commit_group;\n cp.async.bulk.wait_group 0;" ::: "memory");
}

}  // namespace kvarn
