// tensor.cuh -- the sm_103a tensor-core and tensor-copy instructions that
// attend.cu is built from: tensor memory, tcgen05.mma with its descriptors,
// tiled TMA loads, and mbarrier waits that end.
#pragma once

#include <cuda.h>

#include "bulk.cuh"
#include "dspark_common.cuh"
#include "pairs.cuh"

namespace dspark {

// ------------------------------------------------------------- mbarriers

constexpr int kLooks = 1 << 18;  // a second: far beyond any pass

// Wait for a phase of an mbarrier, for warps that wait on one another inside a
// block: a look suspends the thread until the phase is over, or for some
// microseconds.  Gives up (false) after kLooks looks, or once another warp of the
// block has (*abort); whoever gives up first reports the timeout.  Kept to a few
// instructions: the wait stands in the kernel some thirty times, and all that its
// warps run in turn has to fit in the instruction cache.
__device__ __forceinline__ bool role_wait(uint32_t bar, uint32_t parity, volatile int *abort,
                                          int32_t *status) {
#pragma unroll 1
    for (int left = kLooks;;) {
        uint32_t done;
        asm volatile(
            "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
            " selp.u32 %0, 1, 0, p;\n}\n"
            : "=r"(done)
            : "r"(bar), "r"(parity)
            : "memory");
        if (done) return true;
        if (*abort) return false;
        if (--left) continue;
        *abort = 1;
        flag(status, DSPARK_STATUS_TIMEOUT);
        return false;
    }
}

// The same for a whole warp that has come this far (`ok`), with one answer for all its
// lanes: what follows a wait are instructions that the warp executes as a whole
// (tensor memory, shuffles, barriers), so no lane may go on where another gives up.
// Every role of attend.cu waits through this.
__device__ __forceinline__ bool warp_wait(bool ok, uint32_t bar, uint32_t parity, volatile int *abort,
                                          int32_t *status) {
    return __all_sync(0xFFFFFFFFu, ok && role_wait(bar, parity & 1, abort, status));
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void fence_mbar_init() {
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}
// Orders this thread's ordinary shared-memory accesses before later accesses of
// the copy and matrix engines (and theirs, observed by a barrier, before its own).
__device__ __forceinline__ void fence_async_proxy() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void named_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// The same, and whether `ok` holds for all of the threads.
__device__ __forceinline__ bool named_all(int id, int threads, bool ok) {
    uint32_t all;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n"
        " barrier.cta.red.and.pred q, %2, %3, p;\n selp.u32 %0, 1, 0, q;\n}\n"
        : "=r"(all)
        : "r"((uint32_t)ok), "r"(id), "r"(threads)
        : "memory");
    return all != 0;
}

// One box of a 4-D tensor map into shared memory, completing on `bar`.  The
// innermost coordinate is always a multiple of 16 bytes; a box outside the
// tensor arrives as zeros.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, int c0, int c1,
                                            int c2, int c3, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
        : "memory");
}

// Fetch a tensor map ahead of its first use.
__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// ---------------------------------------------------------- tensor memory

__device__ __forceinline__ void tmem_alloc(uint32_t smem_slot, int cols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_slot),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, int cols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols)
                 : "memory");
}
// Ends the warp's loads so far; takes the registers that one of them filled,
// so that no use of them moves ahead of it.
__device__ __forceinline__ void tmem_wait_load(uint32_t *r) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]),
                   "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]),
                   "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]),
                   "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                   "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                   "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]),
                   "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                   "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_store() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tmem_fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// 32 columns of the warp's 32 lanes: register i of a thread is column i of its
// lane.  `addr` carries the warp's lane base in its upper half.
__device__ __forceinline__ void tmem_load32(uint32_t addr, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
}


// The tile of 16 lanes x 64 columns as a product's fragments: of every 8 columns j a
// thread holds columns 8j + 2 (lane % 4) and the next of rows lane / 4 (r[4j],
// r[4j + 1]) and lane / 4 + 8 (r[4j + 2], r[4j + 3]).
__device__ __forceinline__ void tmem_load_rows16(uint32_t addr, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        :
          "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
          "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
          "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
          "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
          "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
}
__device__ __forceinline__ void tmem_store_rows16(uint32_t addr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x256b.x8.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
        "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]),
        "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
        "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]),
        "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
// 16 lanes x 32 columns, of every 4 columns j column 4j + lane % 4 of rows lane / 4
// (r[2j]) and lane / 4 + 8 (r[2j + 1]): pairs of 16-bit values that lie as the 32-bit
// ones above.
__device__ __forceinline__ void tmem_store_pairs16(uint32_t addr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
        "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]),
        "r"(r[14]), "r"(r[15])
        : "memory");
}

// --------------------------------------------------------- tcgen05.mma

// Shared-memory operand in rows of 128 or 64 bytes under the swizzle of that width:
// the 16-byte chunk c of row r at chunk c ^ (r & 7), or c ^ (r / 2 & 3), groups of
// eight rows one after another.  Rows are the M or N index with consecutive k a row
// (K-major; `lead` unused), or the k index with consecutive n a row (N-major; the
// next row's worth of n lies `lead` bytes on).
__device__ __forceinline__ uint64_t smem_operand(uint32_t addr, uint32_t lead, int row_bytes) {
    return (uint64_t)((addr & 0x3FFFF) >> 4) | (uint64_t)((lead >> 4) & 0x3FFF) << 16 |
           (uint64_t)(8 * row_bytes >> 4) << 32 | (uint64_t)1 << 46 |
           (uint64_t)(row_bytes == 128 ? 2 : 4) << 61;
}

// Instruction word of a 16-bit product with 32-bit accumulators, M = 128:
// `bf16` operands or half, B stored N-major or K-major.
constexpr uint32_t mma_word(bool bf16, int n, bool b_n_major) {
    return 1u << 4 | (bf16 ? 1u << 7 | 1u << 10 : 0u) | (b_n_major ? 1u << 16 : 0u) |
           (uint32_t)(n >> 3) << 17 | (uint32_t)(128 >> 4) << 24;
}

// What to take off an instruction word for M = 64: rows 16 w .. 16 w + 15 then lie in
// lanes 32 w .. 32 w + 15 of tensor memory, of the product and of a left operand there.
constexpr uint32_t kHalfRows = (uint32_t)(64 >> 4) << 24;

// The same for E4M3 operands, both K-major.
constexpr uint32_t mma_word_e4m3(int n) {
    return 1u << 4 | (uint32_t)(n >> 3) << 17 | (uint32_t)(128 >> 4) << 24;
}

// D += A B (D = A B when !accumulate), one K step of 16, A in shared memory.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t word,
                                       bool accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(word), "r"((uint32_t)accumulate)
        : "memory");
}
// The same for E4M3 operands, one K step of 32.
__device__ __forceinline__ void mma_ss_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t word,
                                            bool accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(word), "r"((uint32_t)accumulate)
        : "memory");
}
// The 16-bit product with A in tensor memory (two 16-bit k a column).
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t word,
                                       bool accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(word), "r"((uint32_t)accumulate)
        : "memory");
}
// Arrive on `bar` once every product issued so far by this thread is done.
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
        : "memory");
}

__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}\n"
                 : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

}  // namespace dspark
