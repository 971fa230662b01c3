// spw_tcgen05.cuh -- what the tensor-core kernels (spmm.cu, gemm.cu) share: descriptors,
// tcgen05 and TMA instructions as inline PTX (no TMA multicast anywhere), the SM-pair
// helpers, and the waits that give up when another warp has flagged an abort.
#pragma once

#include <cuda.h>

#include "spw_internal.cuh"

namespace spw {

// Tensor map of a row-major fp16 matrix (rows x cols at ld_bytes, a multiple of 16) for
// boxes of box_rows x box_cols, with the 128-byte swizzle or none; elements outside it read as 0.
int encode_map_f16(CUtensorMap* map, const void* p, uint64_t cols, uint64_t rows, uint64_t ld_bytes,
                   uint32_t box_cols, uint32_t box_rows, bool swizzle = true);

// ------------------------------------------------------------------ tcgen05 helpers
__device__ inline uint64_t umma_desc_sw128(uint32_t saddr) {
    // K-major, 128-byte swizzle: 8-row atoms of 1024 bytes (stride byte offset 1024),
    // leading byte offset 16 (unused for swizzled K-major), version 1, layout type 2.
    uint64_t d = 0;
    d |= (uint64_t)((saddr >> 4) & 0x3FFF);
    d |= (uint64_t)(16 >> 4) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

// kind::f16 instruction descriptor: fp32 accumulator, fp16 A and B, both K-major.
// K-major, 64-byte swizzle: 8-row atoms of 512 bytes (the 2:4 values, 64 bytes per row).
__device__ inline uint64_t umma_desc_sw64(uint32_t saddr) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr >> 4) & 0x3FFF);
    d |= (uint64_t)(16 >> 4) << 16;
    d |= (uint64_t)(512 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)4 << 61;
    return d;
}

// Sparse MMA (2:4 A): A holds two of every four K positions (16 halves per row for K =
// 32), the metadata selecting them sits in tensor memory at e_tmem (an even column;
// idesc bits 0-1 pick the column pair's half), idesc bit 2 marks the MMA sparse.
__device__ inline void umma_f16_sp(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                   uint32_t e_tmem, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.sp.cta_group::1.kind::f16 [%0], %1, %2, [%5], %3, {%6, %6, %6, %6}, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(e_tmem), "r"(0u)
        : "memory");
}

// Shared -> tensor memory copy of a 128-row x 16-byte matrix (row r to lane r, four
// 32-bit columns), issued by the MMA thread: it runs in order with that thread's later
// tcgen05.mma, so the MMAs that read the columns need no other synchronisation.  The
// source is one K-major, unswizzled matrix: 8-row core matrices of 128 contiguous bytes.
__device__ inline void tmem_cp_128x128b(uint32_t taddr, uint32_t saddr) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr >> 4) & 0x3FFF);
    d |= (uint64_t)(128 >> 4) << 16;  // between core matrices along K (one here)
    d |= (uint64_t)(128 >> 4) << 32;  // between 8-row core matrices
    d |= (uint64_t)1 << 46;           // descriptor version; layout type 0: no swizzle
    asm volatile("tcgen05.cp.cta_group::1.128x128b [%0], %1;" ::"r"(taddr), "l"(d) : "memory");
}

// No swizzle: core matrices of 8 rows x 16 bytes, 128 contiguous bytes each; lbo and sbo are
// the strides between them along K and along M or N (K-major), or the other way round
// (MN-major: a core matrix is then 8 K rows of 8 M or N elements).
__device__ inline uint64_t umma_desc_plain(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr >> 4) & 0x3FFF);
    d |= (uint64_t)(lbo >> 4) << 16;
    d |= (uint64_t)(sbo >> 4) << 32;
    d |= (uint64_t)1 << 46;
    return d;
}

__host__ __device__ constexpr uint32_t idesc_f16(int M, int N) {
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ inline void umma_f16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ inline void umma_commit(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
        : "memory");
}

__device__ inline void tc_fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ inline void tc_fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}

// True in one lane of a converged warp.  Code that issues tcgen05 instructions runs with all
// lanes and elects the issuer around them: the operands then stay in uniform registers (one
// lane running the whole loop behind a lane test cost about 250 cycles an MMA).
__device__ inline bool elect_one() {
    uint32_t e;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(e)::"memory");
    return e != 0;
}

// ---- SM-pair (cta_group::2) helpers: a cluster of two CTAs computes one 256-row tile;
// CTA rank 0 issues the MMAs for both.
__device__ inline uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// Address of the same shared-memory location in CTA `rank` of the cluster.
__device__ inline uint32_t map_to_rank(uint32_t saddr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
    return r;
}

// Every thread of both CTAs (no thread may leave early): orders everything before it in
// either CTA before everything after it in both.
__device__ inline void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ inline void mbar_arrive_cluster(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// Waits with cluster-scope acquire (for arrivals made by the other CTA of the pair).
__device__ inline bool mbar_try_wait_cluster(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
}
__device__ inline bool mbar_test_wait_cluster(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
}

__device__ inline void umma_f16_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                     uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Arrive on the barrier at this shared-memory address (this CTA's, or the other CTA's
// through its cluster address) once the MMAs issued so far have completed.
__device__ inline void umma_commit_pair_local(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
                 : "memory");
}
// The same barrier in both CTAs of the pair (issued by rank 0): two commits, one to each
// CTA's copy of the barrier, both completing with the same MMAs.
__device__ inline void umma_commit_pair_both(uint32_t bar) {
    umma_commit_pair_local(bar);
    umma_commit_pair_local(map_to_rank(bar, 1u));
}

__device__ inline void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
          "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
          "=r"(r[31])
        : "r"(taddr)
        : "memory");
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

__device__ inline void tma_load_2d(uint32_t dst, const CUtensorMap* map, int c0, int c1,
                                   uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"((uint64_t)map), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}

// Bounded wait that also gives up when another warp has flagged an abort.
// A limit shorter than the default polls with the non-blocking test (see mbar_wait).
__device__ inline bool wait_or_abort(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                     long long limit) {
    const bool blocking = limit >= kWaitLimitCycles;
    if (blocking && mbar_try_wait(bar, parity)) return true;
    const long long start = clock64();
    while (!(blocking ? mbar_try_wait(bar, parity) : mbar_test_wait(bar, parity))) {
        if (*abort_flag) return false;
        if (clock64() - start > limit) return false;
    }
    return true;
}

// The same for a barrier the other CTA of a pair arrives on (cluster-scope acquire).
__device__ inline bool wait_or_abort_cluster(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                             long long limit) {
    const bool blocking = limit >= kWaitLimitCycles;
    if (blocking && mbar_try_wait_cluster(bar, parity)) return true;
    const long long start = clock64();
    while (!(blocking ? mbar_try_wait_cluster(bar, parity) : mbar_test_wait_cluster(bar, parity))) {
        if (*abort_flag) return false;
        if (clock64() - start > limit) return false;
    }
    return true;
}

__device__ inline void flag_abort(volatile int* abort_flag, int* status) {
    *abort_flag = 1;
    raise_status(status, SPW_ERR_TIMEOUT);
}

}  // namespace spw
