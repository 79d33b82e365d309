// mx_tcgen05.cuh -- PTX wrappers for the fifth-generation tensor cores of
// sm_100a as the grouped product uses them: tensor memory, block-scaled 8-bit
// matrix instructions, scale copies into tensor memory, and their descriptors.
#pragma once

#include "mx_device.cuh"

namespace mx {

// ------------------------------------------------------------------ descriptors
// Shared-memory matrix descriptor: start address, leading and stride byte
// offsets in units of 16 bytes, version 1, swizzle mode (0 none, 2 128-byte).
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo, uint32_t sbo, uint32_t swizzle) {
    return (uint64_t)((addr & 0x3ffffu) >> 4) | (uint64_t)(lbo >> 4) << 16 | (uint64_t)(sbo >> 4) << 32 |
           (uint64_t)1 << 46 | (uint64_t)swizzle << 61;
}

// Instruction descriptor of a block-scaled 8-bit product with E8M0 scales:
// operand types (0 e4m3, 1 e5m2), majors (1: the contraction is the outer
// dimension) and scale type; the launch adds N / 8 at bit 17 and M / 16 at bit
// 24.  The scales' byte within a 32-bit column is added by with_scale_byte.
inline uint32_t block_scaled_idesc(bool a_e5m2, bool b_e5m2, bool a_outer, bool b_outer) {
    return (uint32_t)a_e5m2 << 7 | (uint32_t)b_e5m2 << 10 | (uint32_t)a_outer << 15 | (uint32_t)b_outer << 16 | 1u << 23;
}
__device__ __forceinline__ uint32_t with_scale_byte(uint32_t idesc, uint32_t byte) {
    return idesc | byte << 4 | byte << 29;
}

// One lane of a converged warp.  The tensor core and copy instructions take
// their operands from the warp's uniform registers; under this predicate the
// compiler knows that a single lane is left, which under `lane == 0` it does not.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}

// ------------------------------------------------------------------ pairs
// kPair: two CTAs of a cluster work on one tile; the matrix instructions and
// scale copies are issued by the one of rank 0 and run in both.
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t n;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
    return n;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of this CTA's shared variable in the CTA of rank 0, or here.
template <bool kPair>
__device__ __forceinline__ uint32_t leader_addr(const void *p) {
    const uint32_t here = smem_addr(p);
    if (!kPair) return here;
    uint32_t there;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(there) : "r"(here));
    return there;
}
// Arrivals on a barrier of either CTA of the pair.  A release at cluster scope
// waits for everything the thread has in flight, which the roles that pace the
// loop cannot afford: with releases on every arrival and acquires on every wait
// the 128 x 256 loop took about 2000 clocks a stage instead of 1100.  So only
// what a thread wrote itself is released (the scale bytes); the others order
// nothing that a thread still has under way: operand bytes are counted by the
// barrier, tensor memory has been waited for, and a word that was read is in a
// register, on which the arrival depends.
__device__ __forceinline__ void mbar_arrive_at(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_release_at(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_expect_at(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

// ------------------------------------------------------------------ work
// Cancels the launch of a cluster that has not started and takes its place: 16
// bytes about it arrive in shared memory, counted on `bar`.
__device__ __forceinline__ void cancel_launch(uint4 *answer, uint64_t *bar) {
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];"
                 ::"r"(smem_addr(answer)), "r"(smem_addr(bar)) : "memory");
}
// The first CTA of the cancelled cluster, or -1 if none was left.
__device__ __forceinline__ int cancelled_block(const uint4 *answer) {
    uint32_t x, ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\t"
        "ld.shared.b128 r, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
        "selp.u32 %1, 1, 0, p;\n\t"
        "mov.u32 %0, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%0, _, _, _}, r;\n\t}"
        : "=r"(x), "=r"(ok) : "r"(smem_addr(answer)) : "memory");
    return ok ? (int)x : -1;
}
// The address of this CTA's shared variable in the CTA of the given rank.
template <bool kPair>
__device__ __forceinline__ uint32_t addr_in(const void *p, uint32_t rank) {
    const uint32_t here = smem_addr(p);
    if (!kPair) return here;
    uint32_t there;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(here), "r"(rank));
    return there;
}
// A word into another CTA's shared memory, counted on a barrier there.
__device__ __forceinline__ void store_word_at(uint32_t addr, uint32_t value, uint32_t bar) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];"
                 ::"r"(addr), "r"(value), "r"(bar) : "memory");
}

// ------------------------------------------------------------------ tensor memory
template <bool kPair>
__device__ __forceinline__ void tmem_alloc(uint32_t *where, uint32_t columns) {
    if (kPair) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_addr(where)), "r"(columns) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    } else {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_addr(where)), "r"(columns) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
}
template <bool kPair>
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t columns) {
    if (kPair) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns));
    else asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns));
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Arrive on `bar` (of both CTAs of a pair) once every matrix instruction and
// scale copy issued by this thread has completed.
template <bool kPair>
__device__ __forceinline__ void tc_commit(uint64_t *bar) {
    if (kPair)
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                     ::"r"(smem_addr(bar)), "h"((uint16_t)3) : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                     ::"r"(smem_addr(bar)) : "memory");
}

// 32 rows x 16 bytes of shared memory into 4 columns, in all four lane
// quarters (each CTA of a pair from its own shared memory into its own columns).
template <bool kPair>
__device__ __forceinline__ void tc_copy_scales(uint32_t tmem, uint64_t desc) {
    if (kPair) asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
    else asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}

template <bool kPair>
__device__ __forceinline__ void tc_mma_scaled(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t scale_a,
                                              uint32_t scale_b, bool accumulate) {
    if (kPair)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%5], [%6], p;\n\t}"
            ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate), "r"(scale_a), "r"(scale_b) : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%5], [%6], p;\n\t}"
            ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate), "r"(scale_a), "r"(scale_b) : "memory");
}

// 32 consecutive columns of this warp's 32 lanes: lane l gets row l's values.
__device__ __forceinline__ void tc_load32(uint32_t addr, uint32_t *v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
          "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
          "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(addr));
}
__device__ __forceinline__ void tc_wait_load() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// ------------------------------------------------------------------ copies
// Tiled loads into this CTA's shared memory; the bytes are signalled on `bar`,
// in a pair that of the CTA of rank 0.
template <bool kPair>
__device__ __forceinline__ void tma_load_2d_to(void *dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
    if (kPair)
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3}], [%4];"
            ::"r"(smem_addr(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar) : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3}], [%4];"
            ::"r"(smem_addr(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar) : "memory");
}
template <bool kPair>
__device__ __forceinline__ void tma_load_3d_to(void *dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar) {
    if (kPair)
        asm volatile(
            "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3, %4}], [%5];"
            ::"r"(smem_addr(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3, %4}], [%5];"
            ::"r"(smem_addr(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
}

// A box of shared memory into a tensor, parts outside it left out; tracked in
// bulk groups.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap *map, int x, int y, int z, const void *src) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];"
                 ::"l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_addr(src)) : "memory");
}

}  // namespace mx
