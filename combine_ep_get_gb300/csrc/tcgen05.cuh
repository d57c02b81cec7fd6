// Inline PTX of the Blackwell tensor path: tensor-map loads, tensor memory,
// tcgen05.mma and its commits, as the experts' kernels use them.  kCtas is
// the CTA group: 1, or 2 for a pair of CTAs on one tile (ranks 0 and 1 of a
// cluster; rank 0 issues the MMAs and owns the "full" barriers).
#pragma once

#include <cuda.h>

#include "ep_internal.cuh"

namespace epg {

// The CTA's rank in its cluster, and the address of the same shared-memory
// offset in the CTA of another rank.
__device__ __forceinline__ uint32_t cluster_ctarank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t map_to_rank(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
// Arrive on a barrier given by its shared::cluster address.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// The same without ordering this thread's memory accesses before it, for a
// barrier that hands over tensor memory that has been read: a release at
// cluster scope waits for the thread's stores, 1500 cycles and more.
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ float load_cluster(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* m) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}
// The warp's index as a value the compiler knows to be the same in all lanes:
// the issuing warps run their loops converged, in uniform registers, and
// elect a lane only to issue (a loop run by one lane alone moved every
// operand of an MMA or a load through the ordinary registers).
__device__ __forceinline__ int uniform_warp() { return __shfl_sync(0xffffffffu, threadIdx.x / 32, 0); }

// A ring of kN barriers: the stage and the parity of its current use.
template <int kN>
struct Ring {
    int stage = 0;
    uint32_t parity = 0;
    __device__ __forceinline__ void next() {
        if (++stage == kN) {
            stage = 0;
            parity ^= 1;
        }
    }
};
// mbar_wait_bounded by a whole warp, one answer for all lanes.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity) ? 1 : 0) != 0;
}

// Tensor-map loads; `bar` is a shared::cluster address (rank 0's for pairs).
template <int kCtas>
__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* m, uint32_t bar, int x, int y) {
    if (kCtas == 1)
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::
                "r"(smem_addr(dst)), "l"(m), "r"(bar), "r"(x), "r"(y) : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::
                "r"(smem_addr(dst)), "l"(m), "r"(bar), "r"(x), "r"(y) : "memory");
}
template <int kCtas>
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* m, uint32_t bar, int x, int y, int z) {
    if (kCtas == 1)
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::
                "r"(smem_addr(dst)), "l"(m), "r"(bar), "r"(x), "r"(y), "r"(z) : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::
                "r"(smem_addr(dst)), "l"(m), "r"(bar), "r"(x), "r"(y), "r"(z) : "memory");
}
template <int kCtas>
__device__ __forceinline__ void tma_load_5d(void* dst, const CUtensorMap* m, uint32_t bar, int x, int y, int z, int u,
                                            int v) {
    if (kCtas == 1)
        asm volatile(
            "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::
                "r"(smem_addr(dst)), "l"(m), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(u), "r"(v) : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.5d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::
                "r"(smem_addr(dst)), "l"(m), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(u), "r"(v) : "memory");
}
// A box from shared to global memory, in the issuing thread's bulk group.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* m, const void* src, int x, int y, int z) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(m),
                 "r"(smem_addr(src)), "r"(x), "r"(y), "r"(z) : "memory");
}
// 16 bytes from global to shared memory in the thread's current group of
// copies, zeros if not `there` (the address is then not read).
__device__ __forceinline__ void copy16_async(uint32_t dst, const void* src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copies_wait() {   // until at most kLeft groups are in flight
    asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

template <int kCtas>
__device__ __forceinline__ void tmem_alloc(uint32_t* dst, uint32_t columns) {
    if (kCtas == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(dst)),
                     "r"(columns) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(dst)),
                     "r"(columns) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
}
template <int kCtas>
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t columns) {
    if (kCtas == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns));
    else
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns));
}
__device__ __forceinline__ void tcgen05_before_sync() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tcgen05_after_sync() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// D[tmem] (+)= A B for 16-bit operands (f16 kind) or 8-bit ones.
template <int kCtas, bool kFp8>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    const uint32_t acc = accumulate ? 1u : 0u;
#define EP_MMA(group, kind)                                                                                  \
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"                                           \
                 "tcgen05.mma.cta_group::" group ".kind::" kind " [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), \
                 "l"(b), "r"(idesc), "r"(acc)                                                                  \
                 : "memory")
    if (kCtas == 1 && !kFp8) EP_MMA("1", "f16");
    if (kCtas == 2 && !kFp8) EP_MMA("2", "f16");
    if (kCtas == 1 && kFp8) EP_MMA("1", "f8f6f4");
    if (kCtas == 2 && kFp8) EP_MMA("2", "f8f6f4");
#undef EP_MMA
}
// The MMAs issued so far arrive on `bar` (in both CTAs of a pair) when done.
template <int kCtas>
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
    if (kCtas == 1)
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                         smem_addr(bar)) : "memory");
    else
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                smem_addr(bar)), "h"(static_cast<uint16_t>(3)) : "memory");
}

// Shared-memory operand descriptor, 128-byte swizzle.  K-major: rows of 128
// bytes, 8-row groups 1024 bytes apart (stride offset; the leading offset is
// not used).  MN-major: 64 elements of MN a 128-byte row, 8-row groups of K
// 1024 bytes apart, the next 64 of MN `lead` bytes on.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, uint32_t lead) {
    return static_cast<uint64_t>((addr >> 4) & 0x3fff) | (static_cast<uint64_t>(lead >> 4) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
// The same descriptor `bytes` (a multiple of 16) further on.
__device__ __forceinline__ uint64_t desc_at(uint64_t desc, uint32_t bytes) { return desc + (bytes >> 4); }
// Instruction descriptor: fp32 accumulation, bf16 (or E4M3) operands.
__device__ __forceinline__ uint32_t instr_desc(bool fp8, bool a_mn, bool b_mn, int m, int n) {
    const uint32_t type = fp8 ? 0u : 1u;
    return (1u << 4) | (type << 7) | (type << 10) | (static_cast<uint32_t>(a_mn) << 15) |
           (static_cast<uint32_t>(b_mn) << 16) | (static_cast<uint32_t>(n >> 3) << 17) |
           (static_cast<uint32_t>(m >> 4) << 24);
}

// 32 lanes x 32 columns of fp32: lane l of the warp gets its 32 columns.
__device__ __forceinline__ void tmem_load32(uint32_t addr, float (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
          "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
          "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
          "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(addr)
        : "memory");
}
// The same for 16 columns.
__device__ __forceinline__ void tmem_load16(uint32_t addr, float (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];\n\ttcgen05.wait::ld.sync.aligned;"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
          "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
        : "r"(addr)
        : "memory");
}

// Host: a tensor map of 16- or 8-bit elements, 128-byte swizzle, zero fill.
// dims and box from the innermost on; strides in bytes from the second.
bool encode_map(CUtensorMap* map, bool fp8, int rank, const void* base, const uint64_t* dims, const uint64_t* strides,
                const uint32_t* box);

}  // namespace epg
