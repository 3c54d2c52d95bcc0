// Fifth-generation tensor core instructions (tcgen05) and what feeds them:
// block-scaled 8-bit products (kind::mxf8f6f4), tensor memory, bulk copies and
// cluster addresses.  GROUP is the number of CTAs that work on one tile (1, 2).
#pragma once

#include <cstdint>

#include "tma.cuh"

namespace tsenor {

// ---- instruction and operand descriptors --------------------------------------------

// kind::mxf8f6f4 with e4m3 operands, fp32 accumulator and one exponent byte
// (ue8m0) per row and 32 of the contracted axis; bits 4-5 and 29-30 choose which
// of the four bytes of a scale word an instruction uses.  t: the operand is
// stored with its contracted axis along rows ("MN-major").
__host__ __device__ constexpr uint32_t mma_desc(int m, int n, bool a_t, bool b_t) {
    return (uint32_t(a_t) << 15) | (uint32_t(b_t) << 16) | (uint32_t(n / 8) << 17) | (1u << 23) |
           (uint32_t(m / 128) << 27);
}
__device__ __forceinline__ uint32_t with_scale_byte(uint32_t desc, uint32_t id) { return desc | (id << 4) | (id << 29); }

// Operand tile in shared memory: 128-byte rows in the 128-byte swizzle that TMA
// writes, 8 rows to a 1024-byte group.  sbo: bytes between groups of 8 rows;
// lbo: bytes between 128-byte wide column groups (MN-major tiles wider than 128).
__device__ __forceinline__ uint64_t tile_desc(uint32_t smem, uint32_t lbo) {
    return uint64_t((smem >> 4) & 0x3fffu) | (uint64_t(lbo >> 4) << 16) | (uint64_t(1024 >> 4) << 32) |
           (uint64_t(1) << 46) | (uint64_t(2) << 61);
}
// Scale entry of 32 rows of 16 bytes, not swizzled, 8 rows to a 128-byte group.
__device__ __forceinline__ uint64_t scale_desc(uint32_t smem) {
    return uint64_t((smem >> 4) & 0x3fffu) | (uint64_t(128 >> 4) << 32) | (uint64_t(1) << 46);
}

// ---- tensor memory ------------------------------------------------------------------

template <int GROUP>
__device__ __forceinline__ void tmem_alloc(uint32_t* slot, int cols) {     // one warp, cols a power of two >= 32
    if constexpr (GROUP == 1)
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32(slot)), "r"(cols) : "memory");
    else
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32(slot)), "r"(cols) : "memory");
}
template <int GROUP>
__device__ __forceinline__ void tmem_free(uint32_t tmem, int cols) {       // the warp that allocated
    if constexpr (GROUP == 1) {
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols));
    } else {
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols));
    }
}
__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 32 lanes (the warp's quarter of the 128) x 32 columns, one row to a thread.  Both of these are for the warp as one:
// lanes that stored by themselves meet again first.
__device__ __forceinline__ void tmem_load32(uint32_t addr, uint32_t (&v)[32]) {
    __syncwarp();
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
// Waits for all of the warp's loads; v: the registers that are read next, so that no use moves before the wait.
__device__ __forceinline__ void tmem_wait_load(uint32_t (&v)[32]) {
    __syncwarp();
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                   "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]),
                   "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]), "+r"(v[23]),
                   "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]), "+r"(v[30]), "+r"(v[31])
                 :: "memory");
}

// ---- asynchronous tensor core work (one thread; runs in issue order) ------------------

// True in one lane of a converged warp.  The roles below keep the whole warp in their
// loops and elect a lane around the instructions themselves: descriptors and
// addresses are then known to be the same in all lanes and sit in uniform
// registers.  Loops entered by one lane alone cost 86 cycles for each mma that was issued.
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}

// One scale entry (512 bytes) to 4 columns of tensor memory, repeated in each quarter of the lanes.
template <int GROUP>
__device__ __forceinline__ void copy_scales(uint32_t tmem, uint64_t desc) {
    if constexpr (GROUP == 1)
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
    else
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}

// D (+)= A B over 32 of the contracted axis, each side times its scales.
template <int GROUP>
__device__ __forceinline__ void mma_scaled(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                                           bool add) {
    if constexpr (GROUP == 1)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
            ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(uint32_t(add)) : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
            ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(uint32_t(add)) : "memory");
}

// Arrives on `bar` when this thread's earlier tensor core work is done.
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                 ::"r"(smem_u32(bar)) : "memory");
}
// The same on the barrier at this place in both CTAs of the pair.
__device__ __forceinline__ void mma_commit_pair(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
        ::"r"(smem_u32(bar)), "h"(uint16_t(3)) : "memory");
}

// ---- limited waits --------------------------------------------------------------------

// Polls of a wait.  In a build for tests they are drawn: none for one wait of g_give_up_one_in, g_wait_polls for the others.
#ifdef TSENOR_GIVE_UP
static __device__ unsigned g_wait_polls = kTmaPolls, g_give_up_one_in;
static inline int give_up(unsigned polls, unsigned one_in) {
    const cudaError_t e = cudaMemcpyToSymbol(g_wait_polls, &polls, sizeof(polls));
    return e != cudaSuccess ? int(e) : int(cudaMemcpyToSymbol(g_give_up_one_in, &one_in, sizeof(one_in)));
}
__device__ __forceinline__ unsigned wait_polls() {
    const unsigned in = *static_cast<volatile unsigned*>(&g_give_up_one_in);
    const unsigned mixed = (unsigned(clock64()) ^ (blockIdx.x * 64u + threadIdx.x / 32u) * 0x9e3779b9u) * 2654435761u;
    return in && (mixed >> 8) % in == 0 ? 0u : *static_cast<volatile unsigned*>(&g_wait_polls);
}
#else
__device__ __forceinline__ unsigned wait_polls() { return kTmaPolls; }
#endif

// For a converged warp.  The limit is on polls, which lanes make by themselves: if the polls of some ran out and of
// others did not, the warp would come apart in front of instructions that it has to meet as one, so all lanes
// get one verdict.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, unsigned parity, unsigned polls = wait_polls()) {
    bool done = false;
    for (unsigned k = 0; k < polls && !done; ++k) done = mbar_try_wait(bar, parity);
    return __all_sync(0xffffffffu, done);
}
// For what a kernel has in flight when it ends, after a wait that gave up too.
__device__ __forceinline__ bool warp_drain(uint64_t* bar, unsigned parity) { return warp_wait(bar, parity, kTmaPolls); }
// As warp_wait, with each poll asleep for up to 2 us: for warps that have nothing else to do while others work.
__device__ __forceinline__ bool warp_sleep(uint64_t* bar, unsigned parity) {
    const unsigned polls = wait_polls();
    uint32_t done = 0;
    for (unsigned k = 0; k < polls && !done; ++k)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done) : "r"(smem_u32(bar)), "r"(parity), "r"(2000u) : "memory");
    return __all_sync(0xffffffffu, done);
}
// And for a barrier on which other CTAs of the cluster arrive: what they wrote before is visible after it.
__device__ __forceinline__ bool warp_cluster_sleep(uint64_t* bar, unsigned parity) {
    const unsigned polls = wait_polls();
    uint32_t done = 0;
    for (unsigned k = 0; k < polls && !done; ++k)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done) : "r"(smem_u32(bar)), "r"(parity), "r"(2000u) : "memory");
    return __all_sync(0xffffffffu, done);
}

// ---- copies and clusters ----------------------------------------------------------------

// `bytes` (a multiple of 16, both ends 16-byte aligned) from global memory into this CTA.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, unsigned bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(smem_u32(dst)), "l"(__cvta_generic_to_global(src)), "r"(bytes), "r"(smem_u32(bar)) : "memory");
}

// Tile load into this CTA that completes on a barrier of either CTA of the pair
// (`bar`: its address in the cluster).
__device__ __forceinline__ void tma_load_pair(void* dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
        "[%0], [%1, {%2, %3}], [%4];"
        ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar) : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// Arrival on a barrier of any CTA of the cluster.
__device__ __forceinline__ void cluster_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Counts `bytes` on `bar` as if a copy had brought them.
__device__ __forceinline__ void mbar_complete_tx(uint64_t* bar, unsigned bytes) {
    asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}
// Stores to an address of a CTA of the cluster.
__device__ __forceinline__ void cluster_store(uint32_t addr, uint32_t x) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(x) : "memory");
}
__device__ __forceinline__ void cluster_store(uint32_t addr, int64_t x) {
    asm volatile("st.shared::cluster.s64 [%0], %1;" ::"r"(addr), "l"(x) : "memory");
}

// 32 bytes to a 32-byte aligned address in one store.
__device__ __forceinline__ void store32(void* p, const uint32_t (&v)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]) : "memory");
}

__device__ __forceinline__ unsigned cluster_rank() {
    unsigned r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Address of this CTA's shared address `smem` in the CTA of rank `rank`.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t smem, unsigned rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem), "r"(rank));
    return a;
}
__device__ __forceinline__ float4 cluster_load4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

}  // namespace tsenor
