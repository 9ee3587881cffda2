// Fifth-generation tensor core helpers (sm_103a): tensor memory allocation,
// descriptors, FP8 MMA issue, commits and accumulator loads, as inline PTX.
#pragma once

#include "q_engine.cuh"
#include "q_packed.cuh"

namespace qk {

// ---------------------------------------------------------------------------
// tensor memory: 128 lanes x 512 columns of 32 bits per SM.  An address holds
// the lane in bits 31-16 and the column in bits 15-0.
// ---------------------------------------------------------------------------

// Whole-warp allocation of COLS columns (a power of two >= 32); the base
// address is written to *dst in shared memory.
template <int COLS> QD void tmem_alloc(uint32_t *dst)
{
    static_assert(COLS >= 32 && COLS <= 512 && (COLS & (COLS - 1)) == 0, "column count");
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "n"(COLS) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
template <int COLS> QD void tmem_free(uint32_t base)
{
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "n"(COLS) : "memory");
}

QD void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
QD void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// ---------------------------------------------------------------------------
// operands and instruction shape
// ---------------------------------------------------------------------------

// Shared-memory descriptor of a K-major operand tile whose rows are 128 bytes,
// stored in the 128-byte swizzle (8-row groups of 1 KiB, tile 1 KiB aligned):
// start address / 16 in bits 13-0, byte distance of the 8-row groups / 16 in
// bits 45-32, descriptor version 1 in bits 48-46, swizzle code 2 in bits 63-61.
// A step of 32 bytes along K adds 2 to the start address.
QD uint64_t smem_desc_k128(const void *tile)
{
    return (uint64_t)((smem_u32(tile) >> 4) & 0x3FFFu) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}

// Instruction descriptor: E4M3 x E4M3 -> FP32, both operands K-major, M x N.
__host__ __device__ constexpr uint32_t idesc_e4m3(int m, int n)
{
    return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// One lane of a converged warp, the same one every time.  Code behind it that
// issues MMAs keeps their descriptors in uniform registers: behind a test of
// the lane number, which the compiler does not know to pick one lane, an MMA
// takes 70 cycles to issue, four times as long.
QD bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// D (+)= A B^T over 32 elements of K; add = 0 overwrites D.  One thread.
QD void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add)
{
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "setp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
                 ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(add) : "memory");
}

// The barrier gets one arrival when every MMA this thread has issued is done
// (this also orders their reads of shared memory before the arrival).
QD void mma_commit(uint64_t *bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// ---------------------------------------------------------------------------
// block-scaled FP4
// ---------------------------------------------------------------------------

// Instruction descriptor: E2M1 x E2M1 -> FP32 with unsigned E4M3 scales, both
// operands K-major, M x N, 64 elements of K.
__host__ __device__ constexpr uint32_t idesc_e2m1(int m, int n)
{
    return (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// Scales in tensor memory: the four scales of a row's 64 elements are one
// 32-bit word, row r's in lane r % 32 (of each of the four quarters) and column
// r / 32 from the address on.  This descriptor is of a copy's source, 32 lanes x
// 16 bytes (four columns) in a row: lane l's words at 16 l, so that the 8-lane
// groups are 128 bytes apart, no swizzle.
QD uint64_t smem_desc_scales(const void *p)
{
    return (uint64_t)((smem_u32(p) >> 4) & 0x3FFFu) | (8ull << 32) | (1ull << 46);
}
// 512 bytes of scales to tensor memory, to all four quarters.  MMAs that the
// same thread issues afterwards read them, those before have read what was there.
QD void scales_to_tmem(uint32_t d, uint64_t desc)
{
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(d), "l"(desc) : "memory");
}
// The same in both CTAs of a pair, each from its own shared memory at this offset.
QD void scales_to_tmem_pair(uint32_t d, uint64_t desc)
{
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(d), "l"(desc) : "memory");
}

// D (+)= A B^T over 64 elements of K, each 16 of a row times their scale; add = 0
// overwrites D.  sa, sb: the scales' columns.  One thread.
QD void mma_f4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb, uint32_t add)
{
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "setp.ne.b32 p, %6, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
                 ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(add) : "memory");
}
QD void mma_f4_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb, uint32_t add)
{
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "setp.ne.b32 p, %6, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
                 ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(add) : "memory");
}

// ---------------------------------------------------------------------------
// clusters
// ---------------------------------------------------------------------------

QD uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// All threads of the cluster; orders shared memory accesses before it.
QD void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Address of shared memory address `addr`'s counterpart in cluster rank `rank`.
QD uint32_t cluster_addr(uint32_t addr, int rank)
{
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
// A word of the cluster's shared memory, which another CTA may write or read meanwhile.
QD int ld_cluster1(uint32_t addr)
{
    int v;
    asm volatile("ld.relaxed.cluster.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
QD void st_cluster1(uint32_t addr, int v) { asm volatile("st.relaxed.cluster.shared::cluster.s32 [%0], %1;" ::"r"(addr), "r"(v) : "memory"); }
// Arrival on a barrier of the cluster.  No data in generic memory is handed
// over with it (only tensor memory that has been read, which the tcgen05
// fences order), so it and the waits for it stay at CTA scope: an acquire at
// cluster scope drops the L1 on every wait.
QD void mbar_arrive_cluster(uint32_t addr)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
// Arrival that hands over what this thread, and those whose word it has, wrote to their CTA's shared memory, to a
// thread of the cluster that waits and fences in turn.  The fences leave memory elsewhere alone: a release of
// everything waits for loads on their way as well, behind copies that keep memory's queues full.
QD void mbar_arrive_shared_cluster(uint32_t addr)
{
    asm volatile("fence.release.sync_restrict::shared::cta.cluster;\n\t"
                 "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
// The phase alone, whichever CTA of the cluster completed it: a fence behind it says what else is seen.
QD bool mbar_try_wait_relaxed_cluster(uint64_t *bar, uint32_t parity)
{
    uint32_t done;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(done) : "r"(smem_u32(bar)), "r"(parity) : "memory");
    return done != 0;
}
QD void shared_acquire_cluster() { asm volatile("fence.acquire.sync_restrict::shared::cluster.cluster;" ::: "memory"); }

// Ahead of a kernel's loads: its tensor map, and a tile into L2 (coherent: a
// later write reaches it there).
QD void prefetch_map(const CUtensorMap *map) { asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory"); }
QD void prefetch_tile(const CUtensorMap *map, int x, int y)
{
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(map), "r"(x), "r"(y) : "memory");
}

// CTA pairs (clusters of two): one MMA spans both CTAs' tensor memory, each CTA
// holding its own 128 rows of A and D and half of B's rows.  All tensor memory
// instructions of such a kernel name the pair.
template <int COLS> QD void tmem_alloc_pair(uint32_t *dst)
{
    static_assert(COLS >= 32 && COLS <= 512 && (COLS & (COLS - 1)) == 0, "column count");
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "n"(COLS) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
template <int COLS> QD void tmem_free_pair(uint32_t base)
{
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(base), "n"(COLS) : "memory");
}
// A tile into this CTA's shared memory whose bytes count on a barrier of the
// pair (bar: a cluster address, this CTA's or its peer's).
QD void tma_load_tile_pair(void *dst, const CUtensorMap *map, int x, int y, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3}], [%4];"
                 ::"r"(smem_u32(dst)), "l"(map), "r"(x), "r"(y), "r"(bar) : "memory");
}
// Bytes that `bar` awaits and that will not come.
QD void mbar_complete_tx(uint64_t *bar, uint32_t bytes)
{
    asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}
// mma_f8 over the pair: the descriptors give offsets that hold in both CTAs.
QD void mma_f8_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add)
{
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "setp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
                 ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(add) : "memory");
}
// mma_commit with one arrival on the barrier at this offset in both CTAs.
QD void mma_commit_pair(uint64_t *bar)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                 ::"r"(smem_u32(bar)), "h"((uint16_t)3) : "memory");
}

// Moves registers between warpgroups (all four warps of one; multiples of 8,
// the kernel's sum at most what it was launched with).
template <int N> QD void regs_more() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> QD void regs_fewer() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// ---------------------------------------------------------------------------
// accumulator loads, complete when they return.  A load and its wait are one
// statement: between two, the compiler may use (it moves) registers that the
// load has yet to write.
// ---------------------------------------------------------------------------

// Lane l of the warp gets 16 columns of tensor memory lane (address lane + l).
QD void tmem_ld16(uint32_t (&r)[16], uint32_t addr)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
                 "tcgen05.wait::ld.sync.aligned;"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(addr) : "memory");
}
// 64 columns alike.
QD void tmem_ld64(uint32_t (&r)[64], uint32_t addr)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x64.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, "
                 "%8, %9, %10, %11, %12, %13, %14, %15, "
                 "%16, %17, %18, %19, %20, %21, %22, %23, "
                 "%24, %25, %26, %27, %28, %29, %30, %31, "
                 "%32, %33, %34, %35, %36, %37, %38, %39, "
                 "%40, %41, %42, %43, %44, %45, %46, %47, "
                 "%48, %49, %50, %51, %52, %53, %54, %55, "
                 "%56, %57, %58, %59, %60, %61, %62, %63}, [%64];\n\t"
                 "tcgen05.wait::ld.sync.aligned;"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
                   "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
                   "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
                   "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
                   "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
                   "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
                   "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
                 : "r"(addr) : "memory");
}
// 16 lanes from the address on, 32 columns: thread t of the warp gets rows
// t / 4 (r[4i], r[4i + 1]) and t / 4 + 8 (r[4i + 2], r[4i + 3]) of columns
// 8i + 2 (t % 4) and the next.
QD void tmem_ld_rows16(uint32_t (&r)[16], uint32_t addr)
{
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x4.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
                 "tcgen05.wait::ld.sync.aligned;"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(addr) : "memory");
}

// Arrival at barrier `id` (1..15, `count` threads in all) without waiting.
QD void named_barrier_arrive(int id, int count) { asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(count) : "memory"); }

QD void mbar_arrive(uint64_t *bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

}  // namespace qk
