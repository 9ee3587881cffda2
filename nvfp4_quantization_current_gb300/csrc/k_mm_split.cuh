// The block-scaled product for few tokens and for results of few tiles.
//
// The weights (b's rows) lie on the 128 tensor memory lanes and the tokens
// (a's rows) on BN columns, so that one token costs an MMA 16 columns wide and
// not 128 rows, and a warp's stores run along C's rows.  These calls are bound
// by reading the weights, and there are too few tiles to fill the machine with
// one CTA each: a cluster of CTAs splits the reduction of a tile, each keeps
// its FP32 sums in registers, and the cluster adds them through its shared
// memory in rank order, each CTA a slice of the columns.  Nothing is added in
// an order that depends on timing, and no workspace is needed.
//
// The first warps, four or for wide tiles eight, scale and add (one thread per
// row of their columns), the next loads, the last issues the MMAs.  Up to 64
// tokens wide, two CTAs fit an SM: about 100 KiB of stages each and at most
// half of tensor memory.
//
// Measured on a GB300, in graphs of calls: one token with 4096 x 4096 weights
// 4.8 us (three sets of inputs in turn, whose weights stay in L2; 6.4 with ten
// sets, whose weights come from memory; the launch and two trips to memory are
// most of it), 16 tokens with 14336 x 4096 12.2 to 12.6 us (4.7 TB/s), one token
// with 18432 x 7168 22.4 us (5.9 TB/s), 333 tokens with 4096 x 4096 14.6 to 14.8
// us (760 TFLOP/s; a block of 128 x 192 takes 1050 cycles, where shared memory
// needs 640 and the MMAs 384; without reading and adding it the call took 11.6 us
// of 14.5, without its column scales 13.6, so that loads and what a call costs
// whatever its size are the larger part).  Tried there and not faster: loads of 32 columns, and
// the 16-lane loads of the pair kernel, which need a quarter of the column
// scales (15.4 us; 15.2 against 16.4 where each weight row has a scale).
#pragma once

#include "q_internal.h"
#include "q_mm.cuh"

namespace qk {

constexpr int kSplitMost = 8;   // CTAs of a cluster

template <int BN> struct SplitSmem {
    static constexpr int kStageBytes = (128 + BN) * kMmBlock;
    static constexpr int kStages = BN == 16 || BN == 128 ? 6 : BN == 32 ? 5 : 4;
    static constexpr int kBufs = BN > 128 ? 2 : 4;
    static constexpr int kCols = BN == 192 ? 512 : BN * kBufs;   // of tensor memory, a power of two
    static constexpr int kEpiWarps = BN >= 128 ? 8 : 4;
    static constexpr int kWarpCols = BN / (kEpiWarps / 4);
    static constexpr int kThreads = 32 * (kEpiWarps + 2);
    static constexpr int kResident = BN <= 64 ? 2 : 1;         // CTAs of an SM
    uint8_t stage[kStages][kStageBytes];       // afterwards this CTA's sums, [BN][128] FP32
    alignas(16) float col_scale[2][4][BN];     // of two groups of four blocks
    uint64_t full[kStages], empty[kStages], acc_full[kBufs], acc_empty[kBufs], drained;
    uint32_t tmem_base;
    int abort_flag;
    static_assert(kStages * kStageBytes >= BN * 128 * 4, "the sums replace the stages");
};

QD float4 ld_cluster4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
    return v;
}
// Whether a CTA of the cluster gave up.
QD bool cluster_gave_up(const int *abort_flag, int split)
{
#pragma unroll 1
    for (int r = 0; r < split; r++)
        if (ld_cluster1(cluster_addr(smem_u32(abort_flag), r)) != 0) return true;
    return false;
}
// TILES: the weights have 128x128 tiles, so that a block's row scale is one
// number and goes into the column scales.
template <int OUT, int BN, bool TILES>
__global__ void __launch_bounds__(SplitSmem<BN>::kThreads, SplitSmem<BN>::kResident)
k_mm_split(const __grid_constant__ CUtensorMap map_p, const __grid_constant__ CUtensorMap map_q, const MmArgs g)
{
    using Smem = SplitSmem<BN>;
    constexpr int kStages = Smem::kStages, kBufs = Smem::kBufs, kEpiWarps = Smem::kEpiWarps, kWarpCols = Smem::kWarpCols;
    constexpr bool kAhead = kWarpCols <= 64;
    extern __shared__ __align__(1024) uint8_t dsm[];
    Smem &sm = *reinterpret_cast<Smem *>(dsm);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int split = (int)gridDim.x, rank = (int)blockIdx.x;   // a cluster is the grid's x extent
    const int p0 = (int)blockIdx.y * 128, q0 = (int)blockIdx.z * BN;
    const int kb0 = (int)(g.kblocks * rank / split), kb_n = (int)(g.kblocks * (rank + 1) / split) - kb0;
    volatile int *const stop = &sm.abort_flag;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; s++) {
            mbar_init(&sm.full[s], 1);
            mbar_init(&sm.empty[s], 1);
        }
        for (int b = 0; b < kBufs; b++) {
            mbar_init(&sm.acc_full[b], 1);
            mbar_init(&sm.acc_empty[b], kEpiWarps);
        }
        mbar_init(&sm.drained, 1);
        sm.abort_flag = g.give_up != 0 && g.give_up != 2 && rank == 0;
        fence_mbar_init();
    }
    if (warp == kEpiWarps && elect_one()) {
        // The weights of the first stages are on their way from memory while the
        // kernel ahead still runs (16 tokens with 14336 x 4096 12.9 us, 12.2 so; one with
        // 18432 x 7168 23.9 and 22.4; with 4096 x 4096, where most of a CTA's weights are
        // its first stages', 6.3 and 6.4; twice as many stages are no better).
        prefetch_map(&map_p);
        prefetch_map(&map_q);
        for (int kb = 0; kb < kStages && kb < kb_n; kb++) prefetch_tile(&map_p, (kb0 + kb) * kMmBlock, p0);
    }
    __syncwarp();
    if (warp == kEpiWarps + 1) tmem_alloc<Smem::kCols>(&sm.tmem_base);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;
    // Launched while the kernel ahead still ran; nothing was read or written so far
    // (what the prefetch put into L2 is read there, after any write to it).
    griddep_wait();
    griddep_launch_dependents();

    if (warp == kEpiWarps) {
        if (elect_one()) {
            int kb = 0;
            for (; kb < kb_n; kb++) {
                const int s = kb % kStages;
                if (kb >= kStages && !mm_wait(&sm.empty[s], ((kb / kStages) & 1) ^ 1, stop, g.status)) break;
                mbar_arrive_expect_tx(&sm.full[s], Smem::kStageBytes);
                tma_load_tile(sm.stage[s], &map_p, (kb0 + kb) * kMmBlock, p0, &sm.full[s]);
                tma_load_tile(sm.stage[s] + 128 * kMmBlock, &map_q, (kb0 + kb) * kMmBlock, q0, &sm.full[s]);
            }
            // All that was issued lands before shared memory is put to other use or goes away, whoever gave up: where
            // the MMAs' warp did, copies that nobody reads may be in flight.
            for (int j = kb > kStages ? kb - kStages : 0; j < kb; j++)
                (void)mbar_wait_bounded(&sm.full[j % kStages], (j / kStages) & 1);
        }
    } else if (warp == kEpiWarps + 1) {
        bool ok = g.give_up != 2 || rank != 0;
        if (!ok) *stop = 1;   // the test's wait that runs out
        for (int kb = 0; ok && kb < kb_n; kb++) {
            const int s = kb % kStages, b = kb % kBufs;
            ok = kb < kBufs || mm_wait(&sm.acc_empty[b], ((kb / kBufs) & 1) ^ 1, stop, g.status);
            ok = ok && mm_wait(&sm.full[s], (kb / kStages) & 1, stop, g.status);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
                const uint64_t a = smem_desc_k128(sm.stage[s]), w = smem_desc_k128(sm.stage[s] + 128 * kMmBlock);
#pragma unroll
                for (int k = 0; k < kMmBlock / 32; k++) mma_f8(tmem + b * BN, a + 2 * k, w + 2 * k, idesc_e4m3(128, BN), k > 0);
                mma_commit(&sm.empty[s]);
                mma_commit(&sm.acc_full[b]);
            }
            __syncwarp();
        }
        if (!ok && elect_one()) {   // aborted: the MMAs in flight end before their memory goes away
            mma_commit(&sm.drained);
            (void)mbar_wait_bounded(&sm.drained, 0);
        }
        __syncwarp();
    } else {
        const int t = threadIdx.x, kb_all = (int)g.kblocks;
        const int quad = warp & 3, first = (warp >> 2) * kWarpCols;   // 32 tensor memory lanes, the columns from `first` on
        const int64_t row = (int64_t)p0 + quad * 32 + lane, col = (int64_t)q0 + t;
        // rows and columns outside the result have zero products: any scale in bounds does
        const float *sp = g.s_p + ((row < g.rows_p ? row : 0) >> g.shift_p) * g.kblocks;
        const float *sq = g.s_q + ((col < g.rows_q ? col : 0) >> g.shift_q) * g.kblocks;
        uint64_t acc[kWarpCols / 2];   // two columns each
#pragma unroll
        for (int j = 0; j < kWarpCols / 2; j++) acc[j] = 0ull;
        // the scales of the next four blocks are on their way while four are used
        float rs[4], rs_next[4], cs_next[4];
        const bool fetches = t < BN;
        auto fetch = [&](int kb) {
            load_scales4(rs_next, sp, kb, kb_all);
            if (fetches) load_scales4(cs_next, sq, kb, kb_all);
        };
        fetch(kb0);
#pragma unroll 1
        for (int kb = 0; kb < kb_n; kb++) {
            const int b = kb % kBufs, i = kb & 3;
            if (i == 0) {
                if (fetches) {
#pragma unroll
                    for (int k = 0; k < 4; k++) sm.col_scale[(kb >> 2) & 1][k][t] = TILES ? cs_next[k] * rs_next[k] : cs_next[k];
                }
#pragma unroll
                for (int k = 0; k < 4; k++) rs[k] = rs_next[k];
                fetch(kb0 + kb + 4);
                named_barrier(1, 32 * kEpiWarps);   // they are there, and every thread is done with the group before the last
            }
            const uint64_t ss = pack2(__float_as_uint(rs[0]), __float_as_uint(rs[0]));
#pragma unroll
            for (int k = 0; k < 3; k++) rs[k] = rs[k + 1];
            const float *const cs = &sm.col_scale[(kb >> 2) & 1][i][first];
            // After a wait that gave up the rest goes by as it is; it is not stored then.
            mm_wait(&sm.acc_full[b], (kb / kBufs) & 1, stop, g.status);
            __syncwarp();
            tc_fence_after();
            const uint32_t addr = tmem + ((uint32_t)(quad * 32) << 16) + b * BN + first;
#pragma unroll
            for (int h = 0; h < kWarpCols / 16; h++) {
                // The 16 columns' scales are fetched ahead of the load, not behind its wait
                // (192 x 2048 x 8192 10.8 us, behind it 11.2), where registers allow: at 96
                // columns a warp they do not (333 x 4096 x 4096 14.5 us against 16.5).
                ulonglong2 cc[4];
                if constexpr (kAhead) {
#pragma unroll
                    for (int j = 0; j < 4; j++) cc[j] = *reinterpret_cast<const ulonglong2 *>(cs + h * 16 + 4 * j);
                    asm volatile("" ::: "memory");
                }
                uint32_t r[16];
                tmem_ld16(r, addr + h * 16);
                if (h + 1 == kWarpCols / 16) {   // all read: the next block may go there
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.acc_empty[b]);
                }
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    const ulonglong2 c = kAhead ? cc[j / 2] : *reinterpret_cast<const ulonglong2 *>(cs + h * 16 + 2 * j);
                    const uint64_t v0 = pack2(r[2 * j], r[2 * j + 1]), v1 = pack2(r[2 * j + 2], r[2 * j + 3]);
                    acc[h * 8 + j] = TILES ? ffma2(v0, c.x, acc[h * 8 + j]) : ffma2(fmul2(v0, c.x), ss, acc[h * 8 + j]);
                    acc[h * 8 + j + 1] = TILES ? ffma2(v1, c.y, acc[h * 8 + j + 1]) : ffma2(fmul2(v1, c.y), ss, acc[h * 8 + j + 1]);
                }
            }
        }
        // Every MMA is done, so the stages are free.  (After an abort they may
        // not be: then there are no sums, and the cluster writes nothing.)
        if (!__any_sync(0xFFFFFFFFu, *stop)) {
            float *sums = reinterpret_cast<float *>(dsm);
#pragma unroll
            for (int j = 0; j < kWarpCols / 2; j++)
                unpack2(acc[j], sums[(first + 2 * j) * 128 + quad * 32 + lane], sums[(first + 2 * j + 1) * 128 + quad * 32 + lane]);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kEpiWarps + 1) tmem_free<Smem::kCols>(tmem);
    // A CTA that gave up has operands where the others look for its sums.  It leaves
    // NaNs there, and who meets one looks at the flags (looking at every call took 0.2 us of it).
    const bool gave_up = sm.abort_flag != 0;
    if (gave_up) {
        if (g.give_up && threadIdx.x == 0 && g.status != nullptr) atomicOr(g.status, kStTimeout);
#pragma unroll 1
        for (int i = threadIdx.x; i < BN * 128; i += Smem::kThreads) reinterpret_cast<uint32_t *>(dsm)[i] = 0x7FFFFFFFu;
        __syncwarp();
    }
    if (split > 1) cluster_sync();   // the cluster's sums are there
    if (warp < kEpiWarps && !gave_up) {
        // a warp takes two columns at a time, four rows per lane
        using T = typename OutT<OUT>::T;
        const int64_t row = (int64_t)p0 + 4 * lane;
        const bool vec = (g.ldc & 3) == 0 && row + 4 <= g.rows_p && !g.accumulate;
        const int j1 = BN * (rank + 1) / split;
        for (int j0 = BN * rank / split + 2 * warp; j0 < j1; j0 += 2 * kEpiWarps) {
            float4 part[2][kSplitMost];
#pragma unroll
            for (int u = 0; u < 2; u++)
#pragma unroll
                for (int r = 0; r < kSplitMost; r++) {
                    const uint32_t at = smem_u32(dsm) + (j0 + u) * 512 + lane * 16;
                    if (r < split && j0 + u < j1) part[u][r] = ld_cluster4(split > 1 ? cluster_addr(at, r) : at);
                }
#pragma unroll
            for (int u = 0; u < 2; u++) {
                const int64_t col = (int64_t)q0 + j0 + u;
                if (j0 + u >= j1 || col >= g.rows_q) break;
                float4 v = part[u][0];
#pragma unroll
                for (int r = 1; r < kSplitMost; r++)
                    if (r < split) {
                        v.x += part[u][r].x;
                        v.y += part[u][r].y;
                        v.z += part[u][r].z;
                        v.w += part[u][r].w;
                    }
                if (v.x != v.x && split > 1 && cluster_gave_up(&sm.abort_flag, split)) continue;
                T *c = static_cast<T *>(g.c) + col * g.ldc + row;
                if (vec) {
                    if constexpr (OUT == F32) *reinterpret_cast<float4 *>(c) = v;
                    else *reinterpret_cast<uint2 *>(c) = make_uint2(bf16_pair(v.x, v.y), bf16_pair(v.z, v.w));
                } else {
                    const float e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        if (row + i < g.rows_p) put_one<OUT>(c + i, e[i], g.accumulate);
                }
            }
        }
    }
    if (split > 1) cluster_sync();   // nobody reads this CTA's sums any more
}

}  // namespace qk
