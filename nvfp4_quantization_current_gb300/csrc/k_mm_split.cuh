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
// Warps 0-3 scale and add (one thread per row), warp 4 loads, warp 5 issues
// the MMAs.  Two CTAs fit an SM: about 100 KiB of stages each and at most half
// of tensor memory.
#pragma once

#include "q_internal.h"
#include "q_mm.cuh"

namespace qk {

constexpr int kSplitThreads = 192;
constexpr int kSplitMost = 8;   // CTAs of a cluster

template <int BN> struct SplitSmem {
    static constexpr int kStageBytes = (128 + BN) * kMmBlock;
    static constexpr int kStages = BN == 16 ? 6 : BN == 32 ? 5 : BN == 64 ? 4 : 3;
    static constexpr int kBufs = BN == 128 ? 2 : 4;
    static constexpr int kCols = BN * kBufs;   // of tensor memory
    uint8_t stage[kStages][kStageBytes];       // afterwards this CTA's sums, [BN][128] FP32
    float col_scale[2][BN];
    uint64_t full[kStages], empty[kStages], acc_full[kBufs], acc_empty[kBufs], drained;
    uint32_t tmem_base;
    int abort_flag;
    static_assert(kStages * kStageBytes >= BN * 128 * 4, "the sums replace the stages");
};

QD float ld_cluster(uint32_t addr)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

template <int OUT, int BN>
__global__ void __launch_bounds__(kSplitThreads)
k_mm_split(const __grid_constant__ CUtensorMap map_p, const __grid_constant__ CUtensorMap map_q, const MmArgs g)
{
    using Smem = SplitSmem<BN>;
    constexpr int kStages = Smem::kStages, kBufs = Smem::kBufs;
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
            mbar_init(&sm.acc_empty[b], 4);
        }
        mbar_init(&sm.drained, 1);
        sm.abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 5) tmem_alloc<Smem::kCols>(&sm.tmem_base);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;

    if (warp == 4) {
        if (elect_one()) {
            int kb = 0;
            for (; kb < kb_n; kb++) {
                const int s = kb % kStages;
                if (kb >= kStages && !mm_wait(&sm.empty[s], ((kb / kStages) & 1) ^ 1, stop, g.status)) break;
                mbar_arrive_expect_tx(&sm.full[s], Smem::kStageBytes);
                tma_load_tile(sm.stage[s], &map_p, (kb0 + kb) * kMmBlock, p0, &sm.full[s]);
                tma_load_tile(sm.stage[s] + 128 * kMmBlock, &map_q, (kb0 + kb) * kMmBlock, q0, &sm.full[s]);
            }
            if (kb < kb_n)   // aborted: the copies in flight land before shared memory goes away
                for (int j = kb > kStages ? kb - kStages : 0; j < kb; j++)
                    (void)mbar_wait_bounded(&sm.full[j % kStages], (j / kStages) & 1);
        }
    } else if (warp == 5) {
        bool ok = true;
        for (int kb = 0; kb < kb_n; kb++) {
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
        const int64_t row = (int64_t)p0 + t, col = (int64_t)q0 + t;
        // rows and columns outside the result have zero products: any scale in bounds does
        const float *sp = g.s_p + ((row < g.rows_p ? row : 0) >> g.shift_p) * g.kblocks;
        const float *sq = g.s_q + ((col < g.rows_q ? col : 0) >> g.shift_q) * g.kblocks;
        float acc[BN];
#pragma unroll
        for (int j = 0; j < BN; j++) acc[j] = 0.0f;
        // a block's scales are fetched four blocks ahead
        float rs[4], cs[4];
        const bool fetches = t < BN;
        auto fetch = [&](float &r, float &c, int kb) {
            const int at = kb0 + kb < kb_all ? kb0 + kb : kb_all - 1;
            r = __ldg(sp + at);
            if (fetches) c = __ldg(sq + at);
        };
#pragma unroll
        for (int i = 0; i < 4; i++) fetch(rs[i], cs[i], i);
        bool ok = true;
#pragma unroll 1
        for (int kb = 0; kb < kb_n; kb++) {
            const int b = kb % kBufs, cb = kb & 1;
            const float s = rs[0];
            if (fetches) sm.col_scale[cb][t] = cs[0];
#pragma unroll
            for (int i = 0; i < 3; i++) {
                rs[i] = rs[i + 1];
                cs[i] = cs[i + 1];
            }
            fetch(rs[3], cs[3], kb + 4);
            ok = ok && mm_wait(&sm.acc_full[b], (kb / kBufs) & 1, stop, g.status);
            ok = __all_sync(0xFFFFFFFFu, ok);
            named_barrier(1, 128);   // the scales are there, and every thread is done with the other buffer's
            if (ok) {
                tc_fence_after();
                constexpr int W = BN < 32 ? 16 : 32;
#pragma unroll
                for (int h = 0; h < BN / W; h++) {
                    uint32_t r[W];
                    const uint32_t addr = tmem + ((uint32_t)(warp * 32) << 16) + b * BN + h * W;
                    if constexpr (W == 16) tmem_ld16(r, addr);
                    else tmem_ld32(r, addr);
                    if (h + 1 == BN / W) {   // all read: the next block may go there
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sm.acc_empty[b]);
                    }
#pragma unroll
                    for (int j = 0; j < W; j++)
                        acc[h * W + j] = __fmaf_rn(__uint_as_float(r[j]) * sm.col_scale[cb][h * W + j], s, acc[h * W + j]);
                }
            }
        }
        // Every MMA is done, so the stages are free.  (After an abort they may
        // not be, but neither is the result then: nothing is written.)
        if (ok) {
            float *sums = reinterpret_cast<float *>(dsm);
#pragma unroll
            for (int j = 0; j < BN; j++) sums[j * 128 + t] = acc[j];
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 5) tmem_free<Smem::kCols>(tmem);
    if (split > 1) cluster_sync();   // the cluster's sums are there
    if (warp < 4 && sm.abort_flag == 0) {
        using T = typename OutT<OUT>::T;
        const int t = threadIdx.x;
        const int64_t row = (int64_t)p0 + t;
        const uint32_t mine = smem_u32(dsm) + 4 * t;
        for (int j = BN * rank / split; j < BN * (rank + 1) / split; j++) {
            const int64_t col = (int64_t)q0 + j;
            if (col >= g.rows_q) break;
            float v = 0.0f;
            for (int r = 0; r < split; r++) {
                uint32_t at = mine + j * 512;
                if (split > 1) asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(mine + j * 512), "r"(r));
                v += ld_cluster(at);
            }
            if (row < g.rows_p) put_one<OUT>(static_cast<T *>(g.c) + col * g.ldc + row, v, g.accumulate);
        }
    }
    if (split > 1) cluster_sync();   // nobody reads this CTA's sums any more
}

}  // namespace qk
