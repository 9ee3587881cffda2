// The NVFP4 product for few tokens and for results of few tiles.
//
// The weights (b's rows) lie on the 128 tensor memory lanes and the tokens
// (a's rows) on BN columns, and a cluster of CTAs splits the reduction of a
// tile, as in the blockwise product's kernel (k_mm_split.cuh).  Here the tensor
// core applies the block scales, so that a tile's sum over its whole share of K
// stays in tensor memory, and is read once.
//
// The first four warps fetch scales, two for the weights and two for the
// tokens, four blocks at a time, and put them where the copies to tensor memory
// take them from; afterwards they, and four more for wide tiles, read the sums.  The next warp loads operands, the last issues the copies and
// the MMAs.
//
// Measured on a GB300, in graphs of calls: one token with 4096 x 4096 weights 4.6 us,
// 16 tokens with 14336 x 4096 7.5 us (4.0 TB/s), one with 18432 x 7168 13.4 to 13.9 us
// (66.6 MB at 4.8 to 5.0 TB/s), 64 with 4096 x 14336 10.0 to 10.6 us.
#pragma once

#include "k_mm_split.cuh"
#include "q_mm4.cuh"

namespace qk {

template <int BN> struct Split4Smem {
    static constexpr int kAtomsQ = (BN + 127) / 128, kPartsQ = BN > 16 ? 2 : 1;   // 128s of tokens, and warps for their scales
    static constexpr int kOperandBytes = (128 + BN) * 128;
    static constexpr int kScaleBytes = (1 + kAtomsQ) * kScaleAtom;
    static constexpr int kStages = BN == 64 ? 3 : BN == 128 ? 6 : 4;
    static constexpr int kScaleCols = 16 * (1 + kAtomsQ);          // tensor memory columns of a stage's scales
    static constexpr int kUsed = BN + 2 * kScaleCols;
    static constexpr int kCols = kUsed <= 128 ? 128 : kUsed <= 256 ? 256 : 512;
    static constexpr int kEpiWarps = BN >= 128 ? 8 : 4;
    static constexpr int kWarpCols = BN / (kEpiWarps / 4);
    static constexpr int kThreads = 32 * (kEpiWarps + 2);
    static constexpr int kResident = BN <= 64 ? 2 : 1;             // CTAs of an SM
    uint8_t stage[kStages][kOperandBytes];       // afterwards this CTA's sums, [BN][128] FP32
    uint8_t scales[2][4][kScaleBytes];           // of two units of four blocks
    uint64_t full[kStages], empty[kStages], sc_full[2], sc_empty[2], done, drained;
    uint32_t tmem_base;
    int abort_flag;
    static_assert(kStages * kOperandBytes >= BN * 128 * 4, "the sums replace the stages");
};

// Half the scale rows (`part`: lines 16 part to 16 part + 15 of the atoms) of ATOMS times 128 rows from row0 on, 32 LAST
// of them in the last, for a CTA's blocks; one warp.  A unit's four blocks are 64
// bytes of a scale row, which four lanes take, so that a load touches 8 lines, and
// are handed over together: a fence waits for the loads that are on their way, so
// the next unit's are issued behind it.
template <int BN, int ATOMS, int LAST, bool WHOLE>
QD void put_split_scales(Split4Smem<BN> &sm, const Mm4Scales &g, int64_t row0, int part, int atom, int kb0, int kb_n, int lane,
                         volatile int *stop, int32_t *status)
{
    row0 += 16 * part;
    for (int u = 0; 4 * u < kb_n; u++) {
        const int slot = u & 1, kb = kb0 + 4 * u;
        ScaleUnit<WHOLE> held[ATOMS];
#pragma unroll
        for (int t = 0; t + 1 < ATOMS; t++) held[t].template load<4>(g, row0 + 128 * t, kb, lane);
        held[ATOMS - 1].template load<LAST>(g, row0 + 128 * (ATOMS - 1), kb, lane);
        const bool got = u < 2 || mm_wait(&sm.sc_empty[slot], ((u >> 1) & 1) ^ 1, stop, status);
        if (!__all_sync(0xFFFFFFFFu, got)) return;
        uint8_t *const to = sm.scales[slot][lane >> 3] + atom * kScaleAtom;
        const int line = 16 * part + (lane & 7);
#pragma unroll
        for (int t = 0; t + 1 < ATOMS; t++) held[t].template put<4>(g, row0 + 128 * t, kb, to + t * kScaleAtom, line, lane);
        held[ATOMS - 1].template put<LAST>(g, row0 + 128 * (ATOMS - 1), kb, to + (ATOMS - 1) * kScaleAtom, line, lane);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.sc_full[slot]);
    }
}

template <int OUT, int BN, bool WHOLE>
__global__ void __launch_bounds__(Split4Smem<BN>::kThreads, Split4Smem<BN>::kResident)
k_mm4_split(const __grid_constant__ CUtensorMap map_p, const __grid_constant__ CUtensorMap map_q, const Mm4Args a)
{
    using Smem = Split4Smem<BN>;
    constexpr int kStages = Smem::kStages, kEpiWarps = Smem::kEpiWarps, kWarpCols = Smem::kWarpCols, kAtomsQ = Smem::kAtomsQ;
    const MmArgs &g = a.store;
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
        for (int s = 0; s < 2; s++) {
            mbar_init(&sm.sc_full[s], 2 + Smem::kPartsQ);
            mbar_init(&sm.sc_empty[s], 1);
        }
        mbar_init(&sm.done, 1);
        mbar_init(&sm.drained, 1);
        sm.abort_flag = g.give_up != 0 && g.give_up != 2 && rank == 0;
        fence_mbar_init();
    }
    if (warp == kEpiWarps && elect_one()) {
        // the weights of the first stages, and their scales, are on their way while the
        // kernel ahead still runs
        prefetch_map(&map_p);
        prefetch_map(&map_q);
        for (int kb = 0; kb < kStages && kb < kb_n; kb++) prefetch_tile(&map_p, (kb0 + kb) * 128, p0);
    }
    if (warp < 4 && p0 + 32 * warp + lane < a.p.rows && (lane & ((1 << a.p.shift) - 1)) == 0)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(a.p.at + ((int64_t)(p0 + 32 * warp + lane) >> a.p.shift) * a.p.pitch + kb0 * 16));
    __syncwarp();
    if (warp == kEpiWarps + 1) tmem_alloc<Smem::kCols>(&sm.tmem_base);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;
    griddep_wait();   // nothing was read or written so far
    griddep_launch_dependents();

    if (warp == kEpiWarps) {
        if (elect_one()) {
            int kb = 0;
            for (; kb < kb_n; kb++) {
                const int s = kb % kStages;
                if (kb >= kStages && !mm_wait(&sm.empty[s], ((kb / kStages) & 1) ^ 1, stop, g.status)) break;
                mbar_arrive_expect_tx(&sm.full[s], Smem::kOperandBytes);
                tma_load_tile(sm.stage[s], &map_p, (kb0 + kb) * 128, p0, &sm.full[s]);
                tma_load_tile(sm.stage[s] + 128 * 128, &map_q, (kb0 + kb) * 128, q0, &sm.full[s]);
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
            const int s = kb % kStages, slot = (kb >> 2) & 1;
            ok = mm_wait(&sm.full[s], (kb / kStages) & 1, stop, g.status);
            if ((kb & 3) == 0) ok = ok && mm_wait(&sm.sc_full[slot], (kb >> 3) & 1, stop, g.status);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
                const uint64_t p = smem_desc_k128(sm.stage[s]), q = smem_desc_k128(sm.stage[s] + 128 * 128);
                const uint64_t src = smem_desc_scales(sm.scales[slot][kb & 3]);
                const uint32_t sp = tmem + BN + (kb & 1) * Smem::kScaleCols, sq = sp + 16;
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    scales_to_tmem(sp + 4 * k, src + 32 * k);
#pragma unroll
                    for (int j = 0; j < kAtomsQ; j++) scales_to_tmem(sq + 4 * (k * kAtomsQ + j), src + 128 * (1 + j) + 32 * k);
                }
#pragma unroll
                for (int k = 0; k < 4; k++)
                    mma_f4(tmem, p + 2 * k, q + 2 * k, idesc_e2m1(128, BN), sp + 4 * k, sq + 4 * kAtomsQ * k, kb > 0 || k > 0);
                mma_commit(&sm.empty[s]);
                if ((kb & 3) == 3) mma_commit(&sm.sc_empty[slot]);
                if (kb + 1 == kb_n) mma_commit(&sm.done);
            }
            __syncwarp();
        }
        if (elect_one()) {   // the MMAs in flight end before their memory goes away, whoever gave up
            if (!ok) mma_commit(&sm.drained);
            (void)mbar_wait_bounded(ok ? &sm.done : &sm.drained, 0);
        }
        __syncwarp();
    } else {
        if (warp < 4) {
            constexpr int kLast = (BN - 128 * (kAtomsQ - 1) + 31) / 32;   // the last tokens, in 32s
            if (warp < 2) put_split_scales<BN, 1, 4, WHOLE>(sm, a.p, p0, warp, 0, kb0, kb_n, lane, stop, g.status);
            else if (warp - 2 < Smem::kPartsQ) put_split_scales<BN, kAtomsQ, kLast, WHOLE>(sm, a.q, q0, warp - 2, 1, kb0, kb_n, lane, stop, g.status);
        }
        __syncwarp();
        const int quad = warp & 3, first = (warp >> 2) * kWarpCols;   // 32 tensor memory lanes, the columns from `first` on
        mm_wait(&sm.done, 0, stop, g.status);
        __syncwarp();
        tc_fence_after();
        // Every MMA is done, so the stages are free.  (After an abort they may
        // not be: then there are no sums, and the cluster writes nothing.)
        if (!__any_sync(0xFFFFFFFFu, *stop)) {
            float *sums = reinterpret_cast<float *>(dsm);
#pragma unroll
            for (int h = 0; h < kWarpCols / 16; h++) {
                uint32_t r[16];
                tmem_ld16(r, tmem + ((uint32_t)(quad * 32) << 16) + first + h * 16);
#pragma unroll
                for (int j = 0; j < 16; j++) sums[(first + h * 16 + j) * 128 + quad * 32 + lane] = __uint_as_float(r[j]);
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kEpiWarps + 1) tmem_free<Smem::kCols>(tmem);
    // A CTA that gave up has operands where the others look for its sums.  It leaves
    // NaNs there, and who meets one looks at the flags.
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
        const float s_p = load_float(a.s_p), s_q = load_float(a.s_q);
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
                // one at a time: the tensors' scales may be far apart, their product too small
                v = make_float4(v.x * s_p * s_q, v.y * s_p * s_q, v.z * s_p * s_q, v.w * s_p * s_q);
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
