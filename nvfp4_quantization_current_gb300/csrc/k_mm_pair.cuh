// The block-scaled product for results of many tiles.
//
// A CTA owns a 128 x 256 tile of C and walks the tiles persistently with the
// CTA beside it (a cluster of two), which owns the 128 rows below: both need
// the same 256 rows of Q, so each loads half of them and multicasts it to
// both.  A stage of 128 elements of K costs a CTA 32 KiB of loads from L2 for
// 128 x 256 x 128 products.  The block products alternate between two
// accumulator buffers, which together fill tensor memory.
//
// Warp 0 loads operand tiles, one thread of warp 1 issues the MMAs, warp 2
// fetches the column scales when Q has 1x128 tiles, and the eight warps 4-11
// keep the FP32 sums of 32 rows x 128 columns each in registers: a block's
// product is read from tensor memory, multiplied by its scales and added while
// the next block's runs.  Finished tiles go through shared memory to C as bulk
// tensor stores (adds, when accumulating in FP32), 32 rows x 128 bytes each.
//
// The hand-over of the accumulator buffers is what the block rate hangs on:
// MMAs, commit, read, release and the next MMAs into the same buffer form a
// chain, of which two are in flight.  It stays inside the CTA (one MMA over
// both CTAs of a pair would need half the loads of Q, but its chain crosses
// the pair twice per block and took twice as long).
#pragma once

#include "q_internal.h"
#include "q_mm.cuh"

namespace qk {

constexpr int kPairThreads = 384;
constexpr int kPairStages = 4;
constexpr int kPairN = 256;       // columns of a CTA's tile
constexpr int kPairStageBytes = (128 + kPairN) * kMmBlock;
constexpr int kPairScaleSlots = 2;
constexpr int kPairEpiWarps = 8;
constexpr int kPairGroup = 8;     // tile rows per group of the tile order

struct PairSmem {
    uint8_t stage[kPairStages][kPairStageBytes];
    uint8_t staging[kPairEpiWarps][4096];
    float col_scale[kPairScaleSlots][kPairN];
    uint64_t full[kPairStages], empty[kPairStages], acc_full[2], acc_empty[2], drained;
    uint64_t sc_full[kPairScaleSlots], sc_empty[kPairScaleSlots];
    uint32_t tmem_base;
    int abort_flag;
};
static_assert(sizeof(PairSmem) <= 232448, "shared memory of a CTA");

// Tile t of the walk, in units of 256 x 256: groups of kPairGroup tile rows,
// each walked column by column, so that the tiles in flight share their
// operands in L2.
QD void pair_tile(int t, int tiles_p, int tiles_q, int &p, int &q)
{
    const int per_group = kPairGroup * tiles_q;
    const int gp = t / per_group * kPairGroup, r = t % per_group;
    const int height = tiles_p - gp < kPairGroup ? tiles_p - gp : kPairGroup;
    p = gp + r % height;
    q = r / height;
}

// Four consecutive block scales from kb on, the last one repeated past the end.
QD void load_scales4(float (&s)[4], const float *row, int kb, int kb_n, bool vec)
{
    if (vec) {   // K / 128 a multiple of 4 and 16-byte aligned rows: kb + 3 exists
        const float4 v = __ldg(reinterpret_cast<const float4 *>(row + (kb < kb_n ? kb : 0)));
        s[0] = v.x;
        s[1] = v.y;
        s[2] = v.z;
        s[3] = v.w;
    } else {
#pragma unroll
        for (int j = 0; j < 4; j++) s[j] = __ldg(row + (kb + j < kb_n ? kb + j : kb_n - 1));
    }
}

// COLS: Q has a scale per row (1x128 tiles); otherwise one per 128 of its rows.
template <int OUT, bool COLS>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
k_mm_pair(const __grid_constant__ CUtensorMap map_p, const __grid_constant__ CUtensorMap map_q,
          const __grid_constant__ CUtensorMap map_c, const MmArgs g)
{
    extern __shared__ __align__(1024) uint8_t dsm[];
    PairSmem &sm = *reinterpret_cast<PairSmem *>(dsm);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int kb_n = (int)g.kblocks;
    const int rows_p = (int)g.rows_p, rows_q = (int)g.rows_q;   // below 2^31, and fewer than 2^31 tiles
    const int tiles_p = (int)((g.rows_p + 255) / 256), tiles_q = (int)((g.rows_q + kPairN - 1) / kPairN);
    const int tiles = tiles_p * tiles_q, pairs = gridDim.x / 2, first = blockIdx.x / 2;
    volatile int *const stop = &sm.abort_flag;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kPairStages; s++) {
            mbar_init(&sm.full[s], 1);
            mbar_init(&sm.empty[s], 2);   // both CTAs have used it
        }
        for (int b = 0; b < 2; b++) {
            mbar_init(&sm.acc_full[b], 1);
            mbar_init(&sm.acc_empty[b], kPairEpiWarps);
        }
        for (int s = 0; s < kPairScaleSlots; s++) {
            mbar_init(&sm.sc_full[s], 32);
            mbar_init(&sm.sc_empty[s], kPairEpiWarps);
        }
        mbar_init(&sm.drained, 1);
        sm.abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) tmem_alloc<512>(&sm.tmem_base);
    tc_fence_before();
    __syncthreads();
    cluster_sync();   // the peer's barriers are ready before anything arrives on them
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;

    if (warp < 4) {
        regs_fewer<56>();
        if (warp == 0 && lane == 0) {
            bool ok = true;
            uint32_t issued = 0;
            int s = 0;
            uint32_t use = 1;   // parity of the release that the stage's next use waits for
            for (int t = first; t < tiles && ok; t += pairs) {
                int tp, tq;
                pair_tile(t, tiles_p, tiles_q, tp, tq);
                const int p0 = tp * 256 + 128 * rank, q0 = tq * kPairN + 128 * rank;
                for (int kb = 0; kb < kb_n; kb++) {
                    if (issued >= kPairStages && !mm_wait(&sm.empty[s], use, stop, g.status)) {
                        ok = false;
                        break;
                    }
                    uint8_t *st = sm.stage[s];
                    mbar_arrive_expect_tx(&sm.full[s], kPairStageBytes);
                    tma_load_tile(st, &map_p, kb * kMmBlock, p0, &sm.full[s]);
                    tma_load_tile_multicast(st + (128 + 128 * rank) * kMmBlock, &map_q, kb * kMmBlock, q0, &sm.full[s], 3);
                    issued++;
                    if (++s == kPairStages) {
                        s = 0;
                        use ^= 1;
                    }
                }
            }
            // every stage is released by both CTAs before this one may leave: the
            // peer's commits arrive here
            for (uint32_t j = issued > kPairStages ? issued - kPairStages : 0; ok && j < issued; j++)
                ok = mm_wait(&sm.empty[j % kPairStages], (j / kPairStages) & 1, stop, g.status);
            if (!ok)   // copies in flight land before shared memory goes away
                for (uint32_t j = issued > kPairStages ? issued - kPairStages : 0; j < issued; j++)
                    (void)mbar_wait_bounded(&sm.full[j % kPairStages], (j / kPairStages) & 1);
        } else if (warp == 1 && lane == 0) {
            int s = 0, buf = 0;
            uint32_t par = 0, acc_use = 1;
            bool ok = true, primed = false;   // primed: both buffers have been used
            for (int t = first; t < tiles && ok; t += pairs) {
                for (int kb = 0; kb < kb_n; kb++) {
                    if (!mm_wait(&sm.full[s], par, stop, g.status) ||
                        (primed && !mm_wait(&sm.acc_empty[buf], acc_use, stop, g.status))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t a = smem_desc_k128(sm.stage[s]);
                    const uint64_t b = smem_desc_k128(sm.stage[s] + 128 * kMmBlock);
#pragma unroll
                    for (int k = 0; k < kMmBlock / 32; k++)
                        mma_f8(tmem + buf * kPairN, a + 2 * k, b + 2 * k, idesc_e4m3(128, kPairN), k > 0);
                    mma_commit(&sm.acc_full[buf]);
                    mma_commit_multicast(&sm.empty[s], 3);
                    if (++s == kPairStages) {
                        s = 0;
                        par ^= 1;
                    }
                    buf ^= 1;
                    if (buf == 0) {
                        acc_use ^= 1;
                        primed = true;
                    }
                }
            }
            if (!ok) {   // MMAs in flight end before their memory goes away
                mma_commit(&sm.drained);
                (void)mbar_wait_bounded(&sm.drained, 0);
            }
        } else if (COLS && warp == 2) {
            // lane l fetches columns l, l + 32, ..: a block's scales are 256 words, 4 K/128 bytes apart
            int slot = 0;
            uint32_t use = 1;
            bool ok = true, primed = false;
            for (int t = first; t < tiles && ok; t += pairs) {
                int tp, tq;
                pair_tile(t, tiles_p, tiles_q, tp, tq);
                uint32_t src[kPairN / 32];   // words from s_q; K rows_q is below 2^39, so they fit
#pragma unroll
                for (int j = 0; j < kPairN / 32; j++) {
                    const int col = tq * kPairN + j * 32 + lane;
                    src[j] = (uint32_t)((col < rows_q ? col : 0) >> g.shift_q) * (uint32_t)kb_n;   // past the result: any scale
                }
                float v[kPairN / 32];
#pragma unroll
                for (int j = 0; j < kPairN / 32; j++) v[j] = __ldg(g.s_q + src[j]);
                for (int kb = 0; kb < kb_n; kb++) {
                    float next[kPairN / 32];
                    const int kn = kb + 1 < kb_n ? kb + 1 : kb;
#pragma unroll
                    for (int j = 0; j < kPairN / 32; j++) next[j] = __ldg(g.s_q + src[j] + kn);
                    const bool got = !primed || mm_wait(&sm.sc_empty[slot], use, stop, g.status);
                    if (!__all_sync(0xFFFFFFFFu, got)) {
                        ok = false;
                        break;
                    }
#pragma unroll
                    for (int j = 0; j < kPairN / 32; j++) {
                        sm.col_scale[slot][j * 32 + lane] = v[j];
                        v[j] = next[j];
                    }
                    mbar_arrive(&sm.sc_full[slot]);
                    if (++slot == kPairScaleSlots) {
                        slot = 0;
                        use ^= 1;
                        primed = true;
                    }
                }
            }
        }
    } else {
        regs_more<224>();
        const int quad = warp & 3, half = (warp - 4) >> 2;   // 32 tensor memory lanes, 128 columns
        const uint32_t acc_addr = tmem + ((uint32_t)(quad * 32) << 16) + half * 128;
        const bool vec = (kb_n & 3) == 0 && ((reinterpret_cast<uintptr_t>(g.s_p) | reinterpret_cast<uintptr_t>(g.s_q)) & 15) == 0;
        int buf = 0, slot = 0;
        uint32_t par = 0, sc_par = 0;
        bool ok = true;
        for (int t = first; t < tiles && ok; t += pairs) {
            int tp, tq;
            pair_tile(t, tiles_p, tiles_q, tp, tq);
            const int row0 = tp * 256 + 128 * rank + quad * 32, row = row0 + lane, col0 = tq * kPairN + half * 128;
            // rows and columns outside the result have zero products: any scale in bounds does
            const float *sp = g.s_p + (int64_t)((row < rows_p ? row : 0) >> g.shift_p) * kb_n;
            const float *sq = g.s_q + (int64_t)((col0 < rows_q ? col0 : 0) >> g.shift_q) * kb_n;
            uint64_t acc[64];
#pragma unroll
            for (int j = 0; j < 64; j++) acc[j] = 0ull;
            float sp_next[4], sq_next[4];
            load_scales4(sp_next, sp, 0, kb_n, vec);
            if (!COLS) load_scales4(sq_next, sq, 0, kb_n, vec);
            float s4[4];   // the scales of blocks kb .. kb | 3, the current one first
            for (int kb = 0; kb < kb_n; kb++) {
                if ((kb & 3) == 0) {
#pragma unroll
                    for (int i = 0; i < 4; i++) s4[i] = COLS ? sp_next[i] : sp_next[i] * sq_next[i];
                    load_scales4(sp_next, sp, kb + 4, kb_n, vec);   // used four blocks from here
                    if (!COLS) load_scales4(sq_next, sq, kb + 4, kb_n, vec);
                }
                bool got = mm_wait(&sm.acc_full[buf], par, stop, g.status);
                if (COLS) got = got && mm_wait(&sm.sc_full[slot], sc_par, stop, g.status);
                if (!__all_sync(0xFFFFFFFFu, got)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint64_t ss = pack2(__float_as_uint(s4[0]), __float_as_uint(s4[0]));
                s4[0] = s4[1];
                s4[1] = s4[2];
                s4[2] = s4[3];
                // the load of 16 columns runs while the 16 before it are added
                uint32_t r[2][16];
                tmem_ld16(r[0], acc_addr + buf * kPairN);
                tmem_wait_ld(r[0]);
#pragma unroll
                for (int h = 0; h < 8; h++) {
                    const uint32_t(&now)[16] = r[h & 1];
                    if (h < 7) {
                        tmem_ld16(r[(h + 1) & 1], acc_addr + buf * kPairN + (h + 1) * 16);
                    } else {   // all read: the next block may go there
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sm.acc_empty[buf]);
                    }
#pragma unroll
                    for (int j = 0; j < 8; j += 2) {
                        uint64_t v0 = pack2(now[2 * j], now[2 * j + 1]), v1 = pack2(now[2 * j + 2], now[2 * j + 3]);
                        if (COLS) {
                            const ulonglong2 cs = *reinterpret_cast<const ulonglong2 *>(&sm.col_scale[slot][half * 128 + h * 16 + 2 * j]);
                            v0 = fmul2(v0, cs.x);
                            v1 = fmul2(v1, cs.y);
                        }
                        acc[h * 8 + j] = ffma2(v0, ss, acc[h * 8 + j]);
                        acc[h * 8 + j + 1] = ffma2(v1, ss, acc[h * 8 + j + 1]);
                    }
                    if (h < 7) tmem_wait_ld(r[(h + 1) & 1]);
                }
                if (COLS) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.sc_empty[slot]);
                    if (++slot == kPairScaleSlots) {
                        slot = 0;
                        sc_par ^= 1;
                    }
                }
                buf ^= 1;
                if (buf == 0) par ^= 1;
            }
            if (ok) mm_store_rows<OUT>(g, &map_c, sm.staging[warp - 4], acc, row0, col0, lane);
        }
        if (lane == 0) bulk_wait_all();
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync();   // nothing of the peer's arrives here any more
    tc_fence_after();
    if (warp == 1) tmem_free<512>(tmem);
}

}  // namespace qk
