// The block-scaled product for results of many tiles.
//
// A pair of CTAs (a cluster of two) owns a 256 x 256 tile of C and walks the
// tiles persistently.  One MMA spans both: each CTA's shared memory holds its
// own 128 rows of P and half of Q's 256, and its tensor memory receives its
// 128 rows x 256 columns in FP32.  (With an MMA per CTA and Q multicast to
// both, a block's operands, 48 KiB written and 48 KiB read per CTA, take the
// 128 bytes a cycle of shared memory 768 cycles, and the MMAs 512.)  Two
// accumulator buffers together fill tensor memory.
//
// Warp 0 of each CTA loads its operand tiles, all of whose bytes count on the
// leader's barriers.  The leader's warps 1 and 2 issue the MMAs of the even and
// the odd blocks, warp 3 fetches scales, four blocks at a time, and the eight
// warps 4-11 keep the FP32 sums of 32 rows x 128 columns each in registers: a
// block's product is read from tensor memory, multiplied by its scales and
// added while the next block's runs.  Finished tiles go through shared memory
// to C as bulk tensor stores (adds, when accumulating in FP32), 32 rows x 128
// bytes each.
//
// The hand-over of the accumulator buffers is what the block rate hangs on:
// MMAs (512 cycles), commit (150 and more until a waiting warp sees it), read
// (about 350), release (some 400 more from the other CTA) and the next MMAs
// into the same buffer form a chain, of which two are in flight; measured, a
// block takes about 800 cycles, and a tile's end some 3000 more.  Inside a CTA
// the release is a named barrier (about 20 cycles from arrival to wake-up, an
// mbarrier takes 160 to 200); as a warp's barrier waits for its own commits
// too, each buffer has an MMA warp of its own.  The other CTA's warps arrive on
// the leader's mbarriers; its warps 1 and 2 wait at the named barriers only to
// say which scales are done with.  Tried and not faster: an MMA per CTA, a block
// in two MMAs of 128 columns with a chain each, sixteen epilogue warps, more
// stages, prefetches into L2, a look at the next block's barriers while one is
// added, the additions between a load of tensor memory and its wait.
//
// Measured on a GB300 in sustained runs, at its 1.4 kW: 16384 x 18432 x 7168
// 1.60 to 1.65 ms (2.6 to 2.7 PFLOP/s, clocks at 1.58 of 2.07 GHz), 8192 x
// 14336 x 4096 370 to 383 us (2.5), with 1x128 tiles of both and an FP32 C
// added to 14336 x 4096 x 8192 494 to 506 us (1.9 to 1.95; its FP32 multiplies
// and adds take 512 cycles of a block, the other's 256).
// Without the epilogue's work the loads and MMAs alone reach 3.1 PFLOP/s there.
//
// A named barrier cannot time out, and need not.  The epilogue warps arrive for
// every block of a tile, whether their own waits were served or given up, so
// without an abort each wait meets its nine arrivals.  After one the arrivals no
// longer go by blocks (a warp whose waits are given up runs ahead of the others,
// and may complete a barrier in their stead): the epilogue warps, which never
// wait there, then go on arriving until both MMA warps have left.  Sums read
// from a buffer that was released too early are not stored, as the flag is up.
#pragma once

#include "q_internal.h"
#include "q_mm.cuh"

namespace qk {

constexpr int kPairEpiWarps = 8;
constexpr int kPairThreads = 32 * (4 + kPairEpiWarps);
constexpr int kPairStages = 4;   // even: each MMA warp uses every other one
constexpr int kPairN = 256;       // columns of a pair's tile
constexpr int kPairStageBytes = 2 * 128 * kMmBlock;
constexpr int kPairScaleSlots = 4;   // a tile's first scales take a trip to memory: fetched 3 slots ahead
constexpr uint32_t kPairScaleBlocks = 4;   // a power of two
constexpr int kPairGroup = 8;     // tile rows per group of the tile order
// Named barriers of the accumulator buffers' release (two from kAccFree on):
// the epilogue's threads arrive, the MMA warp waits.
constexpr int kAccFree = 1, kAccThreads = 32 * (kPairEpiWarps + 1);
// Registers per thread of the epilogue's and the other warps; their sum is what
// the kernel is launched with.
constexpr int kPairEpiRegs = 200, kPairRegs = 104;

// (Constant barrier numbers: one held in a register claims all sixteen.)
QD void acc_release(int buf)
{
    if (buf == 0) named_barrier_arrive(kAccFree, kAccThreads);
    else named_barrier_arrive(kAccFree + 1, kAccThreads);
}
QD void acc_await(int buf)
{
    if (buf == 0) named_barrier(kAccFree, kAccThreads);
    else named_barrier(kAccFree + 1, kAccThreads);
}

struct PairSmem {
    uint8_t stage[kPairStages][kPairStageBytes];
    uint8_t staging[kPairEpiWarps][2 * 4096];
    // the blocks' scales: P's rows, and Q's rows (COLS) or two 128-row tiles
    float row_scale[kPairScaleSlots][kPairScaleBlocks][128];
    float col_scale[kPairScaleSlots][kPairScaleBlocks][kPairN];
    uint64_t full[kPairStages], empty[kPairStages], acc_full[2], peer_free[2], drained[2];
    uint64_t sc_full[kPairScaleSlots], sc_empty[kPairScaleSlots];
    uint32_t tmem_base;
    int abort_flag, issued, landed, left[2];   // left: the buffer's MMA warp waits no more
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

// The scales of all tiles of a CTA's walk (one warp), the next four blocks' on
// their way while four wait for a slot: four rows of P per lane, and eight rows
// of Q or, from lanes 0 and 1, those of Q's two 128-row tiles.  Rows outside the
// matrices have zero products: any scale does.
template <bool COLS>
QD void put_scales(PairSmem &sm, const MmArgs &g, int first, int pairs, int tiles_p, int tiles_q, int rank, int lane,
                   volatile int *stop)
{
    constexpr int NQ = COLS ? kPairN / 32 : 1;
    const int rows_p = (int)g.rows_p, rows_q = (int)g.rows_q, kb_n = (int)g.kblocks, tiles = tiles_p * tiles_q;
    float v[4][kPairScaleBlocks], w[NQ][kPairScaleBlocks];
    int t = first, kb = 0, tp, tq;
    auto load = [&] {
        const int row = tp * 256 + 128 * rank + lane, col = tq * kPairN + (COLS ? lane : 128 * (lane & 1));
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const int r = row + 32 * j < rows_p ? row + 32 * j : 0;
            load_scales4(v[j], g.s_p + (int64_t)(r >> g.shift_p) * kb_n, kb, kb_n);
        }
#pragma unroll
        for (int j = 0; j < NQ; j++) {
            const int c = col + 32 * j < rows_q ? col + 32 * j : 0;
            load_scales4(w[j], g.s_q + (int64_t)(c >> g.shift_q) * kb_n, kb, kb_n);
        }
    };
    if (t >= tiles) return;
    pair_tile(t, tiles_p, tiles_q, tp, tq);
    load();
    uint32_t slot = 0, par = 1;   // par: of the release that the slot's next use waits for
    bool primed = false;
    while (true) {
        const bool got = !primed || mm_wait(&sm.sc_empty[slot], par, stop, g.status);
        if (!__all_sync(0xFFFFFFFFu, got)) return;
#pragma unroll
        for (int i = 0; i < (int)kPairScaleBlocks; i++) {
#pragma unroll
            for (int j = 0; j < 4; j++) sm.row_scale[slot][i][32 * j + lane] = v[j][i];
            if (COLS) {
#pragma unroll
                for (int j = 0; j < NQ; j++) sm.col_scale[slot][i][32 * j + lane] = w[j][i];
            } else if (lane < 2) {
                sm.col_scale[slot][i][lane] = w[0][i];
            }
        }
        mbar_arrive(&sm.sc_full[slot]);
        if (++slot == kPairScaleSlots) {
            slot = 0;
            par ^= 1;
            primed = true;
        }
        kb += kPairScaleBlocks;
        if (kb >= kb_n) {
            kb = 0;
            t += pairs;
            if (t >= tiles) return;
            pair_tile(t, tiles_p, tiles_q, tp, tq);
        }
        load();
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
    const int tiles_p = (int)((g.rows_p + 255) / 256), tiles_q = (int)((g.rows_q + kPairN - 1) / kPairN);
    const int tiles = tiles_p * tiles_q, pairs = gridDim.x / 2, first = blockIdx.x / 2;
    volatile int *const stop = &sm.abort_flag;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kPairStages; s++) {
            mbar_init(&sm.full[s], 1);
            mbar_init(&sm.empty[s], 1);
        }
        for (int b = 0; b < 2; b++) {
            mbar_init(&sm.acc_full[b], 1);
            mbar_init(&sm.peer_free[b], kPairEpiWarps);   // the other CTA's
            mbar_init(&sm.drained[b], 1);
        }
        for (int s = 0; s < kPairScaleSlots; s++) {
            mbar_init(&sm.sc_full[s], 32);
            mbar_init(&sm.sc_empty[s], 1);
        }
        sm.abort_flag = g.give_up == 1;
        sm.issued = sm.landed = 0;
        sm.left[0] = sm.left[1] = 0;
        fence_mbar_init();
    }
    if (warp == 1) tmem_alloc_pair<512>(&sm.tmem_base);
    tc_fence_before();
    __syncthreads();
    cluster_sync();   // the peer's barriers are ready before anything arrives on them
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;
    // Launched while the kernel ahead still ran; nothing was read or written so far.
    griddep_wait();
    griddep_launch_dependents();

    if (warp < 4) {
        regs_fewer<kPairRegs>();
        if (warp == 0 && elect_one()) {
            bool ok = g.give_up < 3 || (int)rank != g.give_up - 3;
            if (!ok) *stop = 1;   // the test's loads that do not begin
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
                    if (rank == 0) mbar_arrive_expect_tx(&sm.full[s], 2 * kPairStageBytes);
                    const uint32_t bar = cluster_addr(smem_u32(&sm.full[s]), 0);
                    tma_load_tile_pair(st, &map_p, kb * kMmBlock, p0, bar);
                    tma_load_tile_pair(st + 128 * kMmBlock, &map_q, kb * kMmBlock, q0, bar);
                    issued++;
                    if (++s == kPairStages) {
                        s = 0;
                        use ^= 1;
                    }
                }
            }
            // every stage is released before this CTA may leave: the leader's commits
            // arrive here
            for (uint32_t j = issued > kPairStages ? issued - kPairStages : 0; ok && j < issued; j++)
                ok = mm_wait(&sm.empty[j % kPairStages], (j / kPairStages) & 1, stop, g.status);
            pair_loads_end<kPairStages>(ok, sm.full, issued, kPairStageBytes, &sm.issued, &sm.landed, &sm.abort_flag, rank);
        } else if (warp < 3 && warp > 0) {
            // One warp per accumulator buffer: every other block.
            const int buf = warp - 1;
            const uint32_t blocks = first < tiles ? (uint32_t)((tiles - 1 - first) / pairs + 1) * (uint32_t)kb_n : 0u;
            const uint64_t a0 = smem_desc_k128(sm.stage[0]), b0 = smem_desc_k128(sm.stage[0] + 128 * kMmBlock);
            const int groups = (kb_n + kPairScaleBlocks - 1) / kPairScaleBlocks;   // of scales, per tile
            int s = buf, kb_r = buf, group_r = 0;   // kb_r, group_r: of the block released next
            while (kb_r >= kb_n) {
                kb_r -= kb_n;
                group_r += groups;
            }
            uint32_t par = 0, freed = 0;
            if (g.give_up == 2 && rank == 0) *stop = 1;   // the test's wait that runs out
            for (uint32_t n = buf; n < blocks + 2; n += 2) {
                if (rank == 0) {
                    if (n >= blocks) break;
                    // a wait that gives up raises the flag, here or in the epilogue
                    mm_wait(&sm.full[s], par, stop, g.status);
                }
                if (__any_sync(0xFFFFFFFFu, *stop)) break;
                bool freed_too = true;   // by the other CTA; else its warps may still be reading the buffer
                if (n >= 2) {   // block n - 2 has been read, in both CTAs
                    acc_await(buf);
                    if (rank == 0) {
                        freed_too = mm_wait(&sm.peer_free[buf], freed, stop, g.status);
                        freed ^= 1;
                    }
                }
                tc_fence_after();
                if (elect_one()) {
                    if (rank == 0 && freed_too) {
                        const uint64_t at = (uint64_t)(s * (kPairStageBytes >> 4));
#pragma unroll
                        for (int k = 0; k < kMmBlock / 32; k++)
                            mma_f8_pair(tmem + buf * kPairN, a0 + at + 2 * k, b0 + at + 2 * k, idesc_e4m3(256, kPairN), k > 0);
                        mma_commit_pair(&sm.acc_full[buf]);
                        mma_commit_pair(&sm.empty[s]);
                    }
                    // block n - 2 was the last to use its group of scales
                    if (n >= 2 && (kb_r % kPairScaleBlocks == kPairScaleBlocks - 1 || kb_r + 1 == kb_n))
                        mbar_arrive(&sm.sc_empty[(group_r + kb_r / kPairScaleBlocks) % kPairScaleSlots]);
                }
                __syncwarp();
                if (n >= 2) {
                    kb_r += 2;
                    while (kb_r >= kb_n) {
                        kb_r -= kb_n;
                        group_r += groups;
                    }
                }
                s += 2;
                if (s >= kPairStages) {
                    s -= kPairStages;
                    par ^= 1;
                }
            }
            if (__any_sync(0xFFFFFFFFu, *stop) && rank == 0 && elect_one()) {   // MMAs in flight end before their memory goes away
                mma_commit_pair(&sm.drained[buf]);
                (void)mbar_wait_bounded(&sm.drained[buf], 0);
            }
            if (lane == 0) *static_cast<volatile int *>(&sm.left[buf]) = 1;
        } else if (warp == 3) {
            put_scales<COLS>(sm, g, first, pairs, tiles_p, tiles_q, (int)rank, lane, stop);
        }
    } else {
        regs_more<kPairEpiRegs>();
        const int quad = warp & 3, half = (warp - 4) >> 2;   // 32 tensor memory lanes, 128 columns
        const uint32_t acc_addr = tmem + ((uint32_t)(quad * 32) << 16) + half * 128;
        const uint32_t to_leader = cluster_addr(smem_u32(&sm.peer_free[0]), 0);
        auto release = [&](int buf) {   // all read: the next block may go there
            tc_fence_before();
            acc_release(buf);
            if (rank != 0 && elect_one()) mbar_arrive_cluster(to_leader + 8 * buf);
        };
        uint32_t n = 0;                   // block of this CTA's walk
        uint32_t ring = 0, sc_par = 0;    // its place among the slots' blocks, and the slots' fill
        for (int t = first; t < tiles && !__any_sync(0xFFFFFFFFu, *stop); t += pairs) {
            int tp, tq;
            pair_tile(t, tiles_p, tiles_q, tp, tq);
            uint64_t acc[64];
#pragma unroll
            for (int j = 0; j < 64; j++) acc[j] = 0ull;
            // After a wait that gave up the rest of the tile goes by as it is (a vote
            // per block cost 80 cycles of about 450); it is not stored then.
#pragma unroll 1
            for (int kb = 0; kb < kb_n; kb++, n++) {
                const int buf = n & 1;
                if (ring % kPairScaleBlocks == 0) mm_wait(&sm.sc_full[ring / kPairScaleBlocks], sc_par, stop, g.status);
                mm_wait(&sm.acc_full[buf], (n >> 1) & 1, stop, g.status);
                __syncwarp();
                tc_fence_after();
                const uint32_t addr = acc_addr + buf * kPairN;
                // A block's scales, which arrive under the first read of tensor memory: a
                // row's times its column tile's, or four rows'.  With column scales a
                // thread's 128 sums lie in 4 rows and 32 columns, so that it needs 32 of
                // them per block and not 128: shared memory returns 128 bytes a cycle to
                // the whole SM, and 128 took twice as long as the MMAs.
                const float *const rs = &sm.row_scale[0][0][quad * 32 + (COLS ? lane >> 2 : lane)] + ring * 128;
                const float *const cs = &sm.col_scale[0][0][COLS ? half * 128 + 2 * (lane & 3) : half] + ring * kPairN;
                uint64_t ss[COLS ? 4 : 1];
#pragma unroll
                for (int k = 0; k < (COLS ? 4 : 1); k++) {
                    const uint32_t s = __float_as_uint(COLS ? rs[8 * k] : rs[0] * cs[0]);
                    ss[k] = pack2(s, s);
                }
                if constexpr (!COLS) {
                    // two loads a block: eight of 16 columns waited for tensor memory as often
                    // (8192 x 14336 x 4096 393 us against 377)
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        uint32_t r[64];
                        tmem_ld64(r, addr + h * 64);
                        if (h == 1) release(buf);
#pragma unroll
                        for (int j = 0; j < 32; j++) acc[h * 32 + j] = ffma2(pack2(r[2 * j], r[2 * j + 1]), ss[0], acc[h * 32 + j]);
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < 4; c++) {
                        uint64_t cc[4];
#pragma unroll
                        for (int k = 0; k < 4; k++) cc[k] = *reinterpret_cast<const uint64_t *>(cs + c * 32 + k * 8);
#pragma unroll
                        for (int h = 0; h < 2; h++) {
                            uint32_t r[16];
                            tmem_ld_rows16(r, addr + c * 32 + ((uint32_t)(16 * h) << 16));
                            if (c == 3 && h == 1) release(buf);
#pragma unroll
                            for (int j = 0; j < 8; j++) {
                                const int a = c * 16 + h * 8 + j;
                                acc[a] = ffma2(fmul2(pack2(r[2 * j], r[2 * j + 1]), cc[j >> 1]), ss[2 * h + (j & 1)], acc[a]);
                            }
                        }
                    }
                }
                ring++;
                if (kb + 1 == kb_n) ring = (ring + kPairScaleBlocks - 1) & ~(kPairScaleBlocks - 1);   // a tile begins a slot
                if (ring == kPairScaleSlots * kPairScaleBlocks) {
                    ring = 0;
                    sc_par ^= 1;
                }
            }
            if (!__any_sync(0xFFFFFFFFu, *stop))
                mm_store_tile<OUT, !COLS>(g, &map_c, sm.staging[warp - 4], acc, tp * 256 + 128 * (int)rank + quad * 32,
                                          tq * kPairN + half * 128, lane);
        }
        if (__any_sync(0xFFFFFFFFu, *stop)) {   // nobody keeps an MMA warp waiting
            volatile int *const left = sm.left;
            while (__any_sync(0xFFFFFFFFu, left[0] == 0 || left[1] == 0)) {
                acc_release(0);
                acc_release(1);
            }
        }
        if (lane == 0) bulk_wait_all();
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync();   // nothing of the peer's arrives here any more
    tc_fence_after();
    if (warp == 1) tmem_free_pair<512>(tmem);
    if (g.give_up && threadIdx.x == 0 && g.status != nullptr) atomicOr(g.status, kStTimeout);
}

}  // namespace qk
