// The NVFP4 product for results of many tiles.
//
// A pair of CTAs (a cluster of two) owns a 256 x BN tile of C, BN 256 or, where such tiles would be too few for
// the machine, 128 (the rest here is about 256; two buffers of 128 columns do not overlap), and walks the
// tiles persistently; one MMA spans both, each CTA holding its own 128 rows of P
// and half of Q's 256 (as in k_mm_pair.cuh).  The tensor core applies the block
// scales, so a tile's whole sum is formed in tensor memory: 256 columns, and the
// scales of a stage take 48 of the 512.  Two tiles' columns overlap by 48, [0, 256)
// and [208, 464): the next tile's MMAs begin once the epilogue has read what they
// share, and run while the rest is read, scaled and stored.
//
// Warp 0 of each CTA loads its operand tiles, all of whose bytes count on the
// leader's barriers; the leader's warp 1 issues the copies of scales to tensor
// memory and the MMAs.  Warps 2 to 7 fetch scales: two each for P's 128 rows and
// the halves of Q's 256 (every CTA needs all of Q's; at 128 the last two have none), four blocks at a time (handed over two
// at a time, which made room for one stage more, 8192 x 14336 x 4096 took 188 us for 154).
// The eight warps 8-15 read 32 rows x 128 columns each when a tile is done.
//
// Measured on a GB300, in graphs of calls: 8192 x 14336 x 4096 to BF16 152 to 155 us
// (6.2 to 6.3 PFLOP/s), 8192 x 4096 x 14336 138 to 141 (6.8 to 7.0), 16384 x 18432 x 7168
// 615 to 660 (6.6 to 7.0), 14336 x 4096 x 8192 added to FP32 163 to 166 (5.8 to 5.9).  A tile
// of 8192 x 14336 x 4096 takes the MMA warp 12170 cycles, of which it waits 1690 for
// scales, then 1620 for operands (of 12346 cycles 3180 for operands and then 1070 for scales, where it waited for
// operands first: each hides part of the other) and 740 for the sums' place; at the nominal rate its MMAs
// take 8192.  The tensor pipe is active 69 % of the time (BF16, 4864 x 4096 x 8192).
// Called for seconds on end, 8192 x 14336 x 4096 takes 168 us: 1.35 kW, the power
// cap active, 1.78 GHz.  The scales' way: loaded and handed over stage by stage 260
// us, units of four blocks in slots of their own 212, without a release that waited
// for the loads 171; copies of four bytes straight to their places 560.
#pragma once

#include "q_internal.h"
#include "q_mm4.cuh"

namespace qk {

constexpr int kPair4EpiWarps = 8, kPair4ScaleWarps = 6;
constexpr int kPair4Threads = 32 * (2 + kPair4ScaleWarps + kPair4EpiWarps);
constexpr int kPair4Unit = 4, kPair4Slots = 2;   // blocks whose scales are handed over together (ScaleUnit), and places for them
// Registers per thread of the epilogue's and the other warps; their sum is what
// the kernel is launched with.
constexpr int kPair4EpiRegs = 152, kPair4Regs = 104;

// Operand stages are what shared memory goes to first: memory's queues are full, a stage's copies take some 2000 cycles and
// its MMAs 512 (8192 x 4096 x 14336 179 us at three stages, 146 at four, 142 at five).  A BF16 C is stored from registers
// and needs no staging to speak of; an FP32 C goes through staging as bulk stores and adds (adds from registers took 224
// us of 14336 x 4096 x 8192, bulk ones 174, both at four stages; with half the staging, pieces of 16 rows, and five 162, but K =
// 2048 103 for 101).  At BN 128 there is room for two pieces: 333 x 4096 x 4096 10.4 us, 11.3 with one.
template <int OUT, int BN> struct Pair4Smem {
    static constexpr int kBufs = BN == 128 ? 2 : 1, kStages = BN == 256 ? 5 : OUT == F32 ? 6 : 7, kStaging = OUT == F32 ? 2048 * kBufs : 1024;
    static constexpr int kAtomsQ = BN / 128, kOperandBytes = (128 + BN / 2) * 128, kScaleBytes = (1 + kAtomsQ) * kScaleAtom;
    static constexpr int kSecond = BN == 128 ? 128 : 208, kScales = kSecond + BN;   // first tensor memory columns of the second buffer, and of the scales
    static_assert(kScales + 16 * (1 + kAtomsQ) <= 512, "tensor memory");
    uint8_t stage[kStages][kOperandBytes];
    uint8_t staging[kPair4EpiWarps][kStaging];
    uint8_t scales[kPair4Slots][kPair4Unit][kScaleBytes];   // P's rows, and Q's in 128s
    uint64_t full[kStages], empty[kStages], sc_full[kPair4Slots], sc_empty[kPair4Slots], acc_full[2], acc_free, drained;
    uint32_t tmem_base;
    int abort_flag, issued, landed;
};
static_assert(sizeof(Pair4Smem<F32, 256>) <= 232448 && sizeof(Pair4Smem<BF16, 256>) <= 232448 && sizeof(Pair4Smem<F32, 128>) <= 232448 &&
              sizeof(Pair4Smem<BF16, 128>) <= 232448, "shared memory of a CTA");

// Tile t of the walk, in units of 256 x BN: groups of `group` tile rows, each
// walked column by column, so that the tiles in flight share their operands in
// L2.  The launcher says how many: where there are few tile rows, all of them, up
// to 32, where there are few columns, two (power is what these calls run into, and
// it goes by the traffic: 8192 x 14336 x 4096, 32 x 56 tiles, 160 us at 32 rows, 172
// at 8, 165 at one; 8192 x 4096 x 14336, 32 x 16, 161, 154 and 148, at two 148;
// 16384 x 18432 x 7168, 64 x 72, 647 at 32, 727 at 64, 679 at 8).
QD void pair4_tile(int t, int tiles_p, int tiles_q, int group, int &p, int &q)
{
    const int per_group = group * tiles_q;
    const int gp = t / per_group * group, r = t % per_group;
    const int height = tiles_p - gp < group ? tiles_p - gp : group;
    p = gp + r % height;
    q = r / height;
}

// The scales of 64 rows (half `part` of an atom) for all tiles of a CTA's walk, one warp.  Loads are issued
// behind the fence of the hand-over ahead, which would wait for them: among the operands'
// copies, which keep memory's queues full, a load takes some 4000 cycles.
template <bool WHOLE, int BN, class Smem>
QD void put_scales4(Smem &sm, const Mm4Args &a, int atom, int part, int first, int pairs, int tiles_p, int tiles_q, int rank,
                    int lane, volatile int *stop)
{
    const Mm4Scales &g = atom == 0 ? a.p : a.q;
    const int kb_n = (int)a.store.kblocks, tiles = tiles_p * tiles_q;
    const uint32_t bar = cluster_addr(smem_u32(&sm.sc_full[0]), 0);
    // places in the walk: of the four blocks that are loaded next, and of those that are handed over
    struct Place {
        int t, kb;
        int64_t row0;
    };
    auto settle = [&](Place &at) {
        int tp, tq;
        pair4_tile(at.t, tiles_p, tiles_q, a.group, tp, tq);
        at.row0 = (atom == 0 ? (int64_t)tp * 256 + 128 * rank : (int64_t)tq * BN + 128 * (atom - 1)) + 16 * part;
    };
    auto advance = [&](Place &at) {
        at.kb += kPair4Unit;
        if (at.kb >= kb_n) {
            at.kb = 0;
            at.t += pairs;
            if (at.t < tiles) settle(at);
        }
    };
    // Two loads of four blocks on their way, where registers allow.
    constexpr int kSets = WHOLE ? 2 : 1;
    ScaleUnit<WHOLE> held[kSets];
    if (first >= tiles) return;
    Place next = {first, 0, 0};
    settle(next);
    Place now = next;
    auto load = [&](ScaleUnit<WHOLE> &to) {
        if (next.t >= tiles) return;
        to.template load<4>(g, next.row0, next.kb, lane);
        advance(next);
    };
#pragma unroll
    for (int i = 0; i < kSets; i++) load(held[i]);
    for (uint32_t use = 0; now.t < tiles; use++) {
#pragma unroll
        for (uint32_t slot = 0; slot < kPair4Slots; slot++) {
            if (now.t >= tiles) return;
            const bool got = use == 0 || mm_wait(&sm.sc_empty[slot], (use & 1) ^ 1, stop, a.store.status);
            if (!__all_sync(0xFFFFFFFFu, got)) return;
            held[slot % kSets].template put<4>(g, now.row0, now.kb, sm.scales[slot][lane >> 3] + atom * kScaleAtom, 16 * part + (lane & 7), lane);
            fence_proxy_async();
            __syncwarp();
            // The copies that the leader's thread asks for read both CTAs' scales.  (8192 x 14336 x 4096 153 us; 167
            // where a release of all memory comes by way of a warp without loads, 213 from here.)
            if (lane == 0) mbar_arrive_shared_cluster(bar + 8 * slot);
            advance(now);
            load(held[slot % kSets]);
        }
    }
}

// One lane's row of 64 sums to a BF16 C (ADD: added to one), columns col on, as vectors of 32 bytes (16 where C's rows lie
// on 16-byte boundaries only; 8 columns lie in C or outside together).
template <bool ADD> QD void store_row64(const MmArgs &g, const uint64_t (&acc)[32], int64_t row, int64_t col, bool wide)
{
    if (row >= g.rows_p) return;
    uint16_t *const c = static_cast<uint16_t *>(g.c) + row * g.ldc + col;
    uint4 was[ADD ? 8 : 1];   // what is added to, all of it before the first store
    if constexpr (ADD) {
#pragma unroll
        for (int i = 0; i < 8; i++) was[i] = col + 8 * i < g.rows_q ? load_16(c + 8 * i) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int i = 0; i < 4; i++) {
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; j++) {
            float a, b;
            unpack2(acc[8 * i + j], a, b);
            if constexpr (ADD) {
                const uint4 &v = was[2 * i + j / 4];
                const uint32_t two = j % 4 == 0 ? v.x : j % 4 == 1 ? v.y : j % 4 == 2 ? v.z : v.w;
                a += __uint_as_float(two << 16);
                b += __uint_as_float(two & 0xFFFF0000u);
            }
            w[j] = bf16_pair(a, b);
        }
        const uint4 lo = make_uint4(w[0], w[1], w[2], w[3]), hi = make_uint4(w[4], w[5], w[6], w[7]);
        if (wide && col + 16 * i + 16 <= g.rows_q) {
            stg32(c + 16 * i, lo, hi);
        } else {
            if (col + 16 * i < g.rows_q) stg16(c + 16 * i, lo);
            if (col + 16 * i + 8 < g.rows_q) stg16(c + 16 * i + 8, hi);
        }
    }
}

// A warp's 32 rows x 64 sums to a BF16 C of any pitch (ADD: added to one), 8 columns at a time through 1 KiB of staging.
template <bool ADD> QD void store_any64(const MmArgs &g, float *staging, const uint64_t (&acc)[32], int64_t row0, int64_t col0, int lane)
{
#pragma unroll
    for (int p = 0; p < 8; p++) {
        // chunk i of row r at place i ^ (r / 4 % 2): a quarter of a warp's 16-byte accesses lie on all banks
        ulonglong2 *const to = reinterpret_cast<ulonglong2 *>(staging) + 2 * lane;
        const int odd = (lane >> 2) & 1;
        to[odd] = make_ulonglong2(acc[4 * p], acc[4 * p + 1]);
        to[odd ^ 1] = make_ulonglong2(acc[4 * p + 2], acc[4 * p + 3]);
        __syncwarp();
        const int64_t col = col0 + 8 * p + (lane & 7);
        float was[ADD ? 8 : 1];   // what is added to, all of it before the first store
        if constexpr (ADD) {
#pragma unroll
            for (int it = 0; it < 8; it++) {
                const int64_t row = row0 + 4 * it + (lane >> 3);
                was[it] = row < g.rows_p && col < g.rows_q ? load_bf16(static_cast<const uint16_t *>(g.c) + row * g.ldc + col) : 0.0f;
            }
        }
#pragma unroll
        for (int it = 0; it < 8; it++) {
            const int r = 4 * it + (lane >> 3), chunk = ((lane >> 2) & 1) ^ ((r >> 2) & 1);
            float v = staging[8 * r + 4 * chunk + (lane & 3)];
            if constexpr (ADD) v += was[it];
            if (row0 + r < g.rows_p && col < g.rows_q) static_cast<uint16_t *>(g.c)[(row0 + r) * g.ldc + col] = (uint16_t)bf16_bits(v);
        }
        __syncwarp();
    }
}

// A warp's 32 rows x 64 sums to an FP32 C, in pieces of 16 rows x 128 bytes through BUFS (one or two) times 2 KiB of staging, where 16-byte chunk i of
// row r is at place i ^ (r % 8), the 128-byte swizzle of the bulk stores.  (DIRECT: by the warp's lanes, a C of any pitch.)
template <int BUFS, bool DIRECT> QD void store_f32_64(const MmArgs &g, const CUtensorMap *map_c, uint8_t *const staging0, const uint64_t (&acc)[32], int64_t row0, int64_t col0, int lane)
{
#pragma unroll
    for (int p = 0; p < 4; p++) {
        const int64_t row = row0 + 16 * (p & 1), col = col0 + 32 * (p >> 1);
        uint8_t *const staging = staging0 + (p & (BUFS - 1)) * 2048;
        if (!DIRECT && lane == 0) {   // the last piece that was here has left it
            if constexpr (BUFS == 2) bulk_wait_read_but1();
            else bulk_wait_read_all();
        }
        __syncwarp();
        if ((lane >> 4) == (p & 1)) {
#pragma unroll
            for (int i = 0; i < 8; i++)
                *reinterpret_cast<ulonglong2 *>(staging + (lane & 15) * 128 + ((i ^ (lane & 7)) << 4)) =
                    make_ulonglong2(acc[(p >> 1) * 16 + 2 * i], acc[(p >> 1) * 16 + 2 * i + 1]);
        }
        if constexpr (!DIRECT) {
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
                if (row < g.rows_p && col < g.rows_q) {
                    if (g.store == kStoreBulkAdd) bulk_add_tile(map_c, staging, (int)col, (int)row);
                    else tma_store_tile(map_c, staging, (int)col, (int)row);
                }
                bulk_commit();   // an empty group too: the waits count them
            }
        } else {
            __syncwarp();
            float *const c = static_cast<float *>(g.c) + row * g.ldc + col + lane;
            const int rows = col + lane >= g.rows_q || row >= g.rows_p ? 0 : g.rows_p - row < 16 ? (int)(g.rows_p - row) : 16;
            float was[16];   // what is added to, all of it before the first store
#pragma unroll
            for (int r = 0; r < 16; r++) was[r] = g.accumulate && r < rows ? load_float(c + r * g.ldc) : 0.0f;
#pragma unroll
            for (int r = 0; r < 16; r++) {
                const float v = *reinterpret_cast<const float *>(staging + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4);
                if (r < rows) c[r * g.ldc] = g.accumulate ? was[r] + v : v;
            }
        }
    }
}

// What C is like: its rows are multiples of 16 bytes, and a BF16 one is overwritten; or (at BN 256) rows of any pitch; or a BF16
// C that is added to.  (Kernels of their own: the code for the others, though not reached, took 161 us of 8192 x 14336 x 4096
// where the kernel without it takes 154, and 49.6 us of 4096 x 4095 x 4096 for 47.6.  4096 x 4095 x 4096 added to: FP32 65 us, BF16
// 122, a BF16 C of 4096 columns 49.)
enum { kPlainC = 0, kAnyC = 1, kAddC = 2 };

template <int OUT, int BN, bool WHOLE, int KIND>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPair4Threads, 1)
k_mm4_pair(const __grid_constant__ CUtensorMap map_p, const __grid_constant__ CUtensorMap map_q,
           const __grid_constant__ CUtensorMap map_c, const Mm4Args a)
{
    const MmArgs &g = a.store;
    using Smem = Pair4Smem<OUT, BN>;
    constexpr int kStages = Smem::kStages, kAtomsQ = Smem::kAtomsQ;
    extern __shared__ __align__(1024) uint8_t dsm[];
    Smem &sm = *reinterpret_cast<Smem *>(dsm);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int kb_n = (int)g.kblocks;
    const int tiles_p = (int)((g.rows_p + 255) / 256), tiles_q = (int)((g.rows_q + BN - 1) / BN);
    const int tiles = tiles_p * tiles_q, pairs = gridDim.x / 2, first = blockIdx.x / 2;
    volatile int *const stop = &sm.abort_flag;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; s++) {
            mbar_init(&sm.full[s], 1);
            mbar_init(&sm.empty[s], 1);
        }
        for (int s = 0; s < kPair4Slots; s++) {
            mbar_init(&sm.sc_full[s], 2 * 2 * (1 + kAtomsQ));
            mbar_init(&sm.sc_empty[s], 1);
        }
        for (int b = 0; b < 2; b++) mbar_init(&sm.acc_full[b], 1);
        mbar_init(&sm.acc_free, 2 * kPair4EpiWarps);
        mbar_init(&sm.drained, 1);
        sm.abort_flag = g.give_up == 1;
        sm.issued = sm.landed = 0;
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

    if (warp < 2 + kPair4ScaleWarps) {
        regs_fewer<kPair4Regs>();
        if (warp == 0 && elect_one()) {
            bool ok = g.give_up < 3 || (int)rank != g.give_up - 3;
            if (!ok) *stop = 1;   // the test's loads that do not begin
            uint32_t issued = 0;
            int s = 0;
            uint32_t use = 1;   // parity of the release that the stage's next use waits for
            for (int t = first; t < tiles && ok; t += pairs) {
                int tp, tq;
                pair4_tile(t, tiles_p, tiles_q, a.group, tp, tq);
                const int p0 = tp * 256 + 128 * rank, q0 = tq * BN + BN / 2 * rank;
                for (int kb = 0; kb < kb_n; kb++) {
                    if (issued >= kStages && !mm_wait(&sm.empty[s], use, stop, g.status)) {
                        ok = false;
                        break;
                    }
                    uint8_t *st = sm.stage[s];
                    if (rank == 0) mbar_arrive_expect_tx(&sm.full[s], 2 * Smem::kOperandBytes);
                    const uint32_t bar = cluster_addr(smem_u32(&sm.full[s]), 0);
                    tma_load_tile_pair(st, &map_p, kb * 128, p0, bar);
                    tma_load_tile_pair(st + 128 * 128, &map_q, kb * 128, q0, bar);
                    issued++;
                    if (++s == kStages) {
                        s = 0;
                        use ^= 1;
                    }
                }
            }
            // every stage is released before this CTA may leave: the leader's commits
            // arrive here
            for (uint32_t j = issued > kStages ? issued - kStages : 0; ok && j < issued; j++)
                ok = mm_wait(&sm.empty[j % kStages], (j / kStages) & 1, stop, g.status);
            // and every slot of scales, whose last releases nobody else waits for
            const uint32_t units = ok ? issued / (uint32_t)kb_n * (uint32_t)((kb_n + kPair4Unit - 1) / kPair4Unit) : 0u;
            for (uint32_t u = units > kPair4Slots ? units - kPair4Slots : 0; ok && u < units; u++)
                ok = mm_wait(&sm.sc_empty[u % kPair4Slots], (u / kPair4Slots) & 1, stop, g.status);
            pair_loads_end<kStages>(ok, sm.full, issued, Smem::kOperandBytes, &sm.issued, &sm.landed, &sm.abort_flag, rank);
        } else if (warp == 1) {
            if (rank == 0) {
                const uint64_t a0 = smem_desc_k128(sm.stage[0]), b0 = smem_desc_k128(sm.stage[0] + 128 * 128);
                const uint64_t src0 = smem_desc_scales(sm.scales[0][0]);
                const uint32_t sp = tmem + Smem::kScales, sq = sp + 16;
                bool ok = g.give_up != 2;
                if (!ok) *stop = 1;   // the test's wait that runs out
                int s = 0;
                uint32_t par = 0, tile = 0, unit = 0;
                for (int t = first; t < tiles && ok; t += pairs, tile++) {
                    const uint32_t d = tmem + (tile & 1) * Smem::kSecond;
                    // the columns that this tile shares with the one before have been read
                    if (tile > 0) ok = mm_wait(&sm.acc_free, (tile - 1) & 1, stop, g.status);
                    for (int kb = 0; kb < kb_n; kb++) {
                        const uint32_t slot = unit % kPair4Slots;
                        // (scales first: the fence behind them runs while operands are on their way)
                        if (kb % kPair4Unit == 0) ok = ok && mm_wait<true>(&sm.sc_full[slot], (unit / kPair4Slots) & 1, stop, g.status);
                        ok = ok && mm_wait(&sm.full[s], par, stop, g.status);
                        ok = __all_sync(0xFFFFFFFFu, ok);
                        if (!ok) break;
                        tc_fence_after();
                        if (elect_one()) {
                            const uint64_t at = (uint64_t)(s * (Smem::kOperandBytes >> 4));
                            const uint64_t src = src0 + (uint64_t)((slot * kPair4Unit + kb % kPair4Unit) * (Smem::kScaleBytes >> 4));
#pragma unroll
                            for (int k = 0; k < 4; k++) {
                                scales_to_tmem_pair(sp + 4 * k, src + 32 * k);
#pragma unroll
                                for (int j = 0; j < kAtomsQ; j++) scales_to_tmem_pair(sq + 4 * (k * kAtomsQ + j), src + 128 * (1 + j) + 32 * k);
                            }
#pragma unroll
                            for (int k = 0; k < 4; k++)
                                mma_f4_pair(d, a0 + at + 2 * k, b0 + at + 2 * k, idesc_e2m1(256, BN), sp + 4 * k, sq + 4 * kAtomsQ * k, kb > 0 || k > 0);
                            mma_commit_pair(&sm.empty[s]);
                            if (kb % kPair4Unit == kPair4Unit - 1 || kb + 1 == kb_n) mma_commit_pair(&sm.sc_empty[slot]);
                            if (kb + 1 == kb_n) mma_commit_pair(&sm.acc_full[tile & 1]);
                        }
                        __syncwarp();
                        if (kb % kPair4Unit == kPair4Unit - 1 || kb + 1 == kb_n) unit++;
                        if (++s == kStages) {
                            s = 0;
                            par ^= 1;
                        }
                    }
                }
                if (__any_sync(0xFFFFFFFFu, !ok || *stop) && elect_one()) {   // aborted: MMAs in flight end before their memory goes away
                    mma_commit_pair(&sm.drained);
                    (void)mbar_wait_bounded(&sm.drained, 0);
                }
            }
        } else if (warp >= 2) {
            const int w = warp - 2, atom = w >> 1;
            if (atom <= kAtomsQ) put_scales4<WHOLE, BN>(sm, a, atom, w & 1, first, pairs, tiles_p, tiles_q, (int)rank, lane, stop);
        }
    } else {
        regs_more<kPair4EpiRegs>();
        const int quad = warp & 3, half = (warp - 2 - kPair4ScaleWarps) >> 2;   // 32 tensor memory lanes, half the columns
        const uint32_t to_leader = cluster_addr(smem_u32(&sm.acc_free), 0);
        const float fp = load_float(a.s_p), fq = load_float(a.s_q);
        const uint64_t sp = pack2(__float_as_uint(fp), __float_as_uint(fp)), sq = pack2(__float_as_uint(fq), __float_as_uint(fq));
        const bool wide = ((reinterpret_cast<uintptr_t>(g.c) | (uintptr_t)(2 * g.ldc)) & 31) == 0;   // of a BF16 C
        uint32_t tile = 0;
        for (int t = first; t < tiles && !__any_sync(0xFFFFFFFFu, *stop); t += pairs, tile++) {
            int tp, tq;
            pair4_tile(t, tiles_p, tiles_q, a.group, tp, tq);
            mm_wait(&sm.acc_full[tile & 1], (tile >> 1) & 1, stop, g.status);
            __syncwarp();
            tc_fence_after();
            const uint32_t addr = tmem + ((uint32_t)(quad * 32) << 16) + (tile & 1) * Smem::kSecond + half * (BN / 2);
            // (BN 256) The columns shared with the next tile are the last 48 of the second half, then
            // the first 48 of the first: each half begins at its end of the tile.
            auto part = [&](int h, bool shared) {
                uint32_t r[64];
                tmem_ld64(r, addr + h * 64);
                if (shared) {
                    tc_fence_before();
                    if (elect_one()) mbar_arrive_cluster(to_leader);
                }
                uint64_t acc[32];
#pragma unroll
                for (int j = 0; j < 32; j++) acc[j] = fmul2(fmul2(pack2(r[2 * j], r[2 * j + 1]), sp), sq);
                if (__any_sync(0xFFFFFFFFu, *stop)) return;
                const int64_t row = (int64_t)tp * 256 + 128 * (int)rank + quad * 32, col = (int64_t)tq * BN + half * (BN / 2) + h * 64;
                uint8_t *const staging = sm.staging[warp - 2 - kPair4ScaleWarps];
                if constexpr (OUT == BF16 && KIND == kAddC) {
                    if (g.ldc % 8 == 0) store_row64<true>(g, acc, row + lane, col, wide);
                    else store_any64<true>(g, reinterpret_cast<float *>(staging), acc, row, col, lane);
                } else if constexpr (OUT == BF16 && KIND == kAnyC) store_any64<false>(g, reinterpret_cast<float *>(staging), acc, row, col, lane);
                else if constexpr (OUT == BF16) store_row64<false>(g, acc, row + lane, col, wide);
                else store_f32_64<Smem::kBufs, KIND == kAnyC>(g, &map_c, staging, acc, row, col, lane);
            };
            if constexpr (BN == 256) {
                part(half, true);
                part(1 - half, false);
            } else {
                part(0, true);
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
