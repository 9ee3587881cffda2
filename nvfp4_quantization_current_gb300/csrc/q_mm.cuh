// What the kernels of the block-scaled product share: their arguments, bounded
// waits that end when the CTA aborts, and the way out of the accumulators.
#pragma once

#include "q_tcgen05.cuh"

namespace qk {

constexpr int kMmBlock = 128;   // elements of K per scale, and bytes per operand row of a stage

// How finished sums reach C.
enum MmStore { kStoreDirect = 0, kStoreBulk = 1, kStoreBulkAdd = 2 };

// C = P Q^T: P's rows lie on tensor memory lanes, Q's rows on its columns.
struct MmArgs {
    const float *s_p, *s_q;
    int64_t rows_p, rows_q, kblocks;
    int shift_p, shift_q;       // row -> scale row: 0 for 1x128 tiles, 7 for 128x128
    void *c;
    int64_t ldc;
    int32_t *status;
    bool accumulate;
    int store;
    // For a test, of every cluster: 1 a wait has run out (in the split kernel's first CTA, in both of a pair), 2 the MMAs'
    // first one does, 3 and 4 the loads of a pair's first or second CTA never begin (the split kernel: as 1).
    int give_up;
};

// Waits for a phase of `bar`; false when the CTA's abort flag is up or the
// wait ran out (which raises it and reports the timeout).  The hardware wakes
// the warp: polling sees the phase some 130 cycles sooner, but the polls' power
// costs the large products 2 to 3%.
// SHARED: for what other CTAs of the cluster have put into their shared memory (mbar_arrive_shared_cluster).
template <bool SHARED = false> QD bool mm_wait(uint64_t *bar, uint32_t parity, volatile int *abort_flag, int32_t *status)
{
    unsigned long long t0 = 0;
    for (uint32_t n = 1;; n++) {
        if (SHARED ? mbar_try_wait_relaxed_cluster(bar, parity) : mbar_try_wait(bar, parity)) {
            if constexpr (SHARED) shared_acquire_cluster();
            return true;
        }
        if (n % 1024 == 0) {   // the timer and the flag are off the way of the waits that are served
            if (*abort_flag) return false;
            const unsigned long long now = globaltimer();
            if (t0 == 0) t0 = now;
            if (now - t0 > kWaitNs) {
                *abort_flag = 1;
                if (status != nullptr) atomicOr(status, kStTimeout);
                return false;
            }
        }
    }
}

// Four consecutive block scales from kb on, the last one repeated past the end.
QD void load_scales4(float (&s)[4], const float *row, int kb, int kb_n)
{
    if (((kb_n | kb) & 3) == 0 && (reinterpret_cast<uintptr_t>(row) & 15) == 0) {   // kb + 3 exists
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

template <int OUT> struct OutT;
template <> struct OutT<BF16> { using T = uint16_t; };
template <> struct OutT<F32> { using T = float; };

template <int OUT> QD void put_one(typename OutT<OUT>::T *p, float v, bool accumulate)
{
    if constexpr (OUT == F32) {
        *p = accumulate ? *p + v : v;
    } else {
        *p = (uint16_t)bf16_bits(accumulate ? __uint_as_float((uint32_t)*p << 16) + v : v);
    }
}

// The end of the loads of a pair's CTA (one thread), `n` stages of `part` bytes; ok: every one of them has been read.  If not,
// the copies in flight land here, before shared memory goes away.  Those of both CTAs count on the leader's barriers, so
// the leader waits for them (bounded), and its peer for the leader's word.  Uses of a stage that one CTA has issued and
// the other has not would never complete: the leader leaves out what is missing.  (Neither can be more than STAGES ahead.)
// Where the MMAs end early, the loads of both CTAs do: each waits for its stages' releases.  `issued`, `landed`: words of
// shared memory, zero so far.
template <int STAGES>
QD void pair_loads_end(bool ok, uint64_t *full, uint32_t n, uint32_t part, int *issued, int *landed, int *abort_flag, uint32_t rank)
{
    *static_cast<volatile int *>(issued) = (int)n + 1;
    const int other = (int)rank ^ 1;
    if (!ok) {
        st_cluster1(cluster_addr(smem_u32(abort_flag), other), 1);   // the peer need not wait its time out
        const unsigned long long t0 = globaltimer();
        if (rank == 0) {
            uint32_t peer;
            while ((peer = (uint32_t)ld_cluster1(cluster_addr(smem_u32(issued), other))) == 0 && globaltimer() - t0 < 2 * kWaitNs) {}
            peer = peer == 0 ? n : peer - 1;
            const uint32_t most = n > peer ? n : peer;
            for (uint32_t j = most > STAGES ? most - STAGES : 0; j < most; j++) {
                uint64_t *const bar = &full[j % STAGES];
                if (j >= n) mbar_arrive_expect_tx(bar, part);
                if (j >= peer) mbar_complete_tx(bar, part);
                (void)mbar_wait_bounded(bar, (j / STAGES) & 1);
            }
        } else {
            while (*static_cast<volatile int *>(landed) == 0 && globaltimer() - t0 < (STAGES + 3) * kWaitNs) {}
        }
    }
    if (rank == 0) st_cluster1(cluster_addr(smem_u32(landed), other), 1);
}

QD void bulk_add_tile(const CUtensorMap *map, const void *src, int x, int y)
{
    asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2}], [%3];"
                 ::"l"(map), "r"(x), "r"(y), "r"(smem_u32(src)) : "memory");
}

// One warp's sums, 32 rows (from row0) x 128 columns (from col0), to C in
// pieces of 32 rows x 128 bytes through its two 4 KiB staging buffers: the
// 16-byte chunk i of row r at place i ^ (r % 8), which is the 128-byte swizzle
// of the bulk store and keeps the lanes' accesses off each other's banks.
// Rows and columns outside C are cut off by the store.  C's whose rows are no
// multiple of 16 bytes, and sums onto a BF16 C, are written by the lanes
// themselves, one row at a time, from FP32 staging (so that a sum is rounded
// once).
//
// ROWS: thread t holds row t, acc[j] columns 2j and 2j + 1.  Otherwise
// acc[16c + 8h + 2i + k] is row 16h + 8k + t / 4, columns 32c + 8i + 2 (t % 4)
// and the next (tmem_ld_rows16).
template <int OUT, bool ROWS>
QD void mm_store_tile(const MmArgs &g, const CUtensorMap *map_c, uint8_t *staging, const uint64_t (&acc)[64], int64_t row0,
                      int64_t col0, int lane)
{
    using T = typename OutT<OUT>::T;
    const bool bulk = g.store != kStoreDirect;
    auto place = [&](uint8_t *buf, int r, int i) { return buf + r * 128 + ((i ^ (r & 7)) << 4); };
    auto claim = [&](int piece) {   // the piece before the last one has left this buffer
        if (bulk && lane == 0) bulk_wait_read_but1();
        __syncwarp();
        return staging + (piece & 1) * 4096;
    };
    auto send = [&](const uint8_t *buf, int64_t col) {
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
            if (row0 < g.rows_p && col < g.rows_q) {
                if (g.store == kStoreBulkAdd) bulk_add_tile(map_c, buf, (int)col, (int)row0);
                else tma_store_tile(map_c, buf, (int)col, (int)row0);
            }
            bulk_commit();   // an empty group too, for claim() counts them
        }
    };
    if (OUT == BF16 && bulk) {
#pragma unroll
        for (int p = 0; p < 2; p++) {
            uint8_t *buf = claim(p);
            if constexpr (ROWS) {
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    uint32_t w[4];
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        float a, b;
                        unpack2(acc[p * 32 + i * 4 + j], a, b);
                        w[j] = bf16_pair(a, b);
                    }
                    *reinterpret_cast<uint4 *>(place(buf, lane, i)) = make_uint4(w[0], w[1], w[2], w[3]);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 32; j++) {
                    const int c = j >> 4, h = (j >> 3) & 1, i = (j >> 1) & 3, k = j & 1;
                    float a, b;
                    unpack2(acc[p * 32 + j], a, b);
                    *reinterpret_cast<uint32_t *>(place(buf, 16 * h + 8 * k + (lane >> 2), 4 * c + i) + 4 * (lane & 3)) = bf16_pair(a, b);
                }
            }
            send(buf, col0 + p * 64);
        }
        return;
    }
#pragma unroll
    for (int p = 0; p < 4; p++) {
        uint8_t *buf = claim(p);
        if constexpr (ROWS) {
#pragma unroll
            for (int i = 0; i < 8; i++)
                *reinterpret_cast<ulonglong2 *>(place(buf, lane, i)) = make_ulonglong2(acc[p * 16 + i * 2], acc[p * 16 + i * 2 + 1]);
        } else {
#pragma unroll
            for (int j = 0; j < 16; j++) {
                const int h = j >> 3, i = (j >> 1) & 3, k = j & 1;
                *reinterpret_cast<uint64_t *>(place(buf, 16 * h + 8 * k + (lane >> 2), 2 * i + ((lane & 3) >> 1)) + 8 * (lane & 1)) = acc[p * 16 + j];
            }
        }
        if (bulk) {
            send(buf, col0 + p * 32);
        } else {
            __syncwarp();
            const int64_t col = col0 + p * 32 + lane;
            for (int r = 0; r < 32 && row0 + r < g.rows_p; r++)
                if (col < g.rows_q)
                    put_one<OUT>(static_cast<T *>(g.c) + (row0 + r) * g.ldc + col,
                                 *reinterpret_cast<const float *>(place(buf, r, lane >> 2) + (lane & 3) * 4), g.accumulate);
        }
    }
}

}  // namespace qk
