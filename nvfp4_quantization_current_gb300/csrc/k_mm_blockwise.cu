// Block-scaled FP8 matrix product: the consumer of the blockwise copies.
//
//   C[m, n] (+)= sum_kb s_a[m, kb] s_b[n, kb] P_kb[m, n],
//   P_kb[m, n] = sum of a[m, k] b[n, k] over the 128 elements k of block kb
//
// with a [M, K] and b [N, K] E4M3 codes, K contiguous, and one FP32 scale per
// 1x128 or 128x128 tile of each ("Mixed-precision training: fp16 to fp8",
// "Blockwise scaling": forward X W^T, input gradient dY W, weight gradient
// dY^T X, each from the copy whose blocks run along the reduction).
//
// The scales change every 128 elements of K and are no powers of two, so the
// tensor core cannot carry the sum over blocks: each block's product P_kb goes
// to tensor memory in FP32 and is added, times its two scales, to FP32
// accumulators in registers.  The FP8 products are exact in FP32; a result is
// rounded once more, to the output type.
//
// A CTA owns a 128 x 128 tile of C.  Warp 4 streams operand tiles (128 rows x
// 128 bytes each, TMA into the 128-byte swizzle, kStages in flight), one
// thread of warp 5 issues the MMAs of a block into one of two accumulator
// buffers, and warps 0-3 (one thread per row) scale and add the other.
//
// Every wait is bounded; a role that gives up reports Q_ST_TIMEOUT, raises the
// CTA's abort flag, which ends the other roles' waits, and the copies and MMAs
// in flight are waited for (bounded again) before shared and tensor memory go
// away.
#include "k_mm_pair.cuh"
#include "q_internal.h"
#include "q_mm.cuh"

namespace qk {

namespace {

constexpr int kMmThreads = 192, kMmStages = 6, kMmN = 128;
constexpr int kMmStageBytes = (128 + kMmN) * kMmBlock;
constexpr int kMmSmem = kMmStages * kMmStageBytes + 1024;

template <int OUT>
__global__ void __launch_bounds__(kMmThreads, 1)
k_mm_blockwise(const __grid_constant__ CUtensorMap map_p, const __grid_constant__ CUtensorMap map_q, const MmArgs g)
{
    extern __shared__ __align__(1024) uint8_t dsm[];
    __shared__ __align__(8) uint64_t full[kMmStages], empty[kMmStages], acc_full[2], acc_empty[2], drained;
    __shared__ __align__(16) float col_scale[2][kMmN];
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag;
    uint8_t *stages = dsm + ((1024u - (smem_u32(dsm) & 1023u)) & 1023u);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t p0 = (int64_t)blockIdx.x * 128, q0 = (int64_t)blockIdx.y * kMmN;
    const int kb_n = (int)g.kblocks;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kMmStages; s++) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; b++) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], 128);
        }
        mbar_init(&drained, 1);
        abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 5) tmem_alloc<2 * kMmN>(&tmem_base);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base;
    volatile int *const stop = &abort_flag;

    if (warp == 4) {
        if (lane == 0) {
            int kb = 0;
            for (; kb < kb_n; kb++) {
                const int s = kb % kMmStages;
                if (kb >= kMmStages && !mm_wait(&empty[s], ((kb / kMmStages) & 1) ^ 1, stop, g.status)) break;
                uint8_t *st = stages + s * kMmStageBytes;
                mbar_arrive_expect_tx(&full[s], kMmStageBytes);
                tma_load_tile(st, &map_p, kb * kMmBlock, (int)p0, &full[s]);
                tma_load_tile(st + 128 * kMmBlock, &map_q, kb * kMmBlock, (int)q0, &full[s]);
            }
            if (kb < kb_n)   // aborted: the copies in flight land before shared memory goes away
                for (int j = kb > kMmStages ? kb - kMmStages : 0; j < kb; j++)
                    (void)mbar_wait_bounded(&full[j % kMmStages], (j / kMmStages) & 1);
        }
    } else if (warp == 5) {
        if (lane == 0) {
            int kb = 0;
            for (; kb < kb_n; kb++) {
                const int s = kb % kMmStages, buf = kb & 1;
                if (kb >= 2 && !mm_wait(&acc_empty[buf], ((kb >> 1) & 1) ^ 1, stop, g.status)) break;
                if (!mm_wait(&full[s], (kb / kMmStages) & 1, stop, g.status)) break;
                tc_fence_after();
                const uint64_t a = smem_desc_k128(stages + s * kMmStageBytes);
                const uint64_t b = smem_desc_k128(stages + s * kMmStageBytes + 128 * kMmBlock);
#pragma unroll
                for (int k = 0; k < kMmBlock / 32; k++)
                    mma_f8(tmem + buf * kMmN, a + 2 * k, b + 2 * k, idesc_e4m3(128, kMmN), k > 0);
                mma_commit(&empty[s]);
                mma_commit(&acc_full[buf]);
            }
            if (kb < kb_n) {   // aborted: the MMAs in flight end before their memory goes away
                mma_commit(&drained);
                (void)mbar_wait_bounded(&drained, 0);
            }
        }
    } else {
        const int64_t row = p0 + threadIdx.x;
        const bool live = row < g.rows_p;
        const float *sp = g.s_p + ((live ? row : 0) >> g.shift_p) * g.kblocks;
        const int64_t col = q0 + threadIdx.x;   // the column whose scale this thread fetches
        const bool col_live = col < g.rows_q;
        const float *sq = g.s_q + ((col_live ? col : 0) >> g.shift_q) * g.kblocks;
        float acc[kMmN];
#pragma unroll
        for (int j = 0; j < kMmN; j++) acc[j] = 0.0f;
        for (int kb = 0; kb < kb_n; kb++) {
            const int buf = kb & 1;
            const float srow = sp[kb];
            col_scale[buf][threadIdx.x] = col_live ? sq[kb] : 0.0f;
            named_barrier(1, 128);   // also: every thread is done with this buffer's previous scales
            bool ok = mm_wait(&acc_full[buf], (kb >> 1) & 1, stop, g.status);
            if (!__all_sync(0xFFFFFFFFu, ok)) ok = false;
            if (ok) {
                tc_fence_after();
#pragma unroll
                for (int h = 0; h < kMmN / 32; h++) {
                    uint32_t r[32];
                    tmem_ld32(r, tmem + ((uint32_t)(warp * 32) << 16) + buf * kMmN + h * 32);
#pragma unroll
                    for (int j = 0; j < 32; j++)
                        acc[h * 32 + j] = __fmaf_rn(__uint_as_float(r[j]) * col_scale[buf][h * 32 + j], srow, acc[h * 32 + j]);
                }
                tc_fence_before();
            }
            mbar_arrive(&acc_empty[buf]);
        }
        if (live) {
            using T = typename OutT<OUT>::T;
            T *out = static_cast<T *>(g.c) + row * g.ldc + q0;
#pragma unroll
            for (int j = 0; j < kMmN; j++)
                if (q0 + j < g.rows_q) put_one<OUT>(out + j, acc[j], g.accumulate);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 5) tmem_free<2 * kMmN>(tmem);
}

// Tiles of 128 x 128, one per CTA.
template <int OUT>
cudaError_t mm_one(const uint8_t *p, const uint8_t *q, const MmArgs &g, cudaStream_t st)
{
    alignas(64) CUtensorMap map_p, map_q;
    const int64_t K = g.kblocks * kMmBlock;
    cudaError_t e = make_operand_map(&map_p, p, g.rows_p, K, 128);
    if (e == cudaSuccess) e = make_operand_map(&map_q, q, g.rows_q, K, kMmN);
    if (e == cudaSuccess) e = engine_smem_ready<k_mm_blockwise<OUT>>(kMmSmem);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)((g.rows_p + 127) / 128), (unsigned)((g.rows_q + kMmN - 1) / kMmN));
    k_mm_blockwise<OUT><<<grid, kMmThreads, kMmSmem, st>>>(map_p, map_q, g);
    return cudaGetLastError();
}

// Tiles of 256 x 256 on CTA pairs.
template <int OUT, bool COLS>
cudaError_t mm_pair(const uint8_t *p, const uint8_t *q, MmArgs g, cudaStream_t st)
{
    alignas(64) CUtensorMap map_p, map_q, map_c = {};
    const int64_t K = g.kblocks * kMmBlock;
    cudaError_t e = make_operand_map(&map_p, p, g.rows_p, K, 128);
    if (e == cudaSuccess) e = make_operand_map(&map_q, q, g.rows_q, K, 128);
    const bool bulk = g.ldc % (OUT == F32 ? 4 : 8) == 0 && (OUT == F32 || !g.accumulate);
    g.store = !bulk ? kStoreDirect : g.accumulate ? kStoreBulkAdd : kStoreBulk;
    if (e == cudaSuccess && bulk) e = make_result_map(&map_c, g.c, OUT, g.rows_p, g.rows_q);
    if (e == cudaSuccess) e = engine_smem_ready<k_mm_pair<OUT, COLS>>(sizeof(PairSmem));
    if (e == cudaSuccess) {   // the epilogue's registers have to be there to be moved: it would wait for them forever
        static const cudaError_t enough = [] {
            cudaFuncAttributes a;
            const cudaError_t ea = cudaFuncGetAttributes(&a, k_mm_pair<OUT, COLS>);
            if (ea != cudaSuccess) return ea;
            return a.numRegs * kPairThreads >= 32 * (kPairEpiWarps * kPairEpiRegs + 4 * kPairRegs) ? cudaSuccess : cudaErrorInvalidConfiguration;
        }();
        e = enough;
    }
    if (e != cudaSuccess) return e;
    const int64_t tiles = ((g.rows_p + 255) / 256) * ((g.rows_q + kPairN - 1) / kPairN);
    if (tiles > INT32_MAX) return cudaErrorInvalidValue;
    const int64_t pairs = sm_count() / 2;
    k_mm_pair<OUT, COLS><<<(unsigned)(2 * (tiles < pairs ? tiles : pairs)), kPairThreads, sizeof(PairSmem), st>>>(map_p, map_q, map_c, g);
    return cudaGetLastError();
}

template <int OUT>
cudaError_t mm_t(const uint8_t *p, const uint8_t *q, const MmArgs &g, cudaStream_t st)
{
    if (g.rows_p > 512)
        return g.shift_q ? mm_pair<OUT, false>(p, q, g, st) : mm_pair<OUT, true>(p, q, g, st);
    return mm_one<OUT>(p, q, g, st);
}

}  // namespace

cudaError_t launch_mm_blockwise(const uint8_t *a, const float *s_a, int tile_a, const uint8_t *b, const float *s_b, int tile_b,
                                int64_t M, int64_t N, int64_t K, void *c, int out, bool accumulate, int32_t *status,
                                cudaStream_t st)
{
    MmArgs g = {s_a, s_b, M, N, K / kMmBlock, tile_a ? 7 : 0, tile_b ? 7 : 0, c, N, status, accumulate, kStoreDirect};
    return out == BF16 ? mm_t<BF16>(a, b, g, st) : mm_t<F32>(a, b, g, st);
}

}  // namespace qk
