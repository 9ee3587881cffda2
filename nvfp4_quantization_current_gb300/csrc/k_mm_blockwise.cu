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
// Two kernels: k_mm_pair.cuh for results of many tiles, k_mm_split.cuh for few
// tokens and for results of few tiles.  In both, one warp streams operand tiles
// (128 bytes of each row per stage, TMA into the 128-byte swizzle), one thread
// issues a block's MMAs into one of several accumulator buffers, and other
// warps scale and add the buffers that are done.
//
// Waits on mbarriers are bounded; a role that gives up reports Q_ST_TIMEOUT,
// raises the CTA's abort flag, which ends the other roles' waits, and the copies
// and MMAs in flight are waited for (bounded again) before shared and tensor
// memory go away.  The other waits end because who they wait for does: cluster
// barriers and __syncthreads come where every role has ended, tensor memory is
// allocated when the CTA ahead on the SM, which waits for nothing of this one,
// frees its own, and the named barriers are told of where they are used.
#include "k_mm_pair.cuh"
#include "k_mm_split.cuh"
#include "q_internal.h"
#include "q_mm.cuh"

namespace qk {

namespace {

// Tiles of 128 weights x BN tokens, the reduction of each split over a cluster.
template <int OUT, int BN, bool TILES>
cudaError_t mm_split_t(const uint8_t *p, const uint8_t *q, const MmArgs &g, int split, cudaStream_t st)
{
    alignas(64) CUtensorMap map_p, map_q;
    const int64_t K = g.kblocks * kMmBlock;
    cudaError_t e = make_operand_map(&map_p, p, g.rows_p, K, 128);
    if (e == cudaSuccess) e = make_operand_map(&map_q, q, g.rows_q, K, BN);
    if (e == cudaSuccess) e = engine_smem_ready<k_mm_split<OUT, BN, TILES>>(sizeof(SplitSmem<BN>), true);
    if (e != cudaSuccess) return e;
    const int64_t ty = (g.rows_p + 127) / 128, tz = (g.rows_q + BN - 1) / BN;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)split, (unsigned)ty, (unsigned)tz);
    cfg.blockDim = dim3(SplitSmem<BN>::kThreads);
    cfg.dynamicSmemBytes = sizeof(SplitSmem<BN>);
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // it waits before its first read
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)split;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = split > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, k_mm_split<OUT, BN, TILES>, map_p, map_q, g);
}

template <int OUT, int BN>
cudaError_t mm_split(const uint8_t *p, const uint8_t *q, const MmArgs &g, int split, cudaStream_t st)
{
    return g.shift_p ? mm_split_t<OUT, BN, true>(p, q, g, split, st) : mm_split_t<OUT, BN, false>(p, q, g, split, st);
}

// The registers that the pair kernel's epilogue takes over have to be there at
// its launch: it would wait for them forever.
template <int OUT, bool COLS> cudaError_t pair_registers_ready()
{
    static std::atomic<bool> ready{false};
    if (ready.load(std::memory_order_relaxed)) return cudaSuccess;
    cudaFuncAttributes a;
    const cudaError_t e = cudaFuncGetAttributes(&a, k_mm_pair<OUT, COLS>);
    if (e != cudaSuccess) return e;
    if (a.numRegs * kPairThreads < 32 * (kPairEpiWarps * kPairEpiRegs + 4 * kPairRegs)) return cudaErrorInvalidConfiguration;
    ready.store(true, std::memory_order_relaxed);
    return cudaSuccess;
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
    if (e == cudaSuccess) e = pair_registers_ready<OUT, COLS>();
    if (e != cudaSuccess) return e;
    const int64_t tiles = ((g.rows_p + 255) / 256) * ((g.rows_q + kPairN - 1) / kPairN);
    if (tiles > INT32_MAX) return cudaErrorInvalidValue;
    const int64_t pairs = sm_count() / 2;
    return launch_k(true, k_mm_pair<OUT, COLS>, dim3((unsigned)(2 * (tiles < pairs ? tiles : pairs))), dim3(kPairThreads),
                    sizeof(PairSmem), st, map_p, map_q, map_c, g);
}

// CTAs that clusters of `split` keep resident, one per SM: a cluster stays
// inside a GPC, whose SMs need not be a multiple of it (152 SMs: 144 in
// clusters of four, 120 in clusters of eight).
int cluster_ctas(int split)
{
    static std::atomic<int> known[64][3];   // of a device's splits 2, 4, 8
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;   // no answer, no clusters
    std::atomic<int> &k = known[dev][split == 2 ? 0 : split == 4 ? 1 : 2];
    const int c = k.load(std::memory_order_relaxed);
    if (c > 0) return c;
    constexpr auto kernel = k_mm_split<BF16, 128, true>;   // one CTA fills an SM
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)split);
    cfg.blockDim = dim3(SplitSmem<128>::kThreads);
    cfg.dynamicSmemBytes = sizeof(SplitSmem<128>);
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)split;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    int n = 0;
    if (engine_smem_ready<k_mm_split<BF16, 128, true>>(sizeof(SplitSmem<128>), true) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n <= 0)
        return 0;
    k.store(n * split, std::memory_order_relaxed);
    return n * split;
}

// Which kernel, and how wide and how deep a split: the least estimated time.
// The estimate's terms (us) are a fit to 1500 calls of every plan that 180
// shapes allow (1 to 1024 tokens, weights from 1024 x 1024 to 18432 x 7168 in
// both tilings; GB300, graphs of calls); its choices take 0.8% more time than
// the best plan on the average and 13% at most.  A call has a fixed part, a cluster
// adds its sum, a CTA takes `block` for each block of 128 weights x bn tokens
// (`rows` times as long where each weight row has a scale), two CTAs of an SM
// `share` times one's time, and a CTA that comes after another a start of its
// own.  Some of what it is drawn from, for 4096 x 4096 weights: 333 tokens 14.5
// at 192 wide and two deep, 17.4 at 128, 15.7 on the pair kernel; 700 tokens
// 16.5 there and 23 at 192.  A split has to be resident as a whole: clusters
// that wait for one another's SMs lose more than the split gains (2048 x 8192
// with 100 tokens, 128 wide: 10.5 us at a split of four, 17.0 at eight, whose
// 16 clusters are one more than fit).
struct MmPlan {
    int bn, split;   // bn 0: the pair kernel
};
MmPlan mm_plan(int64_t M, int64_t N, int64_t kblocks, bool rows, int sms)
{
    struct Width {
        int bn;
        double fixed, block, rows;
        int resident;
        double share;
    };
    static constexpr Width kWidths[] = {{16, 2.7, 0.24, 1.1, 2, 1.24},
                                        {32, 2.7, 0.253, 1.15, 2, 1.63},
                                        {64, 4.5, 0.3, 1.17, 2, 1.54},
                                        {128, 5.0, 0.374, 1.23, 1, 1.0},
                                        {192, 6.0, 0.511, 1.2, 1, 1.0}};
    const int64_t ty = (N + 127) / 128, pairs = sms / 2;
    const int64_t pair_tiles = ((M + 255) / 256) * ((N + kPairN - 1) / kPairN);
    MmPlan best = {0, 1};
    double cost = 3.25 + (double)((pair_tiles + pairs - 1) / pairs) * ((double)kblocks * (rows ? 0.589 : 0.407) + 0.75);
    for (const Width &w : kWidths) {
        const int64_t tz = (M + w.bn - 1) / w.bn;
        if ((w.bn > 16 && M <= w.bn / 2) || ty > 65535 || tz > 65535) continue;
        for (int split = 1; split <= kSplitMost && (split == 1 || 2 * split <= kblocks); split *= 2) {
            const int64_t ctas = ty * tz * split, n = (ctas + sms - 1) / sms;   // n: CTAs of an SM
            if (split > 1 && ctas > (int64_t)w.resident * cluster_ctas(split)) break;
            const double blocks = (double)((kblocks + split - 1) / split) * w.block * (rows ? w.rows : 1.0);
            const double times = (double)(n / w.resident) * w.share + (double)(n % w.resident);
            const double c = w.fixed + (split == 8 ? 1.0 : split == 4 ? 0.65 : split == 2 ? 0.43 : 0.0) + blocks * times +
                             1.6 * (double)((n - 1) / w.resident);
            if (c < cost) {
                cost = c;
                best = {w.bn, split};
            }
        }
    }
    return best;
}

template <int OUT>
cudaError_t mm_t(const uint8_t *a, const uint8_t *b, const MmArgs &g, cudaStream_t st)
{
    const int64_t M = g.rows_p, N = g.rows_q;
    const MmPlan plan = mm_plan(M, N, g.kblocks, g.shift_q == 0, sm_count());
    const int split = plan.split;
    MmArgs w = g;   // the weights on the lanes
    w.s_p = g.s_q;
    w.s_q = g.s_p;
    w.rows_p = N;
    w.rows_q = M;
    w.shift_p = g.shift_q;
    w.shift_q = g.shift_p;
    switch (plan.bn) {
    case 0: return g.shift_q ? mm_pair<OUT, false>(a, b, g, st) : mm_pair<OUT, true>(a, b, g, st);
    case 16: return mm_split<OUT, 16>(b, a, w, split, st);
    case 32: return mm_split<OUT, 32>(b, a, w, split, st);
    case 64: return mm_split<OUT, 64>(b, a, w, split, st);
    case 128: return mm_split<OUT, 128>(b, a, w, split, st);
    default: return mm_split<OUT, 192>(b, a, w, split, st);
    }
}

}  // namespace

cudaError_t launch_mm_blockwise(const uint8_t *a, const float *s_a, int tile_a, const uint8_t *b, const float *s_b, int tile_b,
                                int64_t M, int64_t N, int64_t K, void *c, int out, bool accumulate, int32_t *status,
                                int give_up, cudaStream_t st)
{
    MmArgs g = {s_a, s_b, M, N, K / kMmBlock, tile_a ? 7 : 0, tile_b ? 7 : 0, c, N, status, accumulate, kStoreDirect, give_up};
    return out == BF16 ? mm_t<BF16>(a, b, g, st) : mm_t<F32>(a, b, g, st);
}

}  // namespace qk
