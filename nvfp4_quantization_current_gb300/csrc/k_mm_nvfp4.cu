// NVFP4 matrix product: the consumer of the copies of q_nvfp4.
//
//   C[m, n] (+)= s_a s_b sum_kb sb_a[m, kb] sb_b[n, kb] P_kb[m, n],
//   P_kb[m, n] = sum of a[m, k] b[n, k] over the 16 elements k of block kb
//
// with a [M, K] and b [N, K] E2M1 codes, two per byte, K contiguous, an E4M3
// scale per 1x16 or 16x16 block and one FP32 scale per tensor.  The tensor core
// takes the codes and the block scales (tcgen05 kind mxf4nvf4, a scale per 16
// elements) and adds in FP32; the tensors' scales are multiplied in at the end.
#include "k_mm4_pair.cuh"
#include "k_mm4_split.cuh"
#include "q_internal.h"

namespace qk {

namespace {

template <int OUT, int BN, bool WHOLE> cudaError_t mm4_split_t(const uint8_t *p, const uint8_t *q, const Mm4Args &a, int64_t K, int split, cudaStream_t st)
{
    alignas(64) CUtensorMap map_p, map_q;
    cudaError_t e = make_operand_map(&map_p, p, a.store.rows_p, K / 2, 128);
    if (e == cudaSuccess) e = make_operand_map(&map_q, q, a.store.rows_q, K / 2, BN);
    if (e == cudaSuccess) e = engine_smem_ready<k_mm4_split<OUT, BN, WHOLE>>(sizeof(Split4Smem<BN>), true);
    if (e != cudaSuccess) return e;
    const int64_t ty = (a.store.rows_p + 127) / 128, tz = (a.store.rows_q + BN - 1) / BN;
    if (ty > 65535 || tz > 65535) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)split, (unsigned)ty, (unsigned)tz);
    cfg.blockDim = dim3(Split4Smem<BN>::kThreads);
    cfg.dynamicSmemBytes = sizeof(Split4Smem<BN>);
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // it waits before its first read
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)split;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = split > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, k_mm4_split<OUT, BN, WHOLE>, map_p, map_q, a);
}

template <int OUT, int BN>
cudaError_t mm4_split(const uint8_t *p, const uint8_t *q, const Mm4Args &a, int64_t K, bool whole, int split, cudaStream_t st)
{
    return whole ? mm4_split_t<OUT, BN, true>(p, q, a, K, split, st) : mm4_split_t<OUT, BN, false>(p, q, a, K, split, st);
}

// The registers that the pair kernel's epilogue takes over have to be there at
// its launch: it would wait for them forever.
template <int OUT, int BN, bool WHOLE, int KIND> cudaError_t pair4_registers_ready()
{
    static std::atomic<bool> ready{false};
    if (ready.load(std::memory_order_relaxed)) return cudaSuccess;
    cudaFuncAttributes a;
    const cudaError_t e = cudaFuncGetAttributes(&a, k_mm4_pair<OUT, BN, WHOLE, KIND>);
    if (e != cudaSuccess) return e;
    if (a.numRegs * kPair4Threads < 32 * (kPair4EpiWarps * kPair4EpiRegs + (2 + kPair4ScaleWarps) * kPair4Regs)) return cudaErrorInvalidConfiguration;
    ready.store(true, std::memory_order_relaxed);
    return cudaSuccess;
}

// Tiles of 256 x BN on CTA pairs.
template <int OUT, int BN, bool WHOLE, int KIND> cudaError_t mm4_pair_t(const uint8_t *p, const uint8_t *q, Mm4Args a, int64_t K, cudaStream_t st)
{
    alignas(64) CUtensorMap map_p, map_q, map_c = {};
    MmArgs &g = a.store;
    cudaError_t e = make_operand_map(&map_p, p, g.rows_p, K / 2, 128);
    if (e == cudaSuccess) e = make_operand_map(&map_q, q, g.rows_q, K / 2, BN / 2);
    g.store = KIND == kAnyC || OUT == BF16 ? kStoreDirect : g.accumulate ? kStoreBulkAdd : kStoreBulk;
    if (e == cudaSuccess && KIND == kPlainC && OUT == F32) e = make_result_map(&map_c, g.c, OUT, g.rows_p, g.rows_q, 16);
    if (e == cudaSuccess) e = engine_smem_ready<k_mm4_pair<OUT, BN, WHOLE, KIND>>(sizeof(Pair4Smem<OUT, BN>));
    if (e == cudaSuccess) e = pair4_registers_ready<OUT, BN, WHOLE, KIND>();
    if (e != cudaSuccess) return e;
    const int64_t tiles_p = (g.rows_p + 255) / 256, tiles_q = (g.rows_q + BN - 1) / BN, tiles = tiles_p * tiles_q, pairs = sm_count() / 2;
    a.group = tiles_q < tiles_p && tiles_q <= 32 ? 2 : tiles_p < 32 ? (int)tiles_p : 32;
    if (tiles > INT32_MAX) return cudaErrorInvalidValue;
    return launch_k(true, k_mm4_pair<OUT, BN, WHOLE, KIND>, dim3((unsigned)(2 * (tiles < pairs ? tiles : pairs))), dim3(kPair4Threads),
                    sizeof(Pair4Smem<OUT, BN>), st, map_p, map_q, map_c, a);
}

Mm4Scales scales_of(const uint8_t *at, int blk, int64_t rows, int64_t K) { return {at, K / 16, (int)rows, blk ? 4 : 0}; }

// Every row of scales begins on a 16-byte boundary.
bool whole_rows(const Mm4Scales &s) { return ((reinterpret_cast<uintptr_t>(s.at) | (uintptr_t)s.pitch) & 15) == 0; }

template <int OUT, bool WHOLE> cudaError_t mm4_pair(const uint8_t *p, const uint8_t *q, const Mm4Args &a, int64_t K, int bn, bool any, cudaStream_t st)
{
    if constexpr (OUT == BF16)
        if (a.store.accumulate) return mm4_pair_t<OUT, 256, WHOLE, kAddC>(p, q, a, K, st);
    if (any) return mm4_pair_t<OUT, 256, WHOLE, kAnyC>(p, q, a, K, st);
    return bn == 128 ? mm4_pair_t<OUT, 128, WHOLE, kPlainC>(p, q, a, K, st) : mm4_pair_t<OUT, 256, WHOLE, kPlainC>(p, q, a, K, st);
}

// CTAs that clusters of `split` keep resident, one per SM (see the blockwise product's).
int cluster_ctas4(int split)
{
    static std::atomic<int> known[64][3];   // of a device's splits 2, 4, 8
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;   // no answer, no clusters
    std::atomic<int> &k = known[dev][split == 2 ? 0 : split == 4 ? 1 : 2];
    const int c = k.load(std::memory_order_relaxed);
    if (c > 0) return c;
    constexpr auto kernel = k_mm4_split<BF16, 128, true>;   // one CTA fills an SM
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)split);
    cfg.blockDim = dim3(Split4Smem<128>::kThreads);
    cfg.dynamicSmemBytes = sizeof(Split4Smem<128>);
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)split;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    int n = 0;
    if (engine_smem_ready<k_mm4_split<BF16, 128, true>>(sizeof(Split4Smem<128>), true) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n <= 0)
        return 0;
    k.store(n * split, std::memory_order_relaxed);
    return n * split;
}

// Which kernel, and how wide and how deep a split: the least estimated time.
// The estimate's terms (us) are fits to calls of every plan that a shape
// allows, those of the split kernel to 170 shapes (1 to 4096 tokens, weights from 512 x
// 256 to 18432 x 18432, K of every multiple of 32, weights in either blocks), those of the pair kernel to
// 240 (GB300, graphs of calls, 1919 of them); its choices take 0.8% more time than the best plan of these on
// the average and 14% at most.  A call has a fixed part, a cluster adds its sum, a CTA takes `block` for each 256 elements of K
// (`odd` times as long where scale rows begin anywhere), two CTAs of an SM `share`
// times one's time, and a CTA that comes after another a start of its own; a pair takes `tile` for a tile's end.  Some of
// what it is drawn from: one token with 4096 x 4096 weights 4.6 us at a split of four,
// 7.6 without, 8.6 on the pair kernel; 64 tokens with 4096 x 14336 10.0 at 64 and four, 21.4 on the
// pair.  Tiles of 256 x 128 are for results that tiles of 256 x 256 are too few for, the best plan of 36 shapes, by 9% on
// the average: 333 tokens with 4096 x 4096 9.6 us, 10.4 in 256s, 10.8 at 192 wide and
// two deep; 380 with 2304 x 1280 5.7, 6.6 and 8.4; but 768 with 4096 x 4096, two rounds of them, 14.4 and 11.0.
struct Mm4Plan {
    int bn, split;   // split 0: the pair kernel
};
Mm4Plan mm4_plan(int64_t M, int64_t N, int64_t kblocks, bool whole, bool any, int sms)
{
    struct Width {
        int bn;
        double fixed, block, share, odd, split[3], start;
        int resident;
    };
    static constexpr Width kWidths[] = {{16, 3.62, 0.269, 1.473, 1.207, {0.56, 0.62, 0.67}, 2.92, 2},
                                        {32, 4.71, 0.290, 1.477, 1.137, {0.09, 0.0, 0.31}, 3.95, 2},
                                        {64, 6.22, 0.316, 1.589, 1.152, {0.0, 0.0, 0.04}, 5.77, 2},
                                        {128, 6.97, 0.323, 1.0, 1.192, {0.0, 0.0, 0.0}, 6.87, 1},
                                        {192, 8.73, 0.358, 1.0, 1.272, {0.0, 0.0, 0.0}, 9.31, 1}};
    struct Pair {
        int bn;
        double fixed, block, tile, odd, odd_tile;
    };
    static constexpr Pair kPairs[] = {{256, 2.856, 0.361, 1.663, 1.352, 1.438}, {128, 2.843, 0.323, 0.995, 1.383, 1.986}};
    const int64_t ty = (N + 127) / 128, pairs = sms / 2;
    Mm4Plan best = {256, 0};
    double cost = 0.0;
    for (const Pair &p : kPairs) {
        if (p.bn == 128 && any) continue;   // that kernel has no such form
        const int64_t tiles = ((M + 255) / 256) * ((N + p.bn - 1) / p.bn);
        const double c = p.fixed + (double)((tiles + pairs - 1) / pairs) * ((double)kblocks * p.block * (whole ? 1.0 : p.odd) + p.tile * (whole ? 1.0 : p.odd_tile));
        if (p.bn == 256 || c < cost) {
            cost = c;
            best.bn = p.bn;
        }
    }
    for (const Width &w : kWidths) {
        const int64_t tz = (M + w.bn - 1) / w.bn;
        if ((w.bn > 16 && M <= w.bn / 2) || ty > 65535 || tz > 65535) continue;
        for (int i = 0; i <= 3; i++) {
            const int split = 1 << i;
            const int64_t ctas = ty * tz * split, n = (ctas + sms - 1) / sms;   // n: CTAs of an SM
            if (split > 1 && (split > kblocks || ctas > (int64_t)w.resident * cluster_ctas4(split))) break;
            const double times = (double)(n / w.resident) * w.share + (double)(n % w.resident);
            const double c = w.fixed + (i > 0 ? w.split[i - 1] : 0.0) + (double)((kblocks + split - 1) / split) * w.block * times * (whole ? 1.0 : w.odd) +
                             w.start * (double)((n - 1) / w.resident);
            if (c < cost) {
                cost = c;
                best = {w.bn, split};
            }
        }
    }
    return best;
}

template <int OUT>
cudaError_t mm4_t(const uint8_t *a, const uint8_t *b, const Mm4Args &g, int64_t K, cudaStream_t st)
{
    const int64_t M = g.store.rows_p, N = g.store.rows_q;
    const bool whole = whole_rows(g.p) && whole_rows(g.q);
    const bool any = g.store.ldc % (OUT == F32 ? 4 : 8) != 0 || (OUT == BF16 && g.store.accumulate);
    const Mm4Plan plan = mm4_plan(M, N, g.store.kblocks, whole, any, sm_count());
    const int split = plan.split;
    if (split == 0) return whole ? mm4_pair<OUT, true>(a, b, g, K, plan.bn, any, st) : mm4_pair<OUT, false>(a, b, g, K, plan.bn, any, st);
    Mm4Args w = g;   // the weights on the lanes
    w.p = g.q;
    w.q = g.p;
    w.s_p = g.s_q;
    w.s_q = g.s_p;
    w.store.rows_p = N;
    w.store.rows_q = M;
    switch (plan.bn) {
    case 16: return mm4_split<OUT, 16>(b, a, w, K, whole, split, st);
    case 32: return mm4_split<OUT, 32>(b, a, w, K, whole, split, st);
    case 64: return mm4_split<OUT, 64>(b, a, w, K, whole, split, st);
    case 128: return mm4_split<OUT, 128>(b, a, w, K, whole, split, st);
    default: return mm4_split<OUT, 192>(b, a, w, K, whole, split, st);
    }
}

}  // namespace

cudaError_t launch_matmul_nvfp4(const uint8_t *a, const uint8_t *sb_a, const float *s_a, int blk_a, const uint8_t *b,
                                const uint8_t *sb_b, const float *s_b, int blk_b, int64_t M, int64_t N, int64_t K, void *c, int out,
                                bool accumulate, int32_t *status, int give_up, cudaStream_t st)
{
    Mm4Args g = {};
    g.store = {nullptr, nullptr, M, N, (K + kMm4Block - 1) / kMm4Block, 0, 0, c, N, status, accumulate, kStoreDirect, give_up};
    g.p = scales_of(sb_a, blk_a, M, K);
    g.q = scales_of(sb_b, blk_b, N, K);
    g.s_p = s_a;
    g.s_q = s_b;
    return out == BF16 ? mm4_t<BF16>(a, b, g, K, st) : mm4_t<F32>(a, b, g, K, st);
}

}  // namespace qk
