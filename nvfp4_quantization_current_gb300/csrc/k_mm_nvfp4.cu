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
template <int OUT, bool WHOLE> cudaError_t pair4_registers_ready()
{
    static std::atomic<bool> ready{false};
    if (ready.load(std::memory_order_relaxed)) return cudaSuccess;
    cudaFuncAttributes a;
    const cudaError_t e = cudaFuncGetAttributes(&a, k_mm4_pair<OUT, WHOLE>);
    if (e != cudaSuccess) return e;
    if (a.numRegs * kPair4Threads < 32 * (kPair4EpiWarps * kPair4EpiRegs + (2 + kPair4ScaleWarps) * kPair4Regs)) return cudaErrorInvalidConfiguration;
    ready.store(true, std::memory_order_relaxed);
    return cudaSuccess;
}

// Tiles of 256 x 256 on CTA pairs.
template <int OUT, bool WHOLE> cudaError_t mm4_pair(const uint8_t *p, const uint8_t *q, Mm4Args a, int64_t K, cudaStream_t st)
{
    alignas(64) CUtensorMap map_p, map_q, map_c = {};
    MmArgs &g = a.store;
    cudaError_t e = make_operand_map(&map_p, p, g.rows_p, K / 2, 128);
    if (e == cudaSuccess) e = make_operand_map(&map_q, q, g.rows_q, K / 2, 128);
    const bool bulk = g.ldc % (OUT == F32 ? 4 : 8) == 0 && (OUT == F32 || !g.accumulate);
    g.store = !bulk ? kStoreDirect : g.accumulate ? kStoreBulkAdd : kStoreBulk;
    if (e == cudaSuccess && bulk) e = make_result_map(&map_c, g.c, OUT, g.rows_p, g.rows_q);
    if (e == cudaSuccess) e = engine_smem_ready<k_mm4_pair<OUT, WHOLE>>(sizeof(Pair4Smem));
    if (e == cudaSuccess) e = pair4_registers_ready<OUT, WHOLE>();
    if (e != cudaSuccess) return e;
    const int64_t tiles_p = (g.rows_p + 255) / 256, tiles_q = (g.rows_q + 255) / 256, tiles = tiles_p * tiles_q, pairs = sm_count() / 2;
    a.group = tiles_q < tiles_p && tiles_q <= 32 ? 2 : tiles_p < 32 ? (int)tiles_p : 32;
    if (tiles > INT32_MAX) return cudaErrorInvalidValue;
    return launch_k(true, k_mm4_pair<OUT, WHOLE>, dim3((unsigned)(2 * (tiles < pairs ? tiles : pairs))), dim3(kPair4Threads),
                    sizeof(Pair4Smem), st, map_p, map_q, map_c, a);
}

Mm4Scales scales_of(const uint8_t *at, int blk, int64_t rows, int64_t K) { return {at, K / 16, (int)rows, blk ? 4 : 0}; }

// Every row of scales begins on a 16-byte boundary.
bool whole_rows(const Mm4Scales &s) { return ((reinterpret_cast<uintptr_t>(s.at) | (uintptr_t)s.pitch) & 15) == 0; }

template <int OUT>
cudaError_t mm4_t(const uint8_t *a, const uint8_t *b, const Mm4Args &g, int64_t K, cudaStream_t st)
{
    const int64_t M = g.store.rows_p, N = g.store.rows_q;
    const bool whole = whole_rows(g.p) && whole_rows(g.q);
    if (((M + 255) / 256) * ((N + 255) / 256) >= 40) return whole ? mm4_pair<OUT, true>(a, b, g, K, st) : mm4_pair<OUT, false>(a, b, g, K, st);
    Mm4Args w = g;   // the weights on the lanes
    w.p = g.q;
    w.q = g.p;
    w.s_p = g.s_q;
    w.s_q = g.s_p;
    w.store.rows_p = N;
    w.store.rows_q = M;
    const int64_t kb = g.store.kblocks;
    int split = 1;
    const int bn = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : M <= 128 ? 128 : 192;
    while (split < kSplitMost && 2 * split <= kb && ((N + 127) / 128) * ((M + bn - 1) / bn) * split * 2 <= 144) split *= 2;
    switch (bn) {
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
                                bool accumulate, int32_t *status, bool give_up, cudaStream_t st)
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
