// Dropout with the residual sum: y = residual + keep c x, the keep decisions
// drawn again from the counter (q_dropout.cuh) wherever they are needed.  The
// backward pass is the same kernel on dy without a residual.
//
// One thread takes the eight elements of a Philox block: the sum is formed in
// FP32 (one fused multiply-add) and rounded once to the output type.
#include "q_dropout.cuh"
#include "q_internal.h"

namespace qk {

namespace {

constexpr int kDropThreads = 256;

template <int DT> QD float load_one(const void *p, int64_t i);
template <> QD float load_one<BF16>(const void *p, int64_t i)
{
    return __uint_as_float((uint32_t)static_cast<const uint16_t *>(p)[i] << 16);
}
template <> QD float load_one<F32>(const void *p, int64_t i) { return static_cast<const float *>(p)[i]; }

template <int DT> QD void store_one(void *p, int64_t i, float v);
template <> QD void store_one<BF16>(void *p, int64_t i, float v) { static_cast<uint16_t *>(p)[i] = (uint16_t)bf16_bits(v); }
template <> QD void store_one<F32>(void *p, int64_t i, float v) { static_cast<float *>(p)[i] = v; }

template <int DT, bool RES>
__global__ void __launch_bounds__(kDropThreads)
k_drop_add(const void *x, const void *residual, void *y, int64_t n, const DropArgs d)
{
    const int64_t b = (int64_t)blockIdx.x * kDropThreads + threadIdx.x;
    if (b * 8 >= n) return;
    const uint4 draws = drop_draws((uint64_t)b, d);
#pragma unroll
    for (int j = 0; j < 8; j++) {
        const int64_t i = b * 8 + j;
        if (i < n) {
            const float v = load_one<DT>(x, i), r = RES ? load_one<DT>(residual, i) : 0.0f;
            const float kept = RES ? __fmaf_rn(v, d.c, r) : __fmul_rn(v, d.c);
            store_one<DT>(y, i, drop_keep(draws, j, d.threshold) ? kept : r);
        }
    }
}

template <int DT>
cudaError_t drop_t(const void *x, int64_t n, const void *residual, const DropArgs &d, void *y, cudaStream_t st)
{
    const int64_t grid = ((n + 7) / 8 + kDropThreads - 1) / kDropThreads;
    if (residual != nullptr) k_drop_add<DT, true><<<(unsigned)grid, kDropThreads, 0, st>>>(x, residual, y, n, d);
    else k_drop_add<DT, false><<<(unsigned)grid, kDropThreads, 0, st>>>(x, nullptr, y, n, d);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_drop_add(const void *x, int dt, int64_t n, const void *residual, uint32_t threshold, float c,
                            uint64_t seed, uint64_t offset, void *y, cudaStream_t st)
{
    const DropArgs d = {philox_keys(seed), offset, threshold, c};
    return dt == BF16 ? drop_t<BF16>(x, n, residual, d, y, st) : drop_t<F32>(x, n, residual, d, y, st);
}

}  // namespace qk
