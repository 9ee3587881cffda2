// Dropout with the residual sum: y = residual + keep c x, the keep decisions
// drawn again from the counter (q_dropout.cuh) wherever they are needed.  The
// backward pass is the same kernel on dy without a residual.
//
// Bound by memory (two or three tensors of n elements against ten Philox
// rounds per eight): a thread takes the eight elements of kDropUnroll Philox
// blocks, in 16-byte pieces that are all on their way before the first draw is
// computed.  The sum is formed in FP32 (one fused multiply-add) and rounded
// once to the output type.  Measured on a GB300, inputs from memory: 8192 x 4096
// BF16 with the residual 30.7 us (201 MB at 6.6 TB/s), without it 21.6 us, with
// one element per load 84 us; 128 x 4096 1.7 us, of which the launch is most.
#include <type_traits>

#include "q_dropout.cuh"
#include "q_internal.h"

namespace qk {

namespace {

constexpr int kDropThreads = 256, kDropUnroll = 4;

// 16 bytes that this thread alone reads, and may overwrite (y may be x).
QD uint4 load16(const void *p)
{
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

template <bool RES> QD float drop_sum(float x, float r, bool keep, float c)
{
    return keep ? (RES ? __fmaf_rn(x, c, r) : __fmul_rn(x, c)) : r;
}

// Eight elements as 16-byte vectors: one of BF16, two of FP32.
template <int DT> struct Eight {
    static constexpr int N = DT == BF16 ? 1 : 2;
    uint4 v[N];
    QD void load(const void *p, int64_t block)
    {
#pragma unroll
        for (int i = 0; i < N; i++) v[i] = load16(static_cast<const uint4 *>(p) + block * N + i);
    }
    QD void store(void *p, int64_t block) const
    {
#pragma unroll
        for (int i = 0; i < N; i++) stg16(static_cast<uint4 *>(p) + block * N + i, v[i]);
    }
    // Zeroes what the draws drop.
    QD void drop(const uint4 &draws, const DropArgs &d)
    {
        uint32_t *const w = reinterpret_cast<uint32_t *>(v);
#pragma unroll
        for (int j = 0; j < 8; j++)
            if (d.all || !drop_keep(draws, j, d.threshold)) {
                if (DT == BF16) w[j / 2] &= j & 1 ? 0x0000FFFFu : 0xFFFF0000u;
                else w[j] = 0u;
            }
    }
    QD uint32_t absmax() const
    {
        if constexpr (DT == BF16) return absmax_bits<BF16>(v[0]);
        else return max(absmax_bits<F32>(v[0]), absmax_bits<F32>(v[1]));
    }
    // E4M3 codes of alpha (c x).
    QD void codes(float alpha, float c, uint32_t (&o)[2]) const
    {
        auto times_c = [&](float &f0, float &f1) { mul2(f0, f1, c, c); };
        if constexpr (DT == BF16) {
            chunk_fp8<BF16, E4M3>(v[0], alpha, o, times_c);
        } else {
            chunk_fp8<F32, E4M3>(v[0], alpha, o, times_c);
            chunk_fp8<F32, E4M3>(v[1], alpha, o + 1, times_c);
        }
    }
    QD float at(int j) const { return DT == BF16 ? elem<BF16>(v[0], j) : elem<F32>(v[(j >> 2) % N], j & 3); }
};

template <int DT, bool RES> QD Eight<DT> drop_eight(const Eight<DT> &x, const Eight<DT> &r, uint64_t block, const DropArgs &d)
{
    const uint4 draws = drop_draws(block, d);
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; j++) y[j] = drop_sum<RES>(x.at(j), RES ? r.at(j) : 0.0f, !d.all && drop_keep(draws, j, d.threshold), d.c);
    Eight<DT> out;
    if constexpr (DT == BF16) {
        out.v[0] = make_uint4(bf16_pair(y[0], y[1]), bf16_pair(y[2], y[3]), bf16_pair(y[4], y[5]), bf16_pair(y[6], y[7]));
    } else {
#pragma unroll
        for (int i = 0; i < 2; i++)
            out.v[i] = make_uint4(__float_as_uint(y[4 * i]), __float_as_uint(y[4 * i + 1]), __float_as_uint(y[4 * i + 2]),
                                  __float_as_uint(y[4 * i + 3]));
    }
    return out;
}

template <int DT, bool RES>
__global__ void __launch_bounds__(kDropThreads)
k_drop_add(const void *x, const void *residual, void *y, int64_t n, const DropArgs d)
{
    const int64_t b0 = (int64_t)blockIdx.x * (kDropThreads * kDropUnroll) + threadIdx.x, blocks = n / 8;
    Eight<DT> vx[kDropUnroll], vr[kDropUnroll];
    griddep_wait();   // nothing was read or written so far
#pragma unroll
    for (int u = 0; u < kDropUnroll; u++) {
        const int64_t b = b0 + u * kDropThreads;
        if (b < blocks) {
            vx[u].load(x, b);
            if (RES) vr[u].load(residual, b);
        }
    }
#pragma unroll
    for (int u = 0; u < kDropUnroll; u++) {
        const int64_t b = b0 + u * kDropThreads;
        if (b < blocks) drop_eight<DT, RES>(vx[u], vr[u], (uint64_t)b, d).store(y, b);
    }
    if (blockIdx.x == 0 && threadIdx.x < (n & 7)) {   // what is left of the last block
        const int64_t i = blocks * 8 + threadIdx.x;
        const bool keep = !d.all && drop_keep(drop_draws((uint64_t)blocks, d), threadIdx.x, d.threshold);
        using T = typename std::conditional<DT == BF16, uint16_t, float>::type;
        auto value = [&](const void *p) {
            if constexpr (DT == BF16) return __uint_as_float((uint32_t) static_cast<const T *>(p)[i] << 16);
            else return static_cast<const T *>(p)[i];
        };
        const float v = drop_sum<RES>(value(x), RES ? value(residual) : 0.0f, keep, d.c);
        if constexpr (DT == BF16) static_cast<T *>(y)[i] = (T)bf16_bits(v);
        else static_cast<T *>(y)[i] = v;
    }
}

// The rowwise 1x128 copy alone of y = keep c x in FP32 (with a transposed copy
// the tile engine's kernel makes both): codes of RN(alpha RN(c x)), one FP32
// scale per 128 elements.  K is a multiple of 128, so that the copy lies over
// the flat tensor: a thread takes one Philox block of each of four passes, 16
// lanes hold 128 elements.  The four maxima are reduced over the 16 lanes by a
// halving exchange, after which lane l holds that of pass l / 4 % 4, takes its
// quotients once, and the alphas go back by index shuffles.
//
// FP32 is bound by memory: 8192 x 4096 26.0 us (169 MB at 6.5 TB/s).  BF16 takes
// 22.9 (101 MB at 4.4 TB/s), and the draws alone do not account for it: k_drop_add
// without a residual draws the same and moves 134 MB in 21.6.  The draws, the
// reduction over 16 lanes and the cast of one pass follow each other.  256 x 2048
// takes 1.7.  Both copies' kernel took 54.1 us, 28.2 and 5.0 for the rowwise copy.
template <int DT>
__global__ void __launch_bounds__(kDropThreads)
k_drop_q_rows(const void *x, uint8_t *q_row, float *s_row, int64_t n, int32_t *status, const DropArgs d)
{
    static_assert(kDropUnroll == 4, "the exchange is of four maxima");
    const int64_t b0 = (int64_t)blockIdx.x * (kDropThreads * kDropUnroll) + threadIdx.x, blocks = n / 8;
    const int lane = threadIdx.x & 31;
    Eight<DT> v[kDropUnroll] = {};
    uint32_t top[kDropUnroll];
    griddep_wait();   // nothing was read or written so far
#pragma unroll
    for (int u = 0; u < kDropUnroll; u++)
        if (b0 + u * kDropThreads < blocks) v[u].load(x, b0 + u * kDropThreads);
#pragma unroll
    for (int u = 0; u < kDropUnroll; u++) {
        v[u].drop(drop_draws((uint64_t)(b0 + u * kDropThreads), d), d);
        top[u] = v[u].absmax();
    }
    const bool b3 = lane & 8, b2 = lane & 4;
    uint32_t k0 = b3 ? top[2] : top[0], k1 = b3 ? top[3] : top[1];
    k0 = max(k0, __shfl_xor_sync(0xFFFFFFFFu, b3 ? top[0] : top[2], 8));
    k1 = max(k1, __shfl_xor_sync(0xFFFFFFFFu, b3 ? top[1] : top[3], 8));
    uint32_t m = max(b2 ? k1 : k0, __shfl_xor_sync(0xFFFFFFFFu, b2 ? k0 : k1, 4));
    m = group_max<4>(m);
    const uint32_t b = __float_as_uint(__fmul_rn(__uint_as_float(m), d.c));   // max|y| = RN(c max|kept x|)
    const float alpha = alpha_from_amax(448.0f, __uint_as_float(b)), s = __fdiv_rn(1.0f, alpha);
    const int64_t mine = b0 + (lane >> 2 & 3) * kDropThreads;
    if (mine < blocks && (lane & 3) == 0) {
        s_row[mine / 16] = s;
        flag_nonfinite(status, b);
    }
#pragma unroll
    for (int u = 0; u < kDropUnroll; u++) {
        const float a = __shfl_sync(0xFFFFFFFFu, alpha, (lane & 16) + 4 * u);
        uint32_t o[2];
        v[u].codes(a, d.c, o);
        if (b0 + u * kDropThreads < blocks) stg8(q_row + (b0 + u * kDropThreads) * 8, o[0], o[1]);
    }
}

template <int DT>
cudaError_t drop_t(const void *x, int64_t n, const void *residual, const DropArgs &d, void *y, cudaStream_t st)
{
    const int64_t per = 8 * kDropThreads * kDropUnroll, grid = (n + per - 1) / per;
    // Launched while the kernel ahead ends: 8192 x 4096 27.5 us a call in a stream, 29.6
    // otherwise (the inputs partly in L2), 128 x 4096 in a graph 1.6 and 1.8.  (A signal of its own that the
    // kernel behind may start filled the SMs unevenly: 3.3 M elements 7.7 us for 5.1.)
    return launch_k(true, residual != nullptr ? k_drop_add<DT, true> : k_drop_add<DT, false>,
                    dim3((unsigned)grid), dim3(kDropThreads), 0, st, x, residual, y, n, d);
}

}  // namespace

cudaError_t launch_drop_add(const void *x, int dt, int64_t n, const void *residual, uint32_t threshold, float c,
                            uint64_t seed, uint64_t offset, void *y, cudaStream_t st)
{
    const DropArgs d = drop_args(seed, offset, threshold, c);
    return dt == BF16 ? drop_t<BF16>(x, n, residual, d, y, st) : drop_t<F32>(x, n, residual, d, y, st);
}

cudaError_t launch_drop_q_rows(const void *x, int dt, int64_t n, uint32_t threshold, float c, uint64_t seed, uint64_t offset,
                               uint8_t *q_row, float *s_row, int32_t *status, cudaStream_t st)
{
    const DropArgs d = drop_args(seed, offset, threshold, c);
    const int64_t per = 8 * kDropThreads * kDropUnroll, grid = (n + per - 1) / per;
    return launch_k(true, dt == BF16 ? k_drop_q_rows<BF16> : k_drop_q_rows<F32>, dim3((unsigned)grid), dim3(kDropThreads), 0, st,
                    x, q_row, s_row, n, status, d);
}

}  // namespace qk
