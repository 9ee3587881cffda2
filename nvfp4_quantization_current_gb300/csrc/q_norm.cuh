// What the norm's kernels share: element access, sums over the threads of a row,
// and bulk copies of rows into shared memory.
#pragma once

#include "q_engine.cuh"
#include "q_global.cuh"
#include "q_internal.h"
#include "q_packed.cuh"

namespace qk {

// W consecutive elements in one access: 16 bytes, or one element where rows do
// not start on 16-byte boundaries.
template <int DT, int W> struct Piece {
    static constexpr int kBytes = W * In<DT>::BYTES;
    static constexpr int kWords = kBytes < 4 ? 1 : kBytes / 4;
    uint32_t w[kWords];
    QD void load(const void *p, int64_t i)
    {
        const char *const at = static_cast<const char *>(p) + i * In<DT>::BYTES;
        if constexpr (kBytes == 16) {
            asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "l"(at));
        } else if constexpr (kBytes == 4) {
            w[0] = *reinterpret_cast<const uint32_t *>(at);
        } else {
            w[0] = *reinterpret_cast<const uint16_t *>(at);
        }
    }
    QD void shared(const uint8_t *p, int i)
    {
        const uint8_t *const at = p + i * In<DT>::BYTES;
        if constexpr (kBytes == 16) {
            const uint4 v = lds16(at);
            w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
        } else if constexpr (kBytes == 4) {
            w[0] = *reinterpret_cast<const uint32_t *>(at);
        } else {
            w[0] = *reinterpret_cast<const uint16_t *>(at);
        }
    }
    QD void store(void *p, int64_t i) const
    {
        char *const at = static_cast<char *>(p) + i * In<DT>::BYTES;
        if constexpr (kBytes == 16) stg16(at, make_uint4(w[0], w[1], w[2], w[3]));
        else if constexpr (kBytes == 4) *reinterpret_cast<uint32_t *>(at) = w[0];
        else *reinterpret_cast<uint16_t *>(at) = (uint16_t)w[0];
    }
    QD void zero()
    {
#pragma unroll
        for (int i = 0; i < kWords; i++) w[i] = 0u;
    }
    QD float at(int j) const
    {
        if constexpr (DT == F32) return __uint_as_float(w[j]);
        else if constexpr (W == 1) return __uint_as_float(w[0] << 16);
        else return __uint_as_float((j & 1) ? (w[j >> 1] & 0xFFFF0000u) : (w[j >> 1] << 16));
    }
    // Elements 2j and 2j + 1 as two packed FP32 values.
    QD uint64_t pair(int j) const
    {
        static_assert(W % 2 == 0, "pairs");
        if constexpr (DT == F32) return pack2(w[2 * j], w[2 * j + 1]);
        else return pack2(w[j] << 16, w[j] & 0xFFFF0000u);
    }
    QD void set_pair(int j, uint64_t v)
    {
        float a, b;
        unpack2(v, a, b);
        if constexpr (DT == F32) w[2 * j] = __float_as_uint(a), w[2 * j + 1] = __float_as_uint(b);
        else w[j] = bf16_pair(a, b);
    }
    QD void add(const Piece &p)
    {
        if constexpr (W > 1) {
#pragma unroll
            for (int j = 0; j < W / 2; j++) set_pair(j, fadd2(pair(j), p.pair(j)));
        } else {
            const float f[1] = {at(0) + p.at(0)};
            set(f);
        }
    }
    QD void set(const float (&f)[W])
    {
        if constexpr (DT == F32) {
#pragma unroll
            for (int j = 0; j < W; j++) w[j] = __float_as_uint(f[j]);
        } else if constexpr (W == 1) {
            w[0] = bf16_bits(f[0]);
        } else {
#pragma unroll
            for (int j = 0; j < W; j += 2) w[j / 2] = bf16_pair(f[j], f[j + 1]);
        }
    }
};

// W weights from element k on, whichever type they have (k a multiple of W, the weights 16-byte aligned).
template <int W> QD void load_weights(float (&f)[W], const void *w, bool f32, int64_t k)
{
    if (f32) {
        const float *p = static_cast<const float *>(w) + k;
        if constexpr (W % 4 == 0) {
#pragma unroll
            for (int j = 0; j < W; j += 4) {
                const uint4 v = load_16(p + j);
#pragma unroll
                for (int i = 0; i < 4; i++) f[j + i] = elem<F32>(v, i);
            }
        } else {
#pragma unroll
            for (int j = 0; j < W; j++) f[j] = load_float(p + j);
        }
    } else {
        const uint16_t *p = static_cast<const uint16_t *>(w) + k;
        if constexpr (W == 8) {
            const uint4 v = load_16(p);
#pragma unroll
            for (int j = 0; j < 8; j++) f[j] = elem<BF16>(v, j);
        } else if constexpr (W == 4) {
            const uint2 v = load_8(p);
            f[0] = __uint_as_float(v.x << 16), f[1] = __uint_as_float(v.x & 0xFFFF0000u);
            f[2] = __uint_as_float(v.y << 16), f[3] = __uint_as_float(v.y & 0xFFFF0000u);
        } else {
#pragma unroll
            for (int j = 0; j < W; j++) f[j] = load_bf16(p + j);
        }
    }
}

QD float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// Sum over the n consecutive warps from `first` on that share a row, to all of
// their threads; part: a word per warp, used by no other call that is in flight.
// Every thread of the CTA calls it.
QD float row_sum(float v, float *part, int first, int n)
{
    v = warp_sum(v);
    if (n == 1) return v;
    const int lane = threadIdx.x & 31;
    if (lane == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    return warp_sum(lane < n ? part[first + lane] : 0.0f);
}

// A copy of whole 16-byte pieces into this CTA's shared memory, counted on `bar`.
QD void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(smem_u32(dst)), "l"(src), "r"(bytes), "r"(smem_u32(bar)) : "memory");
}
// The same with a policy of what L2 keeps: of lines that it may drop first, or as usual.
QD uint64_t l2_policy(bool drop_first)
{
    uint64_t first, usual;
    asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(first));
    asm("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(usual));
    return drop_first ? first : usual;
}
QD void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar, uint64_t policy)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;"
                 ::"r"(smem_u32(dst)), "l"(src), "r"(bytes), "r"(smem_u32(bar)), "l"(policy) : "memory");
}

constexpr int kRingBytes = 200 * 1024;   // shared memory of an SM's CTAs for rows on their way

}  // namespace qk
