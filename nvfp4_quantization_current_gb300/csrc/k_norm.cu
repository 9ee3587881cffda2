// The root-mean-square norm ahead of a linear layer, with the residual's addition, and its gradient.
//
//   h = x + residual (rounded to its type once; h = x without a residual)
//   s = 1 / sqrt(mean(h^2) + eps) per row,   y = (h s) w
//   dx = s (g - v mean(g v)) + dh,  g = dy w,  v = h s,      dw = sum over rows of dy v
//
// The sums run in FP32 in an order fixed by the shape.  y is either stored
// (norm_add) or cast in registers to the rowwise 1x128 E4M3 copy
// (norm_q_blockwise; k_norm_cast.cu makes both copies).
#include "q_engine.cuh"
#include "q_internal.h"

namespace qk {

namespace {

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
                const float4 v = __ldg(reinterpret_cast<const float4 *>(p + j));
                f[j] = v.x, f[j + 1] = v.y, f[j + 2] = v.z, f[j + 3] = v.w;
            }
        } else {
#pragma unroll
            for (int j = 0; j < W; j++) f[j] = __ldg(p + j);
        }
    } else {
        const uint16_t *p = static_cast<const uint16_t *>(w) + k;
        if constexpr (W == 8) {
            const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p));
#pragma unroll
            for (int j = 0; j < 8; j++) f[j] = elem<BF16>(v, j);
        } else if constexpr (W == 4) {
            const uint2 v = __ldg(reinterpret_cast<const uint2 *>(p));
            f[0] = __uint_as_float(v.x << 16), f[1] = __uint_as_float(v.x & 0xFFFF0000u);
            f[2] = __uint_as_float(v.y << 16), f[3] = __uint_as_float(v.y & 0xFFFF0000u);
        } else {
#pragma unroll
            for (int j = 0; j < W; j++) f[j] = __uint_as_float((uint32_t)__ldg(p + j) << 16);
        }
    }
}

QD float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// Sum over the 2^gshift consecutive threads (gshift >= 5) that share a row, to
// all of them; part: a word per warp, used by no other call that is in flight.
// Every thread of the CTA calls it.
QD float row_sum(float v, float *part, int gshift)
{
    v = warp_sum(v);
    if (gshift == 5) return v;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = 1 << (gshift - 5);
    if (lane == 0) part[warp] = v;
    __syncthreads();
    return warp_sum(lane < n ? part[(warp & ~(n - 1)) + lane] : 0.0f);
}

QD float row_factor(float sum, int64_t K, float eps) { return __fdiv_rn(1.0f, __fsqrt_rn(__fdiv_rn(sum, (float)K) + eps)); }

// What is made of a row: y, its rowwise copy, or nothing (its factor, and its sum with the residual).
enum { kNormStore = 0, kNormCast = 1, kNormFactor = 2 };

// W elements of y from column k of the row that begins at element `base` (zeros where `in` is false): stored, or cast
// with the block of 128 that 128 / W lanes hold.  m: the largest |y| stored, where that is asked for.
template <int DT, int W, int MODE> QD void norm_put(const NormArgs &a, float (&y)[W], bool in, int64_t base, int64_t k, int lane, uint32_t &m)
{
    if constexpr (MODE == kNormStore) {
        if (a.amax != nullptr) {
            float b = 0.0f;
#pragma unroll
            for (int j = 0; j < W; j++) b = fmax_abs(b, y[j]);
            m = max(m, __float_as_uint(b) & 0x7FFFFFFFu);
        }
        Piece<DT, W> out;
        out.set(y);
        if (in) out.store(a.y, base + k);
    } else if constexpr (MODE == kNormCast) {
        static_assert(W >= 4, "rows of the copy are multiples of 128 elements");
        float b = 0.0f;
#pragma unroll
        for (int j = 0; j < W; j++) b = fmax_abs(b, y[j]);
        const uint32_t bits = group_max<128 / W>(__float_as_uint(b) & 0x7FFFFFFFu);
        const float alpha = alpha_from_amax(448.0f, __uint_as_float(bits));
#pragma unroll
        for (int j = 0; j < W; j++) y[j] = y[j] * alpha;
        if (!in) return;
        uint8_t *const q = a.q_row + base + k;
        if constexpr (W == 8) stg8(q, cvt_fp8x4<E4M3>(y[0], y[1], y[2], y[3]), cvt_fp8x4<E4M3>(y[4], y[5], y[6], y[7]));
        else stg4(q, cvt_fp8x4<E4M3>(y[0], y[1], y[2], y[3]));
        if (lane % (128 / W) == 0) {
            a.s_row[(base + k) / 128] = __fdiv_rn(1.0f, alpha);
            flag_nonfinite(a.status, bits);
        }
    }
}

// The largest stored |y|, over the CTA and into *amax: rounding is monotonic, so the largest value is rounded alone.
template <int DT> QD void norm_amax(const NormArgs &a, uint32_t m)
{
    if (DT == BF16) m = bf16_bits(__uint_as_float(m)) << 16;
    cta_max_to(m, reinterpret_cast<uint32_t *>(a.amax), a.status);
}

// A row to 2^gshift threads, the element pieces t, t + 2^gshift, ... of it in
// each thread's registers: read once, whatever is made of it.
template <int DT, int W, int VPT, int MODE, bool RES>
__global__ void __launch_bounds__(1024) k_norm_rows(const NormArgs a)
{
    __shared__ float part[32];
    const int g = 1 << a.gshift, t = threadIdx.x & (g - 1), lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * (blockDim.x >> a.gshift) + (threadIdx.x >> a.gshift);
    const bool live = row < a.M;
    const int K = (int)a.K;
    const int64_t base = row * a.K;
    constexpr bool kAhead = MODE != kNormFactor && VPT * W <= 16;   // weights on their way with the row, where registers allow
    Piece<DT, W> h[VPT];
    float w[kAhead ? VPT : 1][W];
    griddep_wait();   // nothing was read or written so far
    {
        Piece<DT, W> r[VPT];
#pragma unroll
        for (int i = 0; i < VPT; i++) {
            const int k = (t + i * g) * W;
            h[i].zero();
            if (RES) r[i].zero();
            if (live && k < K) {
                h[i].load(a.x, base + k);
                if (RES) r[i].load(a.residual, base + k);
            }
        }
        if constexpr (kAhead) {
#pragma unroll
            for (int i = 0; i < VPT; i++) {
                const int k = (t + i * g) * W;
                if (k < K) load_weights<W>(w[i], a.weight, a.wf32, k);
            }
        }
        if constexpr (RES) {
#pragma unroll
            for (int i = 0; i < VPT; i++) {
                const int k = (t + i * g) * W;
                float f[W];
#pragma unroll
                for (int j = 0; j < W; j++) f[j] = h[i].at(j) + r[i].at(j);
                h[i].set(f);
                if (live && k < K) h[i].store(a.h, base + k);
            }
        }
    }
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; i++)
#pragma unroll
        for (int j = 0; j < W; j++) sum = __fmaf_rn(h[i].at(j), h[i].at(j), sum);
    const float s = row_factor(row_sum(sum, part, a.gshift), K, a.eps);
    if (live && t == 0) a.rstd[row] = s;
    if constexpr (MODE == kNormFactor) return;
    uint32_t m = 0;   // largest |y| of this thread
#pragma unroll
    for (int i = 0; i < VPT; i++) {
        const int k = (t + i * g) * W;
        const bool in = live && k < K;
        float *const wi = w[kAhead ? i : 0];
        if (!kAhead && in) load_weights<W>(w[0], a.weight, a.wf32, k);
        float y[W];
#pragma unroll
        for (int j = 0; j < W; j++) y[j] = in ? h[i].at(j) * s * wi[j] : 0.0f;
        norm_put<DT, W, MODE>(a, y, in, base, k, lane, m);
    }
    if (MODE == kNormStore && a.amax != nullptr) norm_amax<DT>(a, m);
}

// Rows longer than the registers of a CTA: in two passes, the second over what
// the first has left in L2.
template <int DT, int W, int MODE, bool RES>
__global__ void __launch_bounds__(1024) k_norm_long(const NormArgs a)
{
    __shared__ float part[32];
    const int lane = threadIdx.x & 31;
    const int64_t base = (int64_t)blockIdx.x * a.K, step = 1024 * W;
    griddep_wait();   // nothing was read or written so far
    float sum = 0.0f;
    for (int64_t k = threadIdx.x * W; k < a.K; k += step) {
        Piece<DT, W> h, r;
        h.load(a.x, base + k);
        if constexpr (RES) {
            r.load(a.residual, base + k);
            float f[W];
#pragma unroll
            for (int j = 0; j < W; j++) f[j] = h.at(j) + r.at(j);
            h.set(f);
            h.store(a.h, base + k);
        }
#pragma unroll
        for (int j = 0; j < W; j++) sum = __fmaf_rn(h.at(j), h.at(j), sum);
    }
    const float s = row_factor(row_sum(sum, part, 10), a.K, a.eps);
    if (threadIdx.x == 0) a.rstd[blockIdx.x] = s;
    if constexpr (MODE == kNormFactor) return;
    const void *const from = RES ? a.h : a.x;
    uint32_t m = 0;
    for (int64_t k0 = 0; k0 < a.K; k0 += step) {   // whole warps: a block's lanes meet
        const int64_t k = k0 + threadIdx.x * W;
        const bool in = k < a.K;
        Piece<DT, W> h;
        float w[W], y[W];
        h.zero();
        if (in) {
            h.load(from, base + k);
            load_weights<W>(w, a.weight, a.wf32, k);
        }
#pragma unroll
        for (int j = 0; j < W; j++) y[j] = in ? h.at(j) * s * w[j] : 0.0f;
        norm_put<DT, W, MODE>(a, y, in, base, k, lane, m);
    }
    if (MODE == kNormStore && a.amax != nullptr) norm_amax<DT>(a, m);
}

// The gradient.  A row to 2^gshift threads as above; a thread keeps its columns over all rows of its walk, and with them
// its part of dw in registers, which it leaves as one row of `work`.
template <int DT, int W, int VPT, bool DH>
__global__ void __launch_bounds__(512) k_norm_grad(const NormGradArgs a)
{
    __shared__ float part[2][32];
    const int g = 1 << a.gshift, t = threadIdx.x & (g - 1), rows = blockDim.x >> a.gshift;
    const int K = (int)a.K;
    float w[VPT][W], dw[VPT][W];
    griddep_wait();   // nothing was read or written so far
#pragma unroll
    for (int i = 0; i < VPT; i++) {
        const int k = (t + i * g) * W;
#pragma unroll
        for (int j = 0; j < W; j++) w[i][j] = dw[i][j] = 0.0f;
        if (k < K) load_weights<W>(w[i], a.weight, a.wf32, k);
    }
    int flip = 0;
    for (int64_t row0 = (int64_t)blockIdx.x * rows; row0 < a.M; row0 += (int64_t)gridDim.x * rows, flip ^= 1) {
        const int64_t row = row0 + (threadIdx.x >> a.gshift), base = row * a.K;
        const bool live = row < a.M;
        const float s = live ? a.rstd[row] : 0.0f;
        Piece<DT, W> h[VPT], dy[VPT], dh[DH ? VPT : 1];
#pragma unroll
        for (int i = 0; i < VPT; i++) {
            const int k = (t + i * g) * W;
            h[i].zero();
            dy[i].zero();
            if (live && k < K) {
                dy[i].load(a.dy, base + k);
                h[i].load(a.h, base + k);
                if constexpr (DH) dh[i].load(a.dh, base + k);
            }
        }
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < VPT; i++)
#pragma unroll
            for (int j = 0; j < W; j++) {
                const float v = h[i].at(j) * s, d = dy[i].at(j);
                dw[i][j] = __fmaf_rn(d, v, dw[i][j]);
                sum = __fmaf_rn(d * w[i][j], v, sum);
            }
        const float c = __fdiv_rn(row_sum(sum, part[flip], a.gshift), (float)K);
#pragma unroll
        for (int i = 0; i < VPT; i++) {
            const int k = (t + i * g) * W;
            if (live && k < K) {
                float f[W];
#pragma unroll
                for (int j = 0; j < W; j++) {
                    const float v = h[i].at(j) * s, e = __fmaf_rn(-v, c, dy[i].at(j) * w[i][j]);
                    f[j] = DH ? __fmaf_rn(e, s, dh[DH ? i : 0].at(j)) : e * s;
                }
                Piece<DT, W> out;
                out.set(f);
                out.store(a.dx, base + k);
            }
        }
    }
    if (a.work == nullptr) return;
    float *const mine = a.work + ((int64_t)blockIdx.x * rows + (threadIdx.x >> a.gshift)) * a.K;
#pragma unroll
    for (int i = 0; i < VPT; i++) {
        const int k = (t + i * g) * W;
        if (k < K) {
            if constexpr (W % 4 == 0) {
#pragma unroll
                for (int j = 0; j < W; j += 4) *reinterpret_cast<float4 *>(mine + k + j) = make_float4(dw[i][j], dw[i][j + 1], dw[i][j + 2], dw[i][j + 3]);
            } else {
#pragma unroll
                for (int j = 0; j < W; j++) mine[k + j] = dw[i][j];
            }
        }
    }
}

// Longer rows: a CTA's part of dw is kept in its row of `work`.
template <int DT, int W, bool DH>
__global__ void __launch_bounds__(1024) k_norm_grad_long(const NormGradArgs a)
{
    __shared__ float part[2][32];
    float *const mine = a.work == nullptr ? nullptr : a.work + (int64_t)blockIdx.x * a.K;
    griddep_wait();   // nothing was read or written so far
    int flip = 0;
    for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x, flip ^= 1) {
        const int64_t base = row * a.K;
        const float s = a.rstd[row];
        float sum = 0.0f;
        for (int64_t k = threadIdx.x * W; k < a.K; k += 1024 * W) {
            Piece<DT, W> h, dy;
            float w[W];
            dy.load(a.dy, base + k);
            h.load(a.h, base + k);
            load_weights<W>(w, a.weight, a.wf32, k);
#pragma unroll
            for (int j = 0; j < W; j++) sum = __fmaf_rn(dy.at(j) * w[j], h.at(j) * s, sum);
        }
        const float c = __fdiv_rn(row_sum(sum, part[flip], 10), (float)a.K);
        for (int64_t k = threadIdx.x * W; k < a.K; k += 1024 * W) {
            Piece<DT, W> h, dy, dh, out;
            float w[W], f[W];
            dy.load(a.dy, base + k);
            h.load(a.h, base + k);
            if constexpr (DH) dh.load(a.dh, base + k);
            load_weights<W>(w, a.weight, a.wf32, k);
#pragma unroll
            for (int j = 0; j < W; j++) {
                const float v = h.at(j) * s, e = __fmaf_rn(-v, c, dy.at(j) * w[j]);
                f[j] = DH ? __fmaf_rn(e, s, dh.at(j)) : e * s;
                if (mine != nullptr) mine[k + j] = __fmaf_rn(dy.at(j), v, row == blockIdx.x ? 0.0f : mine[k + j]);
            }
            out.set(f);
            out.store(a.dx, base + k);
        }
    }
}

// dw: the rows of `work`, added in the same order every time (eight walks of every eighth row, then the walks).
__global__ void __launch_bounds__(256) k_norm_dw(const float *work, int64_t parts, int64_t K, void *dw, bool f32)
{
    __shared__ float sums[8][32];
    const int c = threadIdx.x & 31, walk = threadIdx.x >> 5;
    const int64_t k = (int64_t)blockIdx.x * 32 + c;
    griddep_wait();
    float sum = 0.0f;
    if (k < K)
        for (int64_t p = walk; p < parts; p += 8) sum += work[p * K + k];
    sums[walk][c] = sum;
    __syncthreads();
    if (walk == 0 && k < K) {
#pragma unroll
        for (int i = 1; i < 8; i++) sum += sums[i][c];
        if (f32) static_cast<float *>(dw)[k] = sum;
        else static_cast<uint16_t *>(dw)[k] = (uint16_t)bf16_bits(sum);
    }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------

int log2_up(int64_t n)
{
    int s = 0;
    while (((int64_t)1 << s) < n) s++;
    return s;
}

template <int DT, int W, int VPT, int MODE> cudaError_t norm_rows(NormArgs a, int gshift, cudaStream_t st)
{
    a.gshift = gshift;
    const int threads = gshift < 8 ? 256 : 1 << gshift, rows = threads >> gshift;
    const int64_t grid = (a.M + rows - 1) / rows;
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    return launch_k(true, a.residual != nullptr ? k_norm_rows<DT, W, VPT, MODE, true> : k_norm_rows<DT, W, VPT, MODE, false>,
                    dim3((unsigned)grid), dim3(threads), 0, st, a);
}

template <int DT, int W, int MODE> cudaError_t norm_w(const NormArgs &a, cudaStream_t st)
{
    constexpr int E = W == 1 ? 4 : 8;   // elements of a thread, times 1, 2 or 4
    const int64_t pieces = (a.K + W - 1) / W;
    const int s1 = log2_up((pieces + E / W - 1) / (E / W)), s2 = log2_up((pieces + 2 * E / W - 1) / (2 * E / W)),
              s4 = log2_up((pieces + 4 * E / W - 1) / (4 * E / W));
    if (s1 <= 5) return norm_rows<DT, W, E / W, MODE>(a, 5, st);
    if (s2 <= 10) return norm_rows<DT, W, 2 * E / W, MODE>(a, s2 < 5 ? 5 : s2, st);
    if (s4 <= 10) return norm_rows<DT, W, 4 * E / W, MODE>(a, s4, st);
    if (a.M > INT32_MAX) return cudaErrorInvalidValue;
    return launch_k(true, a.residual != nullptr ? k_norm_long<DT, W, MODE, true> : k_norm_long<DT, W, MODE, false>,
                    dim3((unsigned)a.M), dim3(1024), 0, st, a);
}

template <int DT, int MODE> cudaError_t norm_t(const NormArgs &a, cudaStream_t st)
{
    if constexpr (MODE != kNormCast) {
        if (a.K % In<DT>::VEC != 0) return norm_w<DT, 1, MODE>(a, st);
    }
    return norm_w<DT, In<DT>::VEC, MODE>(a, st);
}

// How a gradient's rows are laid out: threads of a row (2^gshift; 0: the loop over long rows), CTAs, and rows of `work`.
struct GradPlan {
    int gshift, vpt, threads, ctas, parts;
};
GradPlan grad_plan(int64_t M, int64_t K, int dt)
{
    const int vec = dt == BF16 ? 8 : 4, W = K % vec == 0 ? vec : 1;
    const int64_t pieces = (K + W - 1) / W;
    GradPlan p = {};
    // elements of a thread: 4 or 16 single ones, 8 or 16 in pieces
    for (const int E : {W == 1 ? 4 : 8, 16}) {
        const int s = log2_up((pieces + E / W - 1) / (E / W));
        if (s > (E == 16 ? 9 : 8)) continue;
        p.gshift = s < 5 ? 5 : s;
        p.vpt = E / W;
        break;
    }
    p.threads = p.gshift == 0 ? 1024 : p.gshift < 8 ? 256 : 1 << p.gshift;
    const int rows = p.gshift == 0 ? 1 : p.threads >> p.gshift;
    const int64_t most = p.threads == 256 ? 608 : p.threads == 512 ? 304 : 152, need = (M + rows - 1) / rows;
    p.ctas = (int)(need < most ? need : most);
    p.parts = p.ctas * rows;
    return p;
}

template <int DT, int W, int VPT> cudaError_t grad_rows(const NormGradArgs &a, const GradPlan &p, cudaStream_t st)
{
    return launch_k(true, a.dh != nullptr ? k_norm_grad<DT, W, VPT, true> : k_norm_grad<DT, W, VPT, false>, dim3(p.ctas),
                    dim3(p.threads), 0, st, a);
}

template <int DT, int W> cudaError_t grad_w(const NormGradArgs &a, const GradPlan &p, cudaStream_t st)
{
    constexpr int V = W == 1 ? 4 : 8 / W;
    if (p.gshift == 0)
        return launch_k(true, a.dh != nullptr ? k_norm_grad_long<DT, W, true> : k_norm_grad_long<DT, W, false>, dim3(p.ctas),
                        dim3(p.threads), 0, st, a);
    return p.vpt == V ? grad_rows<DT, W, V>(a, p, st) : grad_rows<DT, W, 16 / W>(a, p, st);
}

}  // namespace

cudaError_t launch_norm_add(const NormArgs &a, int dt, cudaStream_t st)
{
    if (a.amax != nullptr) {
        const cudaError_t e = launch_zero_word(a.amax, st);
        if (e != cudaSuccess) return e;
    }
    return dt == BF16 ? norm_t<BF16, kNormStore>(a, st) : norm_t<F32, kNormStore>(a, st);
}

cudaError_t launch_norm_cast_rows(const NormArgs &a, int dt, cudaStream_t st)
{
    if (a.q_row == nullptr) return dt == BF16 ? norm_t<BF16, kNormFactor>(a, st) : norm_t<F32, kNormFactor>(a, st);
    return dt == BF16 ? norm_t<BF16, kNormCast>(a, st) : norm_t<F32, kNormCast>(a, st);
}

int64_t norm_grad_rows(int64_t M, int64_t K, int dt) { return grad_plan(M, K, dt).parts; }

cudaError_t launch_norm_grad(NormGradArgs a, int dt, void *dw, cudaStream_t st)
{
    const GradPlan p = grad_plan(a.M, a.K, dt);
    a.gshift = p.gshift;
    if (dw == nullptr) a.work = nullptr;
    const bool vec = a.K % (dt == BF16 ? 8 : 4) == 0;
    cudaError_t e = dt == BF16 ? (vec ? grad_w<BF16, 8>(a, p, st) : grad_w<BF16, 1>(a, p, st))
                               : (vec ? grad_w<F32, 4>(a, p, st) : grad_w<F32, 1>(a, p, st));
    if (e != cudaSuccess || dw == nullptr) return e;
    return launch_k(true, k_norm_dw, dim3((unsigned)((a.K + 31) / 32)), dim3(256), 0, st, (const float *)a.work, (int64_t)p.parts,
                    a.K, dw, a.wf32);
}

}  // namespace qk
