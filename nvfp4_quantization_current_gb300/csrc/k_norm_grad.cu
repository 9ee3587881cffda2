// The gradient of the norm ahead of a linear layer (k_norm.cu), per row with
// v = h s and g = dy w
//   dx = s (g - v mean(g v)) + dh,      dw = sum over rows of dy v
// The sums run in FP32 in an order that the shape, the type and whether there is dh fix.  Bound by memory: dy, h and dh
// are read and dx written once, and a CTA's part of dw is a row of scratch that a
// second, small kernel adds up.  Measured on a GB300, in graphs of calls: 8192 x 4096
// BF16 with dh 46.5 to 47.3 us (268 MB at 5.7 to 5.8 TB/s; 41.3 without dw, whose kernel
// waits for the last CTA), without dh 37.2, 3001 x 1111 FP32 11.4 to 13.5 (8.0
// without dw).  One row per CTA at a time, loaded where it is used, took 66.6 and 36.7.
#include "q_norm.cuh"

namespace qk {

namespace {

// The gradient.  The rows of dy, h and dh come by bulk copies into a ring of
// shared memory, so that memory stays busy while rows are summed: a step is R rows,
// each over all threads of the CTA, or 8 R short ones, R for a warp (where E is 8), E
// elements per thread in pieces of W.  A thread keeps its columns over all steps, and with them its part of
// dw in registers, which it leaves as one row of `work`.  Rows that begin between
// 16-byte boundaries are copied with the bytes around them (a 16-byte piece that holds
// one of the row's bytes is the allocation's) and read an element at a time.
template <int DT, int W, int E, int R, bool DH>
__global__ void __launch_bounds__(512) k_norm_grad(const NormGradArgs a, int stages, int stage_bytes)
{
    constexpr bool kWarpRows = E == 8;
    constexpr int VPT = E / W, kMostStages = 8, ES = In<DT>::BYTES, kTensors = DH ? 3 : 2;
    extern __shared__ __align__(128) uint8_t dsm[];
    __shared__ float part[2][R][16];
    __shared__ __align__(8) uint64_t full[kMostStages];
    const int lane = threadIdx.x & 31, rows = kWarpRows ? 8 * R : R;
    const int T = kWarpRows ? 32 : blockDim.x, t = kWarpRows ? lane : threadIdx.x, mine = kWarpRows ? (threadIdx.x >> 5) * R : 0;   // the first row
    const int K = (int)a.K, tensor_bytes = stage_bytes / kTensors;
    const int64_t steps_all = (a.M + rows - 1) / rows;
    const int64_t steps = steps_all > blockIdx.x ? (steps_all - blockIdx.x + gridDim.x - 1) / gridDim.x : 0;
    // step i of this CTA: rows from row0(i) on, whose bytes begin `skew` into their copies
    auto row0 = [&](int64_t i) { return ((int64_t)blockIdx.x + i * gridDim.x) * rows; };
    auto skew = [&](int64_t row) { return W > 1 ? 0 : (int)((row * K * ES) & 15); };
    const uint64_t policy = l2_policy(a.once);
    auto issue = [&](int64_t i) {
        const int64_t r0 = row0(i), n = a.M - r0 < rows ? a.M - r0 : rows;
        const int off = skew(r0);
        const uint32_t bytes = (uint32_t)(off + n * K * ES + 15) & ~15u;
        const int s = (int)(i % stages);
        uint8_t *const st = dsm + (int64_t)s * stage_bytes;
        mbar_arrive_expect_tx(&full[s], bytes * kTensors);
        const int64_t from = r0 * K * ES - off;
        bulk_load(st, static_cast<const char *>(a.dy) + from, bytes, &full[s], policy);
        bulk_load(st + tensor_bytes, static_cast<const char *>(a.h) + from, bytes, &full[s], policy);
        if constexpr (DH) bulk_load(st + 2 * tensor_bytes, static_cast<const char *>(a.dh) + from, bytes, &full[s], policy);
    };
    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; s++) mbar_init(&full[s], 1);
        fence_mbar_init();
    }
    __syncthreads();
    griddep_wait();   // nothing was read or written so far
    if (threadIdx.x == 0)
        for (int64_t i = 0; i < steps && i < stages; i++) issue(i);
    // The weights too, where registers allow; else they are loaded (from L1) where they are used.
    constexpr bool kHeld = E <= 16;
    float w[kHeld ? VPT : 1][W], dw[VPT][W];
#pragma unroll
    for (int i = 0; i < VPT; i++) {
        const int k = (t + i * T) * W;
#pragma unroll
        for (int j = 0; j < W; j++) w[kHeld ? i : 0][j] = dw[i][j] = 0.0f;
        if (kHeld && k < K) load_weights<W>(w[kHeld ? i : 0], a.weight, a.wf32, k);
    }
    const float inv = __fdiv_rn(1.0f, (float)K);
    int s = 0;
    uint32_t parity = 0;
    for (int64_t n = 0; n < steps; n++) {
        const int64_t r0 = row0(n) + mine;
        float f[R];
#pragma unroll
        for (int r = 0; r < R; r++) f[r] = r0 + r < a.M ? load_float(a.rstd + r0 + r) : 0.0f;
        const uint8_t *const st = dsm + (int64_t)s * stage_bytes + skew(row0(n)) + (int64_t)mine * K * ES;
        const bool ok = !a.give_up && mbar_wait_bounded(&full[s], parity);
        Piece<DT, W> h[R][VPT], dy[R][VPT], dh[DH ? R : 1][DH ? VPT : 1];
        float c[R];
#pragma unroll
        for (int r = 0; r < R; r++) {
            const uint8_t *const at = st + r * K * ES;
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < VPT; i++) {
                const int k = (t + i * T) * W;
                h[r][i].zero();
                dy[r][i].zero();
                if (r0 + r < a.M && k < K) {
                    dy[r][i].shared(at, k);
                    h[r][i].shared(at + tensor_bytes, k);
                    if constexpr (DH) dh[r][i].shared(at + 2 * tensor_bytes, k);
                    if (!kHeld) load_weights<W>(w[0], a.weight, a.wf32, k);
                }
#pragma unroll
                for (int j = 0; j < W; j++) {
                    const float v = h[r][i].at(j) * f[r], d = dy[r][i].at(j);
                    dw[i][j] = __fmaf_rn(d, v, dw[i][j]);
                    sum = __fmaf_rn(d * w[kHeld ? i : 0][j], v, sum);
                }
            }
            c[r] = sum;
        }
        // the rows' sums, and word that a wait ran out (no thread waits for another step then)
#pragma unroll
        for (int r = 0; r < R; r++) {
            c[r] = warp_sum(c[r]);
            if (!kWarpRows && lane == 0) part[n & 1][r][threadIdx.x >> 5] = c[r];
        }
        const bool stop = __syncthreads_or(!ok);
#pragma unroll
        for (int r = 0; r < R; r++) {
            if (!kWarpRows) c[r] = warp_sum(lane < (int)(blockDim.x >> 5) ? part[n & 1][r][lane] : 0.0f);
            c[r] *= inv;
        }
        if (stop) {   // the copies in flight land before shared memory goes away
            if (threadIdx.x == 0) {
                for (int64_t j = n; j < steps && j < n + stages; j++) (void)mbar_wait_bounded(&full[j % stages], (uint32_t)((j / stages) & 1));
                if (a.status != nullptr) atomicOr(a.status, kStTimeout);
            }
            break;
        }
        if (threadIdx.x == 0 && n + stages < steps) {   // every thread has the stage in its registers
            fence_proxy_async();
            issue(n + stages);
        }
#pragma unroll
        for (int r = 0; r < R; r++) {
#pragma unroll
            for (int i = 0; i < VPT; i++) {
                const int k = (t + i * T) * W;
                if (r0 + r >= a.M || k >= K) continue;
                float o[W];
                if (!kHeld) load_weights<W>(w[0], a.weight, a.wf32, k);
#pragma unroll
                for (int j = 0; j < W; j++) {
                    const float v = h[r][i].at(j) * f[r], e = __fmaf_rn(-v, c[r], dy[r][i].at(j) * w[kHeld ? i : 0][j]);
                    o[j] = DH ? __fmaf_rn(e, f[r], dh[DH ? r : 0][DH ? i : 0].at(j)) : e * f[r];
                }
                Piece<DT, W> out;
                out.set(o);
                out.store(a.dx, (r0 + r) * K + k);
            }
        }
        if (++s == stages) {
            s = 0;
            parity ^= 1;
        }
    }
    if (a.work == nullptr) return;
    // one row of `work`: the CTA's only part, or the sum of eight, which meet where the rows were
    float *const to = !kWarpRows ? a.work + (int64_t)blockIdx.x * K : reinterpret_cast<float *>(dsm) + (threadIdx.x >> 5) * K;
    if (kWarpRows) __syncthreads();
#pragma unroll
    for (int i = 0; i < VPT; i++) {
        const int k = (t + i * T) * W;
        if (k < K) {
            if constexpr (W % 4 == 0) {
#pragma unroll
                for (int j = 0; j < W; j += 4) *reinterpret_cast<float4 *>(to + k + j) = make_float4(dw[i][j], dw[i][j + 1], dw[i][j + 2], dw[i][j + 3]);
            } else {
#pragma unroll
                for (int j = 0; j < W; j++) to[k + j] = dw[i][j];
            }
        }
    }
    if (kWarpRows) {
        __syncthreads();
        for (int k = threadIdx.x; k < K; k += blockDim.x) {
            float sum = reinterpret_cast<const float *>(dsm)[k];
            for (int r = 1; r < 8; r++) sum += reinterpret_cast<const float *>(dsm)[r * K + k];
            a.work[(int64_t)blockIdx.x * K + k] = sum;
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
        const float s = load_float(a.rstd + row);
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
        const float c = __fdiv_rn(row_sum(sum, part[flip], 0, 32), (float)a.K);
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

// dw: the rows of `work`, added in the same order every time: 64 walks of every 64th row, then the walks.
__global__ void __launch_bounds__(1024) k_norm_dw(const float *work, int64_t parts, int64_t K, void *dw, bool f32)
{
    __shared__ float sums[64][17];
    const int c = threadIdx.x & 15, walk = threadIdx.x >> 4, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t k = (int64_t)blockIdx.x * 16 + c;
    griddep_wait();
    float sum = 0.0f;
    if (k < K) {
#pragma unroll 8
        for (int64_t p = walk; p < parts; p += 64) sum += load_float(work + p * K + k);
    }
    sums[walk][c] = sum;
    __syncthreads();
    if (warp >= 16) return;
    sum = warp_sum(sums[lane][warp] + sums[lane + 32][warp]);   // the walks of column `warp`
    const int64_t at = (int64_t)blockIdx.x * 16 + warp;
    if (lane == 0 && at < K) {
        if (f32) static_cast<float *>(dw)[at] = sum;
        else static_cast<uint16_t *>(dw)[at] = (uint16_t)bf16_bits(sum);
    }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------

// How a gradient's rows are laid out: rows of a step, elements of a thread (0: the loop over long rows), threads, CTAs,
// and the ring.  Two rows a step share a reduction (8192 x 4096 BF16 without dh 41.8 us
// at one, 37.8 at two), unless they spill (with dh 46.4 and 52.3, and dw's 3 in each);
// 16 elements a thread beat 8 on twice the threads (46.8 and 56.7).
struct GradPlan {
    int rows, elements, threads, ctas, stages, stage_bytes;
};
GradPlan grad_plan(int64_t M, int64_t K, int dt, bool dh)
{
    const int es = dt == BF16 ? 2 : 4, tensors = dh ? 3 : 2;
    GradPlan p = {1, 0, 1024, 0, 0, 0};
    // The shared memory of an SM holds the rings of all CTAs, two steps in each at least.
    auto copy_bytes = [&](int rows) { return (rows * K * es + 15) / 16 * 16 + (K * es % 16 != 0 ? 16 : 0); };   // and what lies around the rows
    int per_sm = 1;
    if (K <= 256) {
        p.rows = 32;
        p.elements = 8;
        p.threads = 256;
        per_sm = 2;
    } else if (K <= 16384 && 2 * tensors * copy_bytes(1) <= kRingBytes) {
        p.elements = K <= 8192 ? 16 : 32;
        p.threads = (int)((K + 32 * p.elements - 1) / (32 * p.elements)) * 32;
        p.rows = p.elements == 16 && !dh && K * es % 16 == 0 && 4 * tensors * copy_bytes(2) <= kRingBytes ? 2 : 1;
        per_sm = 512 / p.threads < 8 ? 512 / p.threads : 8;
    }
    if (p.elements != 0) {
        p.stage_bytes = tensors * (int)copy_bytes(p.rows);
        const int fits = kRingBytes / (2 * p.stage_bytes);
        per_sm = per_sm > fits ? fits : per_sm;
        p.stages = kRingBytes / per_sm / p.stage_bytes;
        if (p.stages > 8) p.stages = 8;
    }
    const int64_t most = (int64_t)per_sm * 152, need = (M + p.rows - 1) / p.rows;
    p.ctas = (int)(need < most ? need : most);
    return p;
}

template <int DT, int W, int E, int R, bool DH> cudaError_t grad_rows(const NormGradArgs &a, const GradPlan &p, cudaStream_t st)
{
    const cudaError_t e = engine_smem_ready<k_norm_grad<DT, W, E, R, DH>>(kRingBytes, true);
    if (e != cudaSuccess) return e;
    return launch_k(true, k_norm_grad<DT, W, E, R, DH>, dim3(p.ctas), dim3(p.threads), (size_t)p.stages * p.stage_bytes, st, a,
                    p.stages, p.stage_bytes);
}

template <int DT, int W, bool DH> cudaError_t grad_w(const NormGradArgs &a, const GradPlan &p, cudaStream_t st)
{
    switch (p.elements) {
    case 8: return grad_rows<DT, W, 8, 4, DH>(a, p, st);
    case 16:
        if constexpr (!DH && W > 1)
            if (p.rows == 2) return grad_rows<DT, W, 16, 2, DH>(a, p, st);
        return grad_rows<DT, W, 16, 1, DH>(a, p, st);
    case 32: return grad_rows<DT, W, 32, 1, DH>(a, p, st);
    default: return launch_k(true, k_norm_grad_long<DT, W, DH>, dim3(p.ctas), dim3(p.threads), 0, st, a);
    }
}

template <int DT> cudaError_t grad_t(const NormGradArgs &a, const GradPlan &p, cudaStream_t st)
{
    constexpr int VEC = In<DT>::VEC;
    if (a.K % VEC != 0) return a.dh != nullptr ? grad_w<DT, 1, true>(a, p, st) : grad_w<DT, 1, false>(a, p, st);
    return a.dh != nullptr ? grad_w<DT, VEC, true>(a, p, st) : grad_w<DT, VEC, false>(a, p, st);
}

}  // namespace

int64_t norm_grad_rows(int64_t M, int64_t K, int dt)
{
    // enough with dh and without it
    const GradPlan p = grad_plan(M, K, dt, false), q = grad_plan(M, K, dt, true);
    return p.ctas > q.ctas ? p.ctas : q.ctas;
}

cudaError_t launch_norm_grad(NormGradArgs a, int dt, void *dw, cudaStream_t st)
{
    const GradPlan p = grad_plan(a.M, a.K, dt, a.dh != nullptr);
    if (dw == nullptr) a.work = nullptr;
    // Inputs that L2 does not hold (129 MB) make way for what it could keep: 8192 x 4096 BF16 with dh 47.1 -> 46.5 us, without
    // dw 42.7 -> 41.3; those that it does hold stay (3001 x 1111 FP32, inputs of 27 MB met again 11.4, as if used once 13.3).
    a.once = a.M * a.K * (dt == BF16 ? 2 : 4) * (a.dh != nullptr ? 3 : 2) > ((int64_t)96 << 20);
    const cudaError_t e = dt == BF16 ? grad_t<BF16>(a, p, st) : grad_t<F32>(a, p, st);
    if (e != cudaSuccess || dw == nullptr) return e;
    return launch_k(true, k_norm_dw, dim3((unsigned)((a.K + 15) / 16)), dim3(1024), 0, st, (const float *)a.work,
                    (int64_t)p.ctas, a.K, dw, a.wf32);
}

}  // namespace qk
