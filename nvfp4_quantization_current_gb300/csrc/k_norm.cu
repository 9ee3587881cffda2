// The root-mean-square norm ahead of a linear layer, with the residual's addition.
//
//   h = x + residual (rounded to its type once; h = x without a residual)
//   s = 1 / sqrt(mean(h^2) + eps) per row,   y = (h s) w
//
// The sums run in FP32 in an order that the row's length and type fix, so that a row's
// result is the same in every call.  y is either stored
// (norm_add) or cast in registers to the rowwise 1x128 E4M3 copy
// (norm_q_blockwise; k_norm_cast.cu makes the transposed one from h and s).  All of it
// is bound by memory, and a row is read once: it stays in registers between its sum
// and what is made of it.  Measured on a GB300, in graphs of calls: 8192 x 4096 BF16
// with a residual 42.4 us (268 MB at 6.3 TB/s, a copy's rate being 6.8), without one
// 20.4 to 20.8, in FP32 78.6 to 79.9; its rowwise copy 39 with a residual, 26.2 without (with one,
// 338 warp instructions for 512 elements: issue slots 54 % in use, DRAM 72 %, at 16384 x
// 4096); 16 rows 1.9 to 2.2.
#include "q_norm.cuh"

namespace qk {

namespace {

// The sum of squares of a thread's pieces.  Of 16 single elements, which two threads may share (k_norm_rows), the
// even and the odd ones are summed apart first.
template <int DT, int W, int N> QD float squares(const Piece<DT, W> (&h)[N])
{
    float sum = 0.0f, odd = 0.0f;
    if constexpr (W > 1) {
        uint64_t two = 0;
#pragma unroll
        for (int i = 0; i < N; i++)
#pragma unroll
            for (int j = 0; j < W / 2; j++) two = ffma2(h[i].pair(j), h[i].pair(j), two);
        unpack2(two, sum, odd);
        sum += odd;
    } else {
#pragma unroll
        for (int i = 0; i < N; i++) {
            float &to = N == 16 && i % 2 ? odd : sum;
            to = __fmaf_rn(h[i].at(0), h[i].at(0), to);
        }
        if (N == 16) sum += odd;
    }
    return sum;
}

// 1 / sqrt(sum / K + eps): the approximate root's reciprocal (two units in the last place) after one step of Newton's
// iteration, which squares its error; every thread of a row takes it, and a division, a
// root and a division are some 60 instructions.  A v of zero, infinity or NaN goes
// as it is (the step would make NaNs of the first two).
QD float row_factor(float sum, float inv, float eps)
{
    const float v = __fmaf_rn(sum, inv, eps), y = rsqrtf(v);
    const float e = __fmaf_rn(-(v * y), y, 1.0f);
    return v > 0.0f && v < __int_as_float(0x7F800000) ? __fmaf_rn(0.5f * y, e, y) : y;
}

// What is made of a row: y, its rowwise copy, or nothing (its factor, and its sum with the residual).
enum { kNormStore = 0, kNormCast = 1, kNormFactor = 2 };

// W elements of y to column k of the row that begins at element `base`.  m: the largest |y| stored, where that is asked for.
template <int DT, int W> QD void norm_put(const NormArgs &a, const float (&y)[W], bool in, int64_t base, int64_t k, uint32_t &m)
{
    if (a.amax != nullptr) {
        float b = 0.0f;
#pragma unroll
        for (int j = 0; j < W; j++) b = fmax_abs(b, y[j]);
        if (in) m = max(m, __float_as_uint(b) & 0x7FFFFFFFu);
    }
    Piece<DT, W> out;
    out.set(y);
    if (in) out.store(a.y, base + k);
}

// y = (h s) w.
template <int DT, int W> QD void norm_y(float (&y)[W], const Piece<DT, W> &h, float s, const float (&w)[W])
{
    if constexpr (W > 1) {
        const uint64_t ss = pack2(__float_as_uint(s), __float_as_uint(s));
#pragma unroll
        for (int j = 0; j < W; j += 2)
            unpack2(fmul2(fmul2(h.pair(j / 2), ss), pack2(__float_as_uint(w[j]), __float_as_uint(w[j + 1]))), y[j], y[j + 1]);
    } else {
        y[0] = h.at(0) * s * w[0];
    }
}

// The rowwise copy of N pieces of W elements of y, from column k0 + i step on each, to the row's codes and scales: N blocks
// of 128, each of which LPB = 128 / W lanes share (and lie in the row, or outside it, together).  The N maxima are reduced
// over the lanes by a halving exchange, after which each lane holds one block's, takes its quotients once, and the alphas go
// back by index shuffles.
template <int W, int N> QD void norm_cast(const NormArgs &a, float (&y)[N][W], uint8_t *q, float *s, int k0, int step, int lane)
{
    static_assert(W >= 4, "rows of the copy are multiples of 128 elements");
    constexpr int LPB = 128 / W;
    static_assert(N <= LPB, "a lane holds one block at most");
    uint32_t m[N];
#pragma unroll
    for (int i = 0; i < N; i++) {
        float b = fmax_abs(fmax_abs(y[i][0], y[i][1]), fmax_abs(y[i][2], y[i][3]));
        if constexpr (W == 8) b = fmax_abs(b, fmax_abs(fmax_abs(y[i][4], y[i][5]), fmax_abs(y[i][6], y[i][7])));
        m[i] = __float_as_uint(b) & 0x7FFFFFFFu;
    }
    int o = LPB / 2;
#pragma unroll
    for (int n = N; n > 1; n /= 2, o /= 2)
#pragma unroll
        for (int i = 0; i < n / 2; i++) {
            const bool up = lane & o;
            const uint32_t mine = up ? m[i + n / 2] : m[i], other = up ? m[i] : m[i + n / 2];
            m[i] = max(mine, __shfl_xor_sync(0xFFFFFFFFu, other, o));
        }
#pragma unroll
    for (; o > 0; o /= 2) m[0] = max(m[0], __shfl_xor_sync(0xFFFFFFFFu, m[0], o));
    const float alpha = alpha_from_amax(448.0f, __uint_as_float(m[0]));
    const int k = k0 + (lane % LPB) / (LPB / N) * step, K = (int)a.K;   // of the piece in this lane's block
    if (lane % (LPB / N) == 0 && k < K) {
        s[k / 128] = __fdiv_rn(1.0f, alpha);
        flag_nonfinite(a.status, m[0]);
    }
#pragma unroll
    for (int i = 0; i < N; i++) {
        const float f = N == 1 ? alpha : __shfl_sync(0xFFFFFFFFu, alpha, (lane & ~(LPB - 1)) + i * (LPB / N));
#pragma unroll
        for (int j = 0; j < W; j += 2) mul2(y[i][j], y[i][j + 1], f, f);
        if (k0 + i * step < K) {
            uint8_t *const to = q + k0 + i * step;
            if constexpr (W == 8) stg8(to, cvt_fp8x4<E4M3>(y[i][0], y[i][1], y[i][2], y[i][3]), cvt_fp8x4<E4M3>(y[i][4], y[i][5], y[i][6], y[i][7]));
            else stg4(to, cvt_fp8x4<E4M3>(y[i][0], y[i][1], y[i][2], y[i][3]));
        }
    }
}

// The largest stored |y|, over the CTA and into *amax: rounding is monotonic, so the largest value is rounded alone.
template <int DT> QD void norm_amax(const NormArgs &a, uint32_t m)
{
    if (DT == BF16) m = bf16_bits(__uint_as_float(m)) << 16;
    cta_max_to(m, reinterpret_cast<uint32_t *>(a.amax), a.status);
}

// A row to T threads (whole warps), the element pieces t, t + T, ... of it in
// each thread's registers: read once, whatever is made of it.  Of rows of up to 8192
// single elements a thread takes eight (16 take 5.2 us of 16 x 1111 BF16, eight 3.2), threads t and t + T / 2 what a
// thread of the ring takes.
template <int DT, int W, int VPT, int MODE, bool RES>
__global__ void __launch_bounds__(1024) k_norm_rows(const NormArgs a)
{
    constexpr bool kHalves = W == 1 && VPT == 8;
    __shared__ float part[32], upper[kHalves ? 512 : 1];
    // this thread's row of the CTA's: its warp by the warps of a row (of 32 at most, so that 16 bits of the quotient do)
    constexpr bool kWhole = VPT * W == 32;   // the longest rows: all threads of the largest CTA (numbers that are known spare registers)
    const int T = kWhole ? 1024 : a.row_threads, mine = kWhole ? 0 : (int)((threadIdx.x >> 5) * a.per_warps >> 16);
    const int t = threadIdx.x - mine * T, lane = threadIdx.x & 31;
    const int64_t row = kWhole ? blockIdx.x : (int64_t)blockIdx.x * a.cta_rows + mine;
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
            const int k = (t + i * T) * W;
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
                const int k = (t + i * T) * W;
                if (k < K) load_weights<W>(w[i], a.weight, a.wf32, k);
            }
        }
        if constexpr (RES) {
#pragma unroll
            for (int i = 0; i < VPT; i++) {
                const int k = (t + i * T) * W;
                h[i].add(r[i]);
                if (live && k < K) h[i].store(a.h, base + k);
            }
        }
    }
    float sum = squares<DT, W, VPT>(h);
    if constexpr (kHalves) {
        const int half = T >> 1, at = mine * half + t;
        if (t >= half) upper[at - half] = sum;
        __syncthreads();
        if (t < half) {
            sum = warp_sum(sum + upper[at]);
            if (lane == 0) part[threadIdx.x >> 5] = sum;
        }
        __syncthreads();
        sum = warp_sum(lane < half >> 5 ? part[mine * (T >> 5) + lane] : 0.0f);
    } else {
        sum = row_sum(sum, part, mine * (T >> 5), T >> 5);
    }
    const float s = row_factor(sum, a.inv, a.eps);
    if (live && t == 0) a.rstd[row] = s;
    if constexpr (MODE == kNormFactor) return;
    if constexpr (MODE == kNormCast && kAhead) {
        float y[VPT][W];
#pragma unroll
        for (int i = 0; i < VPT; i++) norm_y<DT, W>(y[i], h[i], s, w[i]);
        if (live) norm_cast<W, VPT>(a, y, a.q_row + base, a.s_row + row * (K / 128), t * W, T * W, lane);   // a warp's rows are live together
        return;
    }
    uint32_t m = 0;   // largest |y| of this thread
#pragma unroll
    for (int i = 0; i < VPT; i++) {
        const int k = (t + i * T) * W;
        const bool in = live && k < K;
        if (!kAhead && in) load_weights<W>(w[0], a.weight, a.wf32, k);
        float y[1][W];
        norm_y<DT, W>(y[0], h[i], s, w[kAhead ? i : 0]);
        if constexpr (MODE == kNormCast) norm_cast<W, 1>(a, y, a.q_row + base, a.s_row + row * (K / 128), in ? k : K, 0, lane);
        else norm_put<DT, W>(a, y[0], in, base, k, m);
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
    const float s = row_factor(row_sum(sum, part, 0, 32), a.inv, a.eps);
    if (threadIdx.x == 0) a.rstd[blockIdx.x] = s;
    if constexpr (MODE == kNormFactor) return;
    const void *const from = RES ? a.h : a.x;
    uint32_t m = 0;
    for (int64_t k0 = 0; k0 < a.K; k0 += step) {   // whole warps: a block's lanes meet
        const int64_t k = k0 + threadIdx.x * W;
        const bool in = k < a.K;
        Piece<DT, W> h;
        float w[W], y[1][W];
        h.zero();
        if (in) {
            h.load(from, base + k);
            load_weights<W>(w, a.weight, a.wf32, k);
        }
        norm_y<DT, W>(y[0], h, s, w);
        if constexpr (MODE == kNormCast) norm_cast<W, 1>(a, y, a.q_row + base, a.s_row + blockIdx.x * (a.K / 128), (int)(in ? k : a.K), 0, lane);
        else norm_put<DT, W>(a, y[0], in, base, k, m);
    }
    if (MODE == kNormStore && a.amax != nullptr) norm_amax<DT>(a, m);
}

// Many rows.  They come by bulk copies into a ring of shared memory, so that
// memory stays busy while rows are summed and written: a step is one row, 16 elements
// per thread in pieces of W (WIDE: rows longer than 512 threads' are).  Rows that begin between 16-byte boundaries are copied with
// the bytes around them (a 16-byte piece that holds one of the row's bytes is the
// allocation's) and read an element at a time.
template <int DT, int W, bool WIDE, int MODE, bool RES>
__global__ void __launch_bounds__(WIDE ? 1024 : 512, RES || WIDE ? 1 : 2) k_norm_ring(const NormArgs a, int stages, int stage_bytes)
{
    constexpr int E = 16, VPT = E / W, kMostStages = 8, ES = In<DT>::BYTES, kTensors = RES ? 2 : 1;
    extern __shared__ __align__(128) uint8_t dsm[];
    __shared__ float part[2][32];
    __shared__ __align__(8) uint64_t full[kMostStages];
    const int lane = threadIdx.x & 31, K = (int)a.K, tensor_bytes = stage_bytes / kTensors;
    const int T = blockDim.x, t = threadIdx.x;
    const int steps = (int)a.M > (int)blockIdx.x ? ((int)a.M - (int)blockIdx.x - 1) / (int)gridDim.x + 1 : 0;
    auto skew = [&](int64_t row) { return W > 1 ? 0 : (int)((row * K * ES) & 15); };
    int64_t next = blockIdx.x;   // the row whose copies are issued next (thread 0's)
    auto issue = [&](int s) {
        const int off = skew(next);
        const uint32_t bytes = (uint32_t)(off + K * ES + 15) & ~15u;
        uint8_t *const st = dsm + s * stage_bytes;
        mbar_arrive_expect_tx(&full[s], bytes * kTensors);
        bulk_load(st, static_cast<const char *>(a.x) + next * K * ES - off, bytes, &full[s]);
        if constexpr (RES) bulk_load(st + tensor_bytes, static_cast<const char *>(a.residual) + next * K * ES - off, bytes, &full[s]);
        next += gridDim.x;
    };
    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; s++) mbar_init(&full[s], 1);
        fence_mbar_init();
    }
    for (int i = threadIdx.x; i < 64; i += blockDim.x) part[i >> 5][i & 31] = 0.0f;   // the CTA may have fewer warps, one even
    __syncthreads();
    griddep_wait();   // nothing was read or written so far
    if (threadIdx.x == 0)
        for (int i = 0; i < steps && i < stages; i++) issue(i);
    float w[VPT][W];
    if constexpr (MODE != kNormFactor) {
#pragma unroll
        for (int i = 0; i < VPT; i++) {
#pragma unroll
            for (int j = 0; j < W; j++) w[i][j] = 0.0f;
            if ((t + i * T) * W < K) load_weights<W>(w[i], a.weight, a.wf32, (t + i * T) * W);
        }
    }
    uint32_t m = 0;   // largest |y| of this thread
    int s = 0;
    uint32_t parity = 0;
    int64_t row = blockIdx.x;
    for (int n = 0; n < steps; n++, row += gridDim.x) {
        const uint8_t *const st = dsm + s * stage_bytes + skew(row);
        const bool ok = !a.give_up && mbar_wait_bounded(&full[s], parity);
        Piece<DT, W> h[VPT];
#pragma unroll
        for (int i = 0; i < VPT; i++) {
            const int k = (t + i * T) * W;
            h[i].zero();
            if (k < K) {
                h[i].shared(st, k);
                if constexpr (RES) {
                    Piece<DT, W> res;
                    res.shared(st + tensor_bytes, k);
                    h[i].add(res);
                }
            }
        }
        const float sum = warp_sum(squares<DT, W, VPT>(h));
        if (lane == 0) part[n & 1][t >> 5] = sum;
        if (__syncthreads_or(!ok)) {   // a wait ran out: the copies in flight land before shared memory goes away
            if (t == 0) {
                for (int j = n; j < steps && j < n + stages; j++) (void)mbar_wait_bounded(&full[j % stages], (uint32_t)((j / stages) & 1));
                if (a.status != nullptr) atomicOr(a.status, kStTimeout);
            }
            break;
        }
        if (t == 0 && n + stages < steps) {   // every thread has the stage in its registers
            fence_proxy_async();
            issue(s);
        }
        float f = part[n & 1][lane & (WIDE ? 31 : 15)];
#pragma unroll
        for (int o = WIDE ? 16 : 8; o > 0; o >>= 1) f += __shfl_xor_sync(0xFFFFFFFFu, f, o);
        f = row_factor(f, a.inv, a.eps);
        if (t == 0) a.rstd[row] = f;
        const int64_t base = row * K;
        if constexpr (RES) {
#pragma unroll
            for (int i = 0; i < VPT; i++)
                if ((t + i * T) * W < K) h[i].store(a.h, base + (t + i * T) * W);
        }
        if constexpr (MODE == kNormCast) {
            float y[VPT][W];
#pragma unroll
            for (int i = 0; i < VPT; i++) {
                norm_y<DT, W>(y[i], h[i], f, w[i]);
            }
            norm_cast<W, VPT>(a, y, a.q_row + base, a.s_row + row * (K / 128), t * W, T * W, lane);
        } else if constexpr (MODE == kNormStore) {
#pragma unroll
            for (int i = 0; i < VPT; i++) {
                const int k = (t + i * T) * W;
                float y[W];
                norm_y<DT, W>(y, h[i], f, w[i]);
                norm_put<DT, W>(a, y, k < K, base, k, m);
            }
        }
        if (++s == stages) {
            s = 0;
            parity ^= 1;
        }
    }
    if (MODE == kNormStore && a.amax != nullptr) norm_amax<DT>(a, m);
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------

// Threads of a row whose threads take E elements each.
int row_threads(int64_t K, int E) { return (int)((K + 32 * E - 1) / (32 * E)) * 32; }

template <int DT, int W, int VPT, int MODE> cudaError_t norm_rows(NormArgs a, cudaStream_t st)
{
    a.row_threads = W == 1 && VPT == 8 ? 2 * row_threads(a.K, 16) : VPT * W == 32 ? 1024 : row_threads(a.K, VPT * W);
    a.cta_rows = a.row_threads < 256 ? 256 / a.row_threads : 1;
    a.per_warps = 65536u / (a.row_threads / 32) + 1;
    const int threads = a.cta_rows * a.row_threads;
    const int64_t grid = (a.M + a.cta_rows - 1) / a.cta_rows;
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    return launch_k(true, a.residual != nullptr ? k_norm_rows<DT, W, VPT, MODE, true> : k_norm_rows<DT, W, VPT, MODE, false>,
                    dim3((unsigned)grid), dim3(threads), 0, st, a);
}

template <int DT, int W, bool WIDE, int MODE, bool RES>
cudaError_t norm_ring_t(const NormArgs &a, int threads, int per_sm, int stages, int stage_bytes, cudaStream_t st)
{
    const cudaError_t e = engine_smem_ready<k_norm_ring<DT, W, WIDE, MODE, RES>>(kRingBytes, true);
    if (e != cudaSuccess) return e;
    const int64_t most = (int64_t)per_sm * sm_count();
    return launch_k(true, k_norm_ring<DT, W, WIDE, MODE, RES>, dim3((unsigned)(a.M < most ? a.M : most)), dim3(threads),
                    (size_t)stages * stage_bytes, st, a, stages, stage_bytes);
}

// Whether the ring's kernel takes the call, and its launch: rows of 257 to 16384
// elements that begin anywhere, or BF16 ones of 2048 on, where there are enough of them to keep every CTA's ring busy
// (8192 x 4096 BF16 without a residual 20.6 us, one row a CTA 26.5; 16384 x 7168 cast with
// one 122 and 151; 8192 x 5001 FP32 57 and 127; but 8192 x 4096 FP32 with a residual
// 85.0 and 78.6, 8192 x 512 BF16 5.9 and 3.4, 2048 x 4096 cast 12.5 and 11.1; and the other way by
// little, 8192 x 4096 BF16 stored with a residual 42.9 and 41.6, 16384 x 7168 142.5 and 148.6).
template <int DT, int W, int MODE, bool RES> bool norm_ring(const NormArgs &a, cudaStream_t st, cudaError_t &e)
{
    constexpr int ES = In<DT>::BYTES;
    if (a.K <= 256 || a.K > 16384 || (W > 1 && a.K < 2048)) return false;
    const bool wide = a.K > 8192;
    const int threads = row_threads(a.K, 16);
    const int stage_bytes = (RES ? 2 : 1) * (int)((a.K * ES + 15) / 16 * 16 + (a.K * ES % 16 != 0 ? 16 : 0));
    const int fit = kRingBytes / (2 * stage_bytes);
    // With a residual fewer rows at a time are better: 16384 x 7168 stored 142 us at two stages, 159 to 164 at three
    // and more; 8192 x 4096 cast 38.3 at 512 threads an SM, 40.3 at 1024, without a residual 28 and 25.
    int per_sm = (wide || !RES ? 1024 : 512) / threads;
    per_sm = per_sm > 8 ? 8 : per_sm;
    per_sm = per_sm > fit ? fit : per_sm;
    if (per_sm == 0 || a.M < (int64_t)(W > 1 ? 8 : 2) * per_sm * sm_count()) return false;
    const int room = kRingBytes / per_sm / stage_bytes, most = RES && MODE == kNormStore ? 2 : 8, stages = room > most ? most : room;
    e = wide ? norm_ring_t<DT, W, true, MODE, RES>(a, threads, per_sm, stages, stage_bytes, st)
             : norm_ring_t<DT, W, false, MODE, RES>(a, threads, per_sm, stages, stage_bytes, st);
    return true;
}

template <int DT, int W, int MODE> cudaError_t norm_w(const NormArgs &a, cudaStream_t st)
{
    if constexpr (DT == BF16 || W == 1) {
        cudaError_t e;
        if (a.residual != nullptr ? norm_ring<DT, W, MODE, true>(a, st, e) : norm_ring<DT, W, MODE, false>(a, st, e)) return e;
    }
    // Elements of a thread.  Rows that the ring may take are laid out as there, so that the order of a row's sum, and with it
    // every bit of the result, is the same in a call of few rows and in one of many.
    constexpr int E = W == 1 ? 4 : 8;
    if (a.K <= 32 * E) return norm_rows<DT, W, E / W, MODE>(a, st);
    if constexpr (W == 1)
        if (a.K <= 8192) return norm_rows<DT, 1, 8, MODE>(a, st);
    if (a.K <= 16384) return norm_rows<DT, W, 16 / W, MODE>(a, st);
    if constexpr (W > 1)
        if (a.K <= 32768) return norm_rows<DT, W, 32 / W, MODE>(a, st);
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

}  // namespace qk
