// The transposed blockwise copy of the norm's result: 128x1 blocks along M of
// y = (h s) w in FP32 (k_norm.cu), y itself never stored.
//
// On the tile engine with two CTAs of 256 threads per SM, tiles of 128 rows x 256
// bytes: while one waits at a barrier, the other works (its issue slots are 49 % in use
// at 16384 x 4096).  Both copies of 8192 x 4096 BF16 with a residual take 58.6 to 59.6
// us, 39.3 of them for the rows alone; walked from the first tile on, 62.1.  A thread (half
// a warp over a row's 16-byte chunks) holds 8 rows of a chunk of h and multiplies by
// the rows' factors and the columns' weights as it goes.  The half warps' column
// maxima meet in shared memory, and the codes are transposed in the consumed stage
// and written as full 128-byte rows.
#include "q_engine.cuh"
#include "q_global.cuh"
#include "q_internal.h"

namespace qk {

namespace {

// N weights from column k on; zeros where `in` is false.
template <int N> QD void col_weights(float (&w)[N], const void *weight, bool f32, int64_t k, bool in)
{
#pragma unroll
    for (int c = 0; c < N; c += 4) {
        float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (in && f32) {
            const uint4 v = load_16(static_cast<const float *>(weight) + k + c);
            f = make_float4(elem<F32>(v, 0), elem<F32>(v, 1), elem<F32>(v, 2), elem<F32>(v, 3));
        } else if (in) {
            const uint2 b = load_8(static_cast<const uint16_t *>(weight) + k + c);
            f = make_float4(__uint_as_float(b.x << 16), __uint_as_float(b.x & 0xFFFF0000u), __uint_as_float(b.y << 16),
                            __uint_as_float(b.y & 0xFFFF0000u));
        }
        w[c] = f.x, w[c + 1] = f.y, w[c + 2] = f.z, w[c + 3] = f.w;
    }
}

struct ColCfg {
    static constexpr int kRows = 128, kThreads = 256, kStages = 3, kRowBytes = 256;
    static constexpr int kTileBytes = kRows * kRowBytes, kSmem = kStages * kTileBytes;
};

template <int DT>
__global__ void __launch_bounds__(ColCfg::kThreads, 2)
k_norm_cols(const __grid_constant__ CUtensorMap tmap, int64_t M, int64_t K, const float *__restrict__ rstd,
            const void *__restrict__ weight, bool wf32, uint8_t *__restrict__ q_colT, float *__restrict__ s_colT, int32_t *status)
{
    constexpr int VEC = In<DT>::VEC, TC = 16 * VEC, CW = VEC / 4, TPC = ColCfg::kThreads / TC;   // TPC: threads per column
    constexpr int kRows = ColCfg::kRows, kRowBytes = ColCfg::kRowBytes;
    __shared__ __align__(16) float part[16][CW][16][4];   // half warps' column maxima, of four columns of each chunk in turn
    __shared__ __align__(16) float calpha[TC];
    const int t = threadIdx.x, warp = t >> 4, lane = t & 15;   // half warps, and chunks of a row
    const int64_t tiles_m = M / kRows, tiles_k = (K + TC - 1) / TC;

    griddep_wait();   // the rows' factors and sums are the kernel's ahead, which left the last of them in L2: the walk begins there
    float s_ahead[8], w_ahead[VEC];
    auto fetch = [&](int64_t tile) {
        if (tile < 0) return;
        const int64_t tm = tile / tiles_k, k = (tile - tm * tiles_k) * TC + lane * VEC;
#pragma unroll
        for (int j = 0; j < 8; j++) s_ahead[j] = load_float(rstd + tm * kRows + 8 * warp + j);
        col_weights<VEC>(w_ahead, weight, wf32, k, k < K);
    };
    fetch(tiles_m * tiles_k - 1 - blockIdx.x);
    run_tiles<ColCfg>(&tmap, tiles_m, tiles_k, TC, true, status, [&](uint8_t *st, int64_t tm, int64_t tk) {
        const int64_t mb = tm * kRows, kb = tk * TC;
        uint4 v[8];
#pragma unroll
        for (int j = 0; j < 8; j++) v[j] = lds16(st + (8 * warp + j) * kRowBytes + lane * 16);
        float s[8], w[VEC];
#pragma unroll
        for (int j = 0; j < 8; j++) s[j] = s_ahead[j];
#pragma unroll
        for (int c = 0; c < VEC; c++) w[c] = w_ahead[c];
        fetch(tm * tiles_k + tk - (int64_t)gridDim.x);   // the next tile's, on their way behind this one
        // y = (h s) w for a pair of a row's elements
        auto y2 = [&](int j, int c, float &y0, float &y1) {
            y0 = elem<DT>(v[j], c);
            y1 = elem<DT>(v[j], c + 1);
            mul2(y0, y1, s[j], s[j]);
            mul2(y0, y1, w[c], w[c + 1]);
        };
        float top[VEC];
#pragma unroll
        for (int c = 0; c < VEC; c++) top[c] = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; j++)
#pragma unroll
            for (int c = 0; c < VEC; c += 2) {
                float y0, y1;
                y2(j, c, y0, y1);
                top[c] = fmax_abs(top[c], y0);
                top[c + 1] = fmax_abs(top[c + 1], y1);
            }
#pragma unroll
        for (int c = 0; c < VEC; c += 4)   // four columns at a time, a quarter warp's 128 bytes: no two lanes on one bank
            *reinterpret_cast<float4 *>(&part[warp][c / 4][lane][0]) = make_float4(top[c], top[c + 1], top[c + 2], top[c + 3]);
        __syncthreads();
        {
            const int col = t / TPC, sub = t % TPC, l = col / VEC, q = col % VEC;   // lane l's column q
            float b = 0.0f;
#pragma unroll
            for (int i = sub; i < 16; i += TPC) b = fmax_abs(b, part[i][q / 4][l][q % 4]);
            const uint32_t bits = group_max<TPC>(__float_as_uint(b) & 0x7FFFFFFFu);
            if (sub == 0) {
                const float alpha = alpha_from_amax(448.0f, __uint_as_float(bits));
                calpha[col] = alpha;
                if (kb + col < K) {
                    s_colT[(kb + col) * (M / 128) + tm] = __fdiv_rn(1.0f, alpha);
                    flag_nonfinite(status, bits);
                }
            }
        }
        __syncthreads();
        float ca[VEC];
#pragma unroll
        for (int c = 0; c < VEC; c += 4) *reinterpret_cast<float4 *>(ca + c) = *reinterpret_cast<const float4 *>(&calpha[lane * VEC + c]);
        uint32_t code[8][CW];
#pragma unroll
        for (int j = 0; j < 8; j++) {
            float f[VEC];
#pragma unroll
            for (int c = 0; c < VEC; c += 2) {
                y2(j, c, f[c], f[c + 1]);
                mul2(f[c], f[c + 1], ca[c], ca[c + 1]);
            }
#pragma unroll
            for (int q = 0; q < CW; q++) code[j][q] = cvt_fp8x4<E4M3>(f[4 * q], f[4 * q + 1], f[4 * q + 2], f[4 * q + 3]);
        }
        park_fp8T<VEC>(st, code, warp, lane);
        __syncthreads();
        // the parked [TC][128] codes as rows of q_colT, 16 bytes of two neighbouring slots at a time (the order that
        // copy_out_fp8T undoes)
#pragma unroll
        for (int it = 0; it < TC * 8 / ColCfg::kThreads; it++) {
            const int idx = it * ColCfg::kThreads + t, col = idx >> 3, pr = idx & 7, sw = col / VEC;
            uint4 o = *reinterpret_cast<const uint4 *>(st + col * 128 + ((2 * pr) ^ (sw & ~1)) * 8);
            if (sw & 1) o = make_uint4(o.z, o.w, o.x, o.y);
            if (kb + col < K) stg16(q_colT + (kb + col) * M + mb + 16 * pr, o);
        }
    });
}

template <int DT>
cudaError_t cols_t(const void *h, int64_t M, int64_t K, const float *rstd, const void *weight, bool wf32, uint8_t *q_colT,
                   float *s_colT, int32_t *status, cudaStream_t st)
{
    constexpr int TC = 16 * In<DT>::VEC;
    alignas(64) CUtensorMap map;
    cudaError_t e = make_tile_map(&map, h, DT, M, K, ColCfg::kRows, ColCfg::kRowBytes);
    if (e == cudaSuccess) e = engine_smem_ready<k_norm_cols<DT>>(ColCfg::kSmem, true);
    if (e != cudaSuccess) return e;
    const int64_t tiles = (M / ColCfg::kRows) * ((K + TC - 1) / TC), most = 2 * sm_count();
    return launch_k(true, k_norm_cols<DT>, dim3((unsigned)(tiles < most ? tiles : most)), dim3(ColCfg::kThreads), ColCfg::kSmem, st,
                    map, M, K, rstd, weight, wf32, q_colT, s_colT, status);
}

}  // namespace

cudaError_t launch_norm_cast_cols(const void *h, int dt, int64_t M, int64_t K, const float *rstd, const void *weight, bool wf32,
                                  uint8_t *q_colT, float *s_colT, int32_t *status, cudaStream_t st)
{
    return dt == BF16 ? cols_t<BF16>(h, M, K, rstd, weight, wf32, q_colT, s_colT, status, st)
                      : cols_t<F32>(h, M, K, rstd, weight, wf32, q_colT, s_colT, status, st);
}

}  // namespace qk
