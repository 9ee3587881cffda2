// What the kernels of the NVFP4 product share: arguments, and the way of the
// block scales from memory to where the tensor core copies them from.
#pragma once

#include "q_global.cuh"
#include "q_mm.cuh"

namespace qk {

constexpr int kMm4Block = 256;      // elements of K per stage: 128 bytes of each operand row, 16 of its scales
constexpr int kScaleAtom = 2048;    // bytes of 128 rows' scales of a stage

// One operand's scales: [rows >> shift, pitch] bytes.
struct Mm4Scales {
    const uint8_t *at;
    int64_t pitch;
    int rows, shift;
};

// C = P Q^T: P's rows lie on tensor memory lanes, Q's rows on its columns.
// (store.status, store.c and so on are those of the epilogue that the products share.)
struct Mm4Args {
    MmArgs store;
    Mm4Scales p, q;
    const float *s_p, *s_q;   // the tensors' scales
    int group;                // of the pair kernel's tile order
};

// The scales of up to 64 rows and four blocks on their way through a warp's registers: lane l has block l / 8 of the
// rows l % 8 + 8 i + 32 j (j < N).  Four lanes take 64 bytes of a scale row, so that a
// load touches 8 lines, and a lane's four rows of one i share a source line of the
// copies to tensor memory: 16 bytes of four lines, one for each 64 elements.
// WHOLE: every row begins on a 16-byte boundary.  Rows that begin anywhere are held as the five aligned vectors that their bytes lie
// in (a vector that holds one of the row's bytes is the allocation's), the fifths of
// a step's 32 rows one per lane, and shifted on their way out.
template <bool WHOLE> struct ScaleUnit {
    uint4 v[2][4], fifth[WHOLE ? 1 : 2];

    // Vector n of a row's unit; zeros where there is no such row, or past its end.
    static QD uint4 vector(const Mm4Scales &g, int64_t row, int kb, int n)
    {
        const uint8_t *const begin = g.at + (row >> g.shift) * g.pitch;
        const uintptr_t p = (reinterpret_cast<uintptr_t>(begin + (int64_t)kb * 16) & ~(uintptr_t)15) + 16 * n;
        if (row >= g.rows || p >= reinterpret_cast<uintptr_t>(begin + g.pitch)) return make_uint4(0u, 0u, 0u, 0u);
        return load_16(reinterpret_cast<const void *>(p));
    }
    template <int N> QD void load(const Mm4Scales &g, int64_t row0, int kb, int lane)
    {
#pragma unroll
        for (int i = 0; i < 2; i++)
#pragma unroll
            for (int j = 0; j < N; j++) v[i][j] = vector(g, row0 + (lane & 7) + 8 * i + 32 * j, kb, lane >> 3);
        if constexpr (!WHOLE) {
#pragma unroll
            for (int i = 0; i < 2; i++)
                fifth[i] = lane >> 3 < N ? vector(g, row0 + (lane & 7) + 8 * i + 32 * (lane >> 3), kb, 4) : make_uint4(0u, 0u, 0u, 0u);
        }
    }
    // To the atom at `to` (of the block of this lane), lines `line` + 8 i on.
    template <int N> QD void put(const Mm4Scales &g, int64_t row0, int kb, uint8_t *to, int line, int lane)
    {
#pragma unroll
        for (int i = 0; i < 2; i++) {
            uint4 r[4];
#pragma unroll
            for (int j = 0; j < 4; j++) {
                r[j] = j < N ? v[i][j] : make_uint4(0u, 0u, 0u, 0u);
                if constexpr (!WHOLE)
                    if (j < N) r[j] = shifted(g, row0 + (lane & 7) + 8 * i + 32 * j, kb, v[i][j], fifth[i], j, lane);
            }
            uint4 *const at = reinterpret_cast<uint4 *>(to) + line + 8 * i;
            at[0] = make_uint4(r[0].x, r[1].x, r[2].x, r[3].x);
            at[32] = make_uint4(r[0].y, r[1].y, r[2].y, r[3].y);
            at[64] = make_uint4(r[0].z, r[1].z, r[2].z, r[3].z);
            at[96] = make_uint4(r[0].w, r[1].w, r[2].w, r[3].w);
        }
    }
    // This lane's 16 scales from its vector and the next, which the lane of the next block has, or for the last block the
    // lane with the row's fifth.  What follows the row's end is cut off: a NaN there would not vanish against the zero codes.
    static QD uint4 shifted(const Mm4Scales &g, int64_t row, int kb, const uint4 &a, const uint4 &fifth, int j, int lane)
    {
        const int64_t first = (int64_t)(kb + (lane >> 3)) * 16;
        const int s = (int)(reinterpret_cast<uintptr_t>(g.at + (row >> g.shift) * g.pitch) & 15);
        auto next = [&](uint32_t mine, uint32_t last) {
            const uint32_t n = __shfl_down_sync(0xFFFFFFFFu, mine, 8), l = __shfl_sync(0xFFFFFFFFu, last, 8 * j + (lane & 7));
            return lane < 24 ? n : l;
        };
        const uint4 b = make_uint4(next(a.x, fifth.x), next(a.y, fifth.y), next(a.z, fifth.z), next(a.w, fifth.w));
        const bool two = s & 8, one = s & 4;
        const uint32_t w0 = two ? a.z : a.x, w1 = two ? a.w : a.y, w2 = two ? b.x : a.z, w3 = two ? b.y : a.w, w4 = two ? b.z : b.x,
                       w5 = two ? b.w : b.y;
        const uint32_t u0 = one ? w1 : w0, u1 = one ? w2 : w1, u2 = one ? w3 : w2, u3 = one ? w4 : w3, u4 = one ? w5 : w4;
        const int bits = 8 * (s & 3), n = g.pitch - first < 16 ? (int)(g.pitch - first) : 16;
        auto cut = [&](uint32_t lo, uint32_t hi, int i) {
            const uint32_t w = __funnelshift_r(lo, hi, bits);
            return 4 * i + 4 <= n ? w : 4 * i >= n ? 0u : w & ((1u << (8 * (n - 4 * i))) - 1u);
        };
        return make_uint4(cut(u0, u1, 0), cut(u1, u2, 1), cut(u2, u3, 2), cut(u3, u4, 3));
    }
};

}  // namespace qk
