// What the kernels of the NVFP4 product share: arguments, and the way of the
// block scales from memory to where the tensor core copies them from.
#pragma once

#include "q_mm.cuh"

namespace qk {

constexpr int kMm4Block = 256;      // elements of K per stage: 128 bytes of each operand row, 16 of its scales
constexpr int kScaleAtom = 2048;    // bytes of 128 rows' scales of a stage

// One operand's scales: [rows >> shift, pitch] bytes, `vec` of them (16, 4 or 1)
// at a time, as the pitch and the address allow.
struct Mm4Scales {
    const uint8_t *at;
    int64_t pitch;
    int rows, shift, vec;
};

// C = P Q^T: P's rows lie on tensor memory lanes, Q's rows on its columns.
// (store.status, store.c and so on are those of the epilogue that the products share.)
struct Mm4Args {
    MmArgs store;
    Mm4Scales p, q;
    const float *s_p, *s_q;   // the tensors' scales
};

// The 16 scales of a row's block kb; zero where there is no such row, or past the end of K.
QD uint4 load_scales16(const Mm4Scales &g, int64_t row, int kb)
{
    if (row >= g.rows) return make_uint4(0u, 0u, 0u, 0u);
    const int64_t first = (int64_t)kb * 16;
    const uint8_t *const src = g.at + (row >> g.shift) * g.pitch + first;
    if (g.vec == 16) return __ldg(reinterpret_cast<const uint4 *>(src));   // a pitch of 16 n: the block is whole
    uint32_t w[4] = {};
    const int n = g.pitch - first < 16 ? (int)(g.pitch - first) : 16;
    if (g.vec == 4) {
#pragma unroll
        for (int i = 0; i < 4; i++)
            if (4 * i < n) w[i] = __ldg(reinterpret_cast<const uint32_t *>(src) + i);
    } else {
#pragma unroll
        for (int i = 0; i < 16; i++)
            if (i < n) w[i / 4] |= (uint32_t)__ldg(src + i) << (8 * (i & 3));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// 128 rows' scales of a block, rows row0 + lane + 32 j in lane `lane`: a thread
// holds what becomes 16 bytes of four source lines, one for each 64 elements.
struct ScaleAtom {
    uint4 r[4];
    QD void load(const Mm4Scales &g, int64_t row0, int kb, int lane)
    {
#pragma unroll
        for (int j = 0; j < 4; j++) r[j] = load_scales16(g, row0 + lane + 32 * j, kb);
    }
    QD void put(uint8_t *atom, int lane) const
    {
        uint4 *const to = reinterpret_cast<uint4 *>(atom) + lane;
        to[0] = make_uint4(r[0].x, r[1].x, r[2].x, r[3].x);
        to[32] = make_uint4(r[0].y, r[1].y, r[2].y, r[3].y);
        to[64] = make_uint4(r[0].z, r[1].z, r[2].z, r[3].z);
        to[96] = make_uint4(r[0].w, r[1].w, r[2].w, r[3].w);
    }
};

}  // namespace qk
