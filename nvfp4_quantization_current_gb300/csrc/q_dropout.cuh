// Dropout from a counter: which elements a call keeps follows from the seed
// and an element's index alone, so neither the forward pass nor the backward
// pass stores a mask.
//
// Element i takes 16 bits of Philox4x32-10 block offset + i / 8 (counter
// (g lo, g hi, 2, 0): stream 2, beside the two streams of the stochastic
// rounding): draw i % 8 = half (i % 2) of output word (i % 8) / 2, low half
// first.  It is kept iff its draw is not below the threshold T = 65536 p
// rounded to an integer, so exactly T of the 65536 draws drop an element, and
// a kept one is multiplied by c = 65536 / (65536 - T), which keeps the mean.
#pragma once

#include "q_common.cuh"

namespace qk {

constexpr uint32_t kDropStream = 2u;

struct DropArgs {
    PhiloxKeys keys;
    uint64_t offset;
    uint32_t threshold;   // T << 16
    float c;
    bool all;             // T = 65536: nothing is kept
};
inline DropArgs drop_args(uint64_t seed, uint64_t offset, uint32_t T, float c)
{
    return {philox_keys(seed), offset, T << 16, c, T == 65536u};
}

// The eight 16-bit draws of elements 8 b .. 8 b + 7, two per word.
QD uint4 drop_draws(uint64_t b, const DropArgs &d) { return sr_bits_rk<kDropStream>(d.offset + b, d.keys); }

// Whether element j of the eight is kept (not for d.all): its draw in the upper
// half of a word against T in the same place; what is below does not matter.
QD bool drop_keep(const uint4 &draws, int j, uint32_t threshold)
{
    const uint32_t w = word(draws, j >> 1);
    return ((j & 1) ? w : (w << 16)) >= threshold;
}

}  // namespace qk
