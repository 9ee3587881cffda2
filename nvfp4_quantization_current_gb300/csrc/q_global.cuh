// Loads of what the kernel ahead in the stream may have written.  A kernel that is
// launched while that one ends reads it behind griddep_wait(), so these are plain
// loads, and volatile: a non-coherent load may be taken for one of data that no
// kernel in flight writes, and be moved ahead of the wait.
#pragma once

#include "q_common.cuh"

namespace qk {

QD uint4 load_16(const void *p)
{
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
QD uint2 load_8(const void *p)
{
    uint2 v;
    asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}
QD float load_float(const void *p)
{
    float v;
    asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p));
    return v;
}
QD float load_bf16(const void *p)
{
    uint16_t v;
    asm volatile("ld.global.u16 %0, [%1];" : "=h"(v) : "l"(p));
    return __uint_as_float((uint32_t)v << 16);
}

}  // namespace qk
