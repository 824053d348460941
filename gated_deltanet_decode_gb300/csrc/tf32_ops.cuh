// fp32 products on the tensor cores in tf32 (sm_103a): operands split in a head
// and a tail, x = hi + lo, and three products hi hi + hi lo + lo hi, which leaves
// out about 2^-22 of a term.  The tensor cores cut their sums short instead of
// rounding them, so long sums are made of short ones, added in fp32.
// Included by one translation unit a kernel.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "gdn_ptx.cuh"

namespace gdn {
namespace {

// The head is x rounded to the 11 bits that a product reads (by an addition to
// its bits: the conversion instruction costs as much as a product); the tail,
// exact, has 12, of which it reads 11.  A head cut short instead leaves tails
// twice as large, and the tails' product, left out, showed (5.6e-6 of a
// result's norm, against 8e-7 for plain fp32).
__device__ __forceinline__ void split(float x, uint32_t &hi, uint32_t &lo)
{
    hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
    lo = __float_as_uint(x - __uint_as_float(hi));
}
// Two at a time: the tails by one instruction.
__device__ __forceinline__ void split2(float x, float y, uint32_t &xh, uint32_t &xl, uint32_t &yh, uint32_t &yl)
{
    xh = (__float_as_uint(x) + 0x1000u) & 0xffffe000u, yh = (__float_as_uint(y) + 0x1000u) & 0xffffe000u;
    const float2 t = fma2(make_float2(__uint_as_float(xh), __uint_as_float(yh)), make_float2(-1.f, -1.f), make_float2(x, y));
    xl = __float_as_uint(t.x), yl = __float_as_uint(t.y);
}
__device__ __forceinline__ void mma8(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

} // namespace
} // namespace gdn
