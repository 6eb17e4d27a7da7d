// Shared by the fp32 kernels over a paged cache: asynchronous copies of key and value tiles.
#pragma once

#include "paged.cuh"

namespace hlta {
namespace paged {
namespace f32 {

// 16 or 4 bytes global -> shared, or zeros when !in
__device__ __forceinline__ void copy16(float *dst, const float *src, bool in)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy4(float *dst, const float *src, bool in)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src), "r"(in ? 4 : 0) : "memory");
}

// Positions [p0, p0 + N) of key head h into K and (unless null) V, rows of `st` floats; positions
// outside u and channels from d to dp (d rounded up to four) as zeros. A warp per row, four channels a
// lane.
template <int N, int THREADS>
__device__ __forceinline__ void copy_tile(const PagedKV &c, int b, int h, int p0, const Span &u, float *K, float *V, int st, int dp)
{
    const int psz = 1 << c.page_log2, warp = threadIdx.x >> 5, x = 4 * (threadIdx.x & 31);
    if (x >= dp) return;
    const bool words = (c.d & 3) == 0;
#pragma unroll 4
    for (int r = warp; r < N; r += THREADS / 32) {
        const int p = p0 + r;
        const bool in = p >= u.lo && p < u.hi;
        const long at = in ? (((long)page_of(c, b, p) * c.H + h) * psz + (p & (psz - 1))) * c.d + x : 0;
        const float *k = (const float *)c.k + at, *v = (const float *)c.v + at;
        float *kd = K + r * st + x, *vd = V + r * st + x;
        if (words) {
            copy16(kd, k, in);
            if (V) copy16(vd, v, in);
        } else {
            for (int y = 0; y < 4; ++y) {
                const bool ch = in && x + y < c.d;
                copy4(kd + y, ch ? k + y : (const float *)c.k, ch);
                if (V) copy4(vd + y, ch ? v + y : (const float *)c.v, ch);
            }
        }
    }
}

}  // namespace f32
}  // namespace paged
}  // namespace hlta
