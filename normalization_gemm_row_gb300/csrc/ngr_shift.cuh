// ngr_shift.cuh -- 16-byte reads of rows that start at any element.
#pragma once

#include <cuda_runtime.h>
#include <cstdint>

namespace ngr {

// 8 elements from any 2-byte aligned address: the one or two aligned 16-byte
// words they lie in, shifted together; a word without any of the elements
// [first, last) (counted from p) is not read.  The distance from the boundary
// is the same for all threads of a row.
__device__ __forceinline__ uint4 load_shifted(const uint16_t *p, int first, int last)
{
    const int d = static_cast<int>((reinterpret_cast<uintptr_t>(p) >> 1) & 7u);
    const uint4 *q = reinterpret_cast<const uint4 *>(p - d);
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    const uint4 lo = first < 8 - d ? __ldg(q) : zero;
    if (d == 0) return lo;
    const uint4 hi = last > 8 - d ? __ldg(q + 1) : zero;
    uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    if (d & 4) {
#pragma unroll
        for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
    }
    if (d & 2) {
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
    }
    if (d & 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace ngr
