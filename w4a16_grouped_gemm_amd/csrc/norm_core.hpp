// norm_core.hpp -- what the RMS norms share: a row's sum over the threads that
// hold it, and the range of its mean of squares.
#pragma once

#include "w8a8.hpp"

namespace moe {

namespace {

template <int TPR>
__device__ __forceinline__ float row_sum(float x, float *s_red)
{
    float v = __uint_as_float(wave_reduce(__float_as_uint(x), [](uint32_t a, uint32_t b) {
        return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
    }));
    if constexpr (TPR > 64) {
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0)
            s_red[wave] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int w = 0; w < TPR / 64; ++w)
            v += s_red[w];
        __syncthreads();
    }
    return v;
}

// A mean of squares plus eps from which the norm is not taken: past binary32's range (or NaN), or so small that
// squares lost bits, or all of them.
__device__ __forceinline__ bool out_of_range(float ms) { return !(ms >= 0x1p-100f && ms < __builtin_inff()); }

}  // namespace

}  // namespace moe
