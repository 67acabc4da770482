// fp8.hpp -- internal interface of the FP8 kernels: e4m3 codes with a binary32
// scale for each 128 values of a row (activations) or 128 x 128 values (weights).
#pragma once

#include "w8a8.hpp"

namespace moe {

constexpr float kFp8Top = 448.0f;        // the largest e4m3 value

// Two binary32 values -> the low (HI: high) half word of two e4m3 codes, round to nearest even (values up to 464 in
// magnitude, which is what rounds to 448 or less).
template <bool HI>
__device__ __forceinline__ uint32_t fp8_pair(float a, float b, uint32_t old)
{
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(a, b, (int)old, HI);
}

// Codes of a block u * m (m a factor of the whole block, in [1, 2)) from the largest magnitude amax of u:
// e4m3(448 u / amax) and the scale m amax / 448, or with powers of two the least scale 2^n that is not less, and
// e4m3(u m / 2^n). The quotient needs no m; it is rounded correctly at every tie of values with few bits (bf16
// values, products of two of them): r the reciprocal, t = 448 u r and one residual step t + fma(-t, amax, 448 u) r.
// 448 = 7 * 2^6, so that 448 u is exact where u has 21 bits or fewer.
struct BlockCodes {
    float factor, top, inv, scale;
    bool none;                                         // all codes 0: a block of zeros, or with a NaN or an infinity

    __device__ __forceinline__ BlockCodes(float amax, float m, bool pow2)
    {
        const bool finite = __builtin_isfinite(amax * m);
        const float v = amax * m;
        none = !(v >= kZeroRow) || !finite;
        if (pow2) {
            // v = 2^x (1 + f), 448 = 2^8 1.75: the exponent is x - 8, one more where 1 + f is above 1.75
            const uint32_t b = __float_as_uint(v);
            const uint32_t s = (b & 0x7F800000u) - (8u << 23) + ((b & 0x007FFFFFu) > 0x00600000u ? 1u << 23 : 0u);
            scale = none ? 0.0f : __uint_as_float(s);
            top = 1.0f;                                // u m times the exact reciprocal: nothing left to correct
            inv = 1.0f;
            factor = none ? 0.0f : __uint_as_float((254u << 23) - s);
            mul = m;
        } else {
            const float f = amax > 0x1p64f ? 0x1p-64f : 1.0f;
            factor = kFp8Top * f;
            top = none ? 1.0f : amax * f;
            inv = none ? 0.0f : __builtin_amdgcn_rcpf(top);
            const float q = v * (1.0f / kFp8Top);      // v / 448, its rounding corrected
            scale = none ? 0.0f : __builtin_fmaf(__builtin_fmaf(-q, kFp8Top, v), 1.0f / kFp8Top, q);
            mul = 1.0f;
        }
        if (!finite)
            scale = __builtin_nanf("");
    }

    template <bool POW2>
    __device__ __forceinline__ float quotient(float u) const
    {
        if constexpr (POW2)
            return none ? 0.0f : u * mul * factor;
        const float y = none ? 0.0f : u * factor;
        const float t = y * inv;
        return __builtin_fmaf(__builtin_fmaf(-t, top, y), inv, t);
    }

    template <bool POW2>
    __device__ __forceinline__ u32x2 codes(const float (&u)[8]) const
    {
        u32x2 o = {0, 0};
#pragma unroll
        for (int d = 0; d < 2; ++d) {
            o[d] = fp8_pair<false>(quotient<POW2>(u[4 * d]), quotient<POW2>(u[4 * d + 1]), 0);
            o[d] = fp8_pair<true>(quotient<POW2>(u[4 * d + 2]), quotient<POW2>(u[4 * d + 3]), o[d]);
        }
        return o;
    }

    float mul;
};

// The largest of 16 neighbouring lanes (a DPP row), in each of them.
__device__ __forceinline__ uint32_t row16_max(uint32_t v)
{
    auto op = [](uint32_t a, uint32_t b) { return b > a ? b : a; };
    v = op(v, dpp<0xB1>(v));                           // quad_perm [1,0,3,2]
    v = op(v, dpp<0x4E>(v));                           // quad_perm [2,3,0,1]
    v = op(v, dpp<0x141>(v));                          // row_half_mirror
    return op(v, dpp<0x140>(v));                       // row_mirror
}

struct Fp8NormLaunch {
    long long rows;
    int K;
    const uint16_t *x;        // [rows][K]
    const uint16_t *residual; // NULL, or [rows][K] added to x
    const uint16_t *weight;   // NULL: no norm (the rows as they are)
    float eps;
    bool pow2;
    uint16_t *sum;            // x + residual as bf16 (with residual)
    uint16_t *y;              // NULL, or the bf16 rows
    uint8_t *q;               // codes
    float *q_scale;           // [rows][K / 128]
    const int32_t *rows_dev;  // NULL, or the row count on the device (at most rows)
};
hipError_t launch_norm_fp8(const Fp8NormLaunch &n, hipStream_t st);
hipError_t launch_fp8_weights(int E, int N, int K, const uint16_t *w, bool pow2, uint8_t *q, float *scale,
                              hipStream_t st);

struct Fp8GemmLaunch {
    moe_gemm_kind kind;
    const uint8_t *a;            // [a_rows][K]
    const float *as;             // [a_rows][K / 128]
    const int32_t *a_row_index;  // NULL, or row r reads activation row a_row_index[r] / top_k
    int top_k;
    const int32_t *offsets;      // [E+1] on the device; NULL: one dense expert with max_rows rows
    int num_experts;
    const uint8_t *wq;           // [E][N][K]
    const float *ws;             // [E][ceil(N / 128)][K / 128]
    void *c;
    bool c_f32;
    int K, N;                    // reduction length; weight rows per expert
    int max_rows, expected_rows;
};
hipError_t launch_fp8_gemm(const Fp8GemmLaunch &g, hipStream_t st);

}  // namespace moe
