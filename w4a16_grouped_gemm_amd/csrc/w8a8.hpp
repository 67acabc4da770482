// w8a8.hpp -- internal interface of the W8A8 kernels (int8 rows with one scale
// each), the RMS norm that produces such rows, and the scored router.
#pragma once

#include "common.hpp"

namespace moe {

constexpr int kMaxNormDim = 65536;       // row length of the norm and the int8 quantizer
constexpr int kMaxRouteGroups = 64;      // one lane of a wave per group

// fp32 pair -> bf16 pair, round to nearest even
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi)
{
    typedef float f2 __attribute__((ext_vector_type(2)));
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2{lo, hi}), b2));
}

// The bits of v from the lane that a DPP control names, 0 where the row mask excludes the lane.
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ uint32_t dpp(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
}

// A wave's reduction: within quads, half rows and rows, then from row to row, whose last lane has it all. op(x, 0) is x.
template <class Op>
__device__ __forceinline__ uint32_t wave_reduce(uint32_t v, Op op)
{
    v = op(v, dpp<0xB1>(v));                           // quad_perm [1,0,3,2]
    v = op(v, dpp<0x4E>(v));                           // quad_perm [2,3,0,1]
    v = op(v, dpp<0x141>(v));                          // row_half_mirror
    v = op(v, dpp<0x140>(v));                          // row_mirror
    v = op(v, dpp<0x142, 0xA>(v));                     // row_bcast:15 to rows 1 and 3
    v = op(v, dpp<0x143, 0xC>(v));                     // row_bcast:31 to rows 2 and 3
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// A row whose largest magnitude is below 2^-100 counts as zero, so that neither
// 1 / max overflows nor max / 127 meets a subnormal.
constexpr float kZeroRow = 0x1p-100f;

// Codes of a row y with the largest magnitude amax: rint(127 y / amax), and the scale amax / 127.
// The quotient 127 y / max|y| is rounded correctly near every tie: with r the
// reciprocal of the maximum, t = 127 y r and one residual step
// t + fma(-t, max, 127 y) r, so that the many bf16 rows whose values lie
// exactly between two codes go to the even code, as the definition says.
struct RowCodes {
    float factor, top, inv, scale;                     // factor 127 times a power of two that keeps 127 y finite
    bool none;                                         // all codes 0: a row of zeros, or with a NaN or an infinity

    __device__ __forceinline__ explicit RowCodes(float amax)
    {
        const bool finite = __builtin_isfinite(amax);
        const float f = amax > 0x1p64f ? 0x1p-64f : 1.0f;
        none = !(amax >= kZeroRow) || !finite;
        factor = 127.0f * f;
        top = amax * f;
        inv = none ? 0.0f : 1.0f / top;
        scale = finite ? (none ? 0.0f : amax / 127.0f) : __builtin_nanf("");
    }

    __device__ __forceinline__ uint32_t code(float v) const
    {
        const float y = none ? 0.0f : v * factor;
        const float t = y * inv;
        return (uint32_t)(int)__builtin_rintf(__builtin_fmaf(__builtin_fmaf(-t, top, y), inv, t)) & 0xFFu;
    }
};

hipError_t launch_route_scored(const moe_shape &sh, const moe_router &r, const float *logits, const float *bias,
                               int32_t *ids, float *w, hipStream_t st);

struct NormLaunch {
    long long rows;
    int K;
    const uint16_t *x;        // [rows][K]
    const uint16_t *residual; // NULL, or [rows][K] added to x
    const uint16_t *weight;   // NULL: no norm (q quantizes the rows as they are)
    float eps;
    uint16_t *sum;            // x + residual as bf16 (with residual)
    uint16_t *y;              // NULL, or the bf16 rows
    int8_t *q;                // NULL, or the int8 rows
    float *q_scale;           // [rows] (with q)
    const int32_t *rows_dev;  // NULL, or the row count on the device (at most rows)
};
hipError_t launch_norm(const NormLaunch &n, hipStream_t st);

struct W8GemmLaunch {
    moe_gemm_kind kind;
    const int8_t *a;             // [a_rows][K]
    const float *as;             // [a_rows]
    const uint16_t *a_bf16;      // instead of a and as, where quantizes_rows: bf16 rows, quantized by the product
    const int32_t *a_row_index;  // NULL, or row r reads activation row a_row_index[r] / top_k
    int top_k;
    const int32_t *offsets;      // [E+1] on the device; NULL: one dense expert with max_rows rows
    int num_experts;
    const int8_t *wq;            // [E][N][K]
    const float *ws;             // [E][N]
    void *c;
    bool c_f32;
    int K, N;                    // reduction length; weight rows per expert
    int max_rows, expected_rows;
};
hipError_t launch_w8_gemm(const W8GemmLaunch &g, hipStream_t st);
// Whether the product g (bf16 results, no row index) takes bf16 rows as well.
bool quantizes_rows(const W8GemmLaunch &g);

}  // namespace moe
