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

}  // namespace moe
