// norm_int8.hip -- RMS norm with the residual's addition and an int8 output, and
// the int8 row quantizer by itself (the same kernel without the norm).
//
//   h = bf16(x + residual)            (x itself without a residual)
//   y = (h * rstd) * weight           rstd = 1 / sqrt(mean h^2 + eps)
//   q = rint(127 y / max|y|), scale = max|y| / 127
// All in binary32; y is rounded to bf16 only where it is stored as bf16, so q is
// quantized from the unrounded rows. h is rounded because it is the residual
// stream that the caller keeps: the norm sees what the next layer will add to.
//
// The quotient 127 y / max|y| is rounded correctly near every tie: with r the
// reciprocal of the maximum, t = 127 y r and one residual step
// t + fma(-t, max, 127 y) r, so that the many bf16 rows whose values lie
// exactly between two codes go to the even code, as the definition says.
//
// Bound by memory: a row is read once and held in registers between the two
// reductions (sum of squares, maximum).
#include "w8a8.hpp"

namespace moe {

namespace {

// A row whose largest magnitude is below 2^-100 counts as zero, so that neither
// 1 / max overflows nor max / 127 meets a subnormal.
constexpr float kZeroRow = 0x1p-100f;
constexpr long long kFewRows = 1024;

template <int TPR>
__device__ __forceinline__ float row_sum(float v, float *s_red)
{
#pragma unroll
    for (int d = 1; d < 64; d *= 2)
        v += __shfl_xor(v, d);
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

template <int TPR>
__device__ __forceinline__ uint32_t row_max(uint32_t v, float *s_red)
{
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const uint32_t o = __shfl_xor(v, d);
        v = o > v ? o : v;
    }
    if constexpr (TPR > 64) {
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0)
            s_red[wave] = __uint_as_float(v);
        __syncthreads();
        v = 0;
#pragma unroll
        for (int w = 0; w < TPR / 64; ++w) {
            const uint32_t o = __float_as_uint(s_red[w]);
            v = o > v ? o : v;
        }
        __syncthreads();
    }
    return v;
}

// TPR threads per row (64: one wave, four rows to a workgroup; else the whole
// workgroup), each with VPT vectors of 8 values at stride TPR.
template <int TPR, int VPT, bool RES, bool NORM, bool Y, bool Q>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void norm_kernel(NormLaunch n)
{
    __shared__ float s_red[TPR / 64];
    constexpr int RPB = TPR < 256 ? 256 / TPR : 1;
    const int lane = threadIdx.x % TPR;
    const long long row = (long long)blockIdx.x * RPB + threadIdx.x / TPR;
    if (row >= n.rows)
        return;                                        // whole workgroups where they meet at barriers
    // Rows past the device's count: of few rows, read all the same (they are there) and left then, one round trip
    // instead of two; of many, left at once.
    if (n.rows_dev && n.rows >= kFewRows && row >= n.rows_dev[0])
        return;
    const int V = n.K >> 3;
    const long long base = row * V;
    const u32x4 *x = reinterpret_cast<const u32x4 *>(n.x) + base;
    const u32x4 *res = reinterpret_cast<const u32x4 *>(n.residual) + base;
    const u32x4 *wt = reinterpret_cast<const u32x4 *>(n.weight);
    u32x4 xv[VPT], rv[RES ? VPT : 1], gv[NORM ? VPT : 1];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = lane + i * TPR, c = v < V ? v : V - 1;
        xv[i] = x[c];
        if constexpr (RES)
            rv[i] = res[c];
    }
    if constexpr (NORM)
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = lane + i * TPR, c = v < V ? v : V - 1;
            gv[i] = wt[c];
        }
    if (n.rows_dev && n.rows < kFewRows && row >= n.rows_dev[0])
        return;
    float sq = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = lane + i * TPR;
        if constexpr (RES) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                xv[i][j] = pack_bf16x2(bf16_to_f32(xv[i][j] & 0xFFFFu) + bf16_to_f32(rv[i][j] & 0xFFFFu),
                                       bf16_to_f32(xv[i][j] >> 16) + bf16_to_f32(rv[i][j] >> 16));
            if (v < V)
                reinterpret_cast<u32x4 *>(n.sum)[base + v] = xv[i];
        }
        if (v >= V)
            xv[i] = u32x4{0u, 0u, 0u, 0u};
        if constexpr (NORM)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float a = bf16_to_f32(xv[i][j] & 0xFFFFu), b = bf16_to_f32(xv[i][j] >> 16);
                sq = __builtin_fmaf(a, a, sq);
                sq = __builtin_fmaf(b, b, sq);
            }
    }
    float rstd = 1.0f;
    if constexpr (NORM)
        rstd = 1.0f / sqrtf(row_sum<TPR>(sq, s_red) / (float)n.K + n.eps);
    auto value = [&](int i, int j) {                   // element j of vector i
        const uint32_t h = j & 1 ? xv[i][j >> 1] >> 16 : xv[i][j >> 1] & 0xFFFFu;
        if constexpr (!NORM)
            return bf16_to_f32(h);
        const uint32_t g = j & 1 ? gv[i][j >> 1] >> 16 : gv[i][j >> 1] & 0xFFFFu;
        return bf16_to_f32(h) * rstd * bf16_to_f32(g);
    };
    if constexpr (Y) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = lane + i * TPR;
            if (v < V)
                reinterpret_cast<u32x4 *>(n.y)[base + v] =
                    u32x4{pack_bf16x2(value(i, 0), value(i, 1)), pack_bf16x2(value(i, 2), value(i, 3)),
                          pack_bf16x2(value(i, 4), value(i, 5)), pack_bf16x2(value(i, 6), value(i, 7))};
        }
    }
    if constexpr (Q) {
        uint32_t top = 0;                              // magnitude bits: a NaN or infinity is above every finite one
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t m = lane + i * TPR < V ? __float_as_uint(value(i, j)) & 0x7FFFFFFFu : 0u;
                top = m > top ? m : top;
            }
        const float amax = __uint_as_float(row_max<TPR>(top, s_red));
        const bool none = !(amax >= kZeroRow) || !__builtin_isfinite(amax);
        // a power of two keeps 127 y finite for rows near the end of the range
        const float f = amax > 0x1p64f ? 0x1p-64f : 1.0f;
        const float top1 = amax * f, inv = none ? 0.0f : 1.0f / top1;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = lane + i * TPR;
            uint32_t o[2];
#pragma unroll
            for (int d = 0; d < 2; ++d) {
                o[d] = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float y = none ? 0.0f : value(i, 4 * d + j) * (127.0f * f);
                    const float t0 = y * inv;
                    const float t1 = __builtin_fmaf(__builtin_fmaf(-t0, top1, y), inv, t0);
                    o[d] |= ((uint32_t)(int)__builtin_rintf(t1) & 0xFFu) << (8 * j);
                }
            }
            if (v < V)
                reinterpret_cast<u32x2 *>(n.q)[base + v] = u32x2{o[0], o[1]};
        }
        if (lane == 0)
            n.q_scale[row] = __builtin_isfinite(amax) ? (none ? 0.0f : amax / 127.0f) : __builtin_nanf("");
    }
}

template <int TPR, int VPT>
hipError_t launch_rows(const NormLaunch &n, hipStream_t st)
{
    constexpr int RPB = TPR < 256 ? 256 / TPR : 1;
    const dim3 grid((unsigned)((n.rows + RPB - 1) / RPB)), block(TPR < 256 ? 256 : TPR);
    if (!n.weight)
        hipLaunchKernelGGL((norm_kernel<TPR, VPT, false, false, false, true>), grid, block, 0, st, n);
    else if (n.residual && n.y && n.q)
        hipLaunchKernelGGL((norm_kernel<TPR, VPT, true, true, true, true>), grid, block, 0, st, n);
    else if (n.residual && n.q)
        hipLaunchKernelGGL((norm_kernel<TPR, VPT, true, true, false, true>), grid, block, 0, st, n);
    else if (n.residual)
        hipLaunchKernelGGL((norm_kernel<TPR, VPT, true, true, true, false>), grid, block, 0, st, n);
    else if (n.y && n.q)
        hipLaunchKernelGGL((norm_kernel<TPR, VPT, false, true, true, true>), grid, block, 0, st, n);
    else if (n.q)
        hipLaunchKernelGGL((norm_kernel<TPR, VPT, false, true, false, true>), grid, block, 0, st, n);
    else
        hipLaunchKernelGGL((norm_kernel<TPR, VPT, false, true, true, false>), grid, block, 0, st, n);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_norm(const NormLaunch &n, hipStream_t st)
{
    // a wave per row while that takes at most two vectors a lane, or as long as there are rows enough to fill the
    // GPU with waves: no barriers
    if (n.K <= 512)
        return launch_rows<64, 1>(n, st);
    if (n.K <= 1024)
        return launch_rows<64, 2>(n, st);
    if (n.K <= 2048 && n.rows >= 2048)
        return launch_rows<64, 4>(n, st);
    if (n.K <= 2048)
        return launch_rows<256, 1>(n, st);
    if (n.K <= 4096)
        return launch_rows<256, 2>(n, st);
    if (n.K <= 8192)
        return launch_rows<256, 4>(n, st);
    if (n.K <= 16384)
        return launch_rows<256, 8>(n, st);
    return launch_rows<1024, 8>(n, st);
}

}  // namespace moe
