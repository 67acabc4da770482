// norm_int8.hip -- RMS norm with the residual's addition and an int8 output, and
// the int8 row quantizer by itself (the same kernel without the norm).
//
//   h = bf16(x + residual)            (x itself without a residual)
//   y = (h * rstd) * weight           rstd = 1 / sqrt(mean h^2 + eps)
//   q = rint(127 y / max|y|), scale = max|y| / 127
// All in binary32; y is rounded to bf16 only where it is stored as bf16, so q is
// quantized from the unrounded rows. h is rounded because it is the residual
// stream that the caller keeps: the norm sees what the next layer will add to.
// A row whose squares binary32 does not hold is done apart (scaled_row).
//
// Bound by memory: a row is read once and held in registers between the two
// reductions (sum of squares, maximum). 8192 x 7168 with the residual, bf16 out,
// 82 us, 5.75 TB/s; int8 rows of 8192 x 4096 19 us (quantizer), 24 us in a run of products.
// Few rows are a chain of latencies: loads, sum, division, maximum, stores. Rows
// go through buffer descriptors of their own, so that no access needs a branch:
// behind branches the compiler does not know how many stores are under way,
// and had the second half of a row's work wait for the stores of the first (1 x 7168
// with the residual 5.0 us, now 2.7; 1 x 2048 2.8 and 2.2).
#include "gemm_core.hpp"
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

template <int TPR>
__device__ __forceinline__ uint32_t row_max(uint32_t v, float *s_red)
{
    v = wave_reduce(v, [](uint32_t a, uint32_t b) { return b > a ? b : a; });
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

// A mean of squares plus eps from which the norm is not taken: past binary32's range (or NaN), or so small that
// squares lost bits, or all of them.
__device__ __forceinline__ bool out_of_range(float ms) { return !(ms >= 0x1p-100f && ms < __builtin_inff()); }

// The norm of a row of finite values out of binary32's range for squares: the squares are those of the row times a
// power of two f, which keeps any bf16 row's within it. Small rows are taken times f, since their rstd may be too
// large (f times the row is exact); of large ones rstd is, which may make it subnormal (off by 2^-22). Read again
// from memory, three times, in loops, so that ordinary rows do not pay for it with registers (from the registers that
// hold the row, 8192 x 7168 to int8 took 40 us instead of 34).
template <int TPR, bool RES, bool Y, bool Q>
__device__ __forceinline__ void scaled_row(const NormLaunch &n, long long row, int lane, bool small, float *s_red)
{
    const size_t at = (size_t)row * n.K;
    const uint32_t bytes = (uint32_t)n.K * 2;
    // with a residual this thread has just stored h; y may stand in x's place, so it is stored after the last read
    const __amdgpu_buffer_rsrc_t rh = make_rsrc((RES ? n.sum : n.x) + at, bytes), rg = make_rsrc(n.weight, bytes);
    const float f = small ? 0x1p90f : 0x1p-73f;
    float sq = 0.0f;
#pragma unroll 1
    for (uint32_t o = lane * 16; o < bytes; o += TPR * 16) {
        const u32x4 h = bload16(rh, o, 0);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float a = bf16_to_f32(h[j] & 0xFFFFu) * f, b = bf16_to_f32(h[j] >> 16) * f;
            sq = __builtin_fmaf(a, a, sq);
            sq = __builtin_fmaf(b, b, sq);
        }
    }
    const float rs = 1.0f / sqrtf(row_sum<TPR>(sq, s_red) / (float)n.K + n.eps * f * f);
    const float rstd = small ? rs : rs * f, hf = small ? f : 1.0f;
    auto load_values = [&](uint32_t o, float (&v)[8]) {
        const u32x4 h = bload16(rh, o, 0), g = bload16(rg, o, 0);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = bf16_to_f32(h[j] & 0xFFFFu) * hf * rstd * bf16_to_f32(g[j] & 0xFFFFu);
            v[2 * j + 1] = bf16_to_f32(h[j] >> 16) * hf * rstd * bf16_to_f32(g[j] >> 16);
        }
    };
    uint32_t top = 0;
    if constexpr (Q) {
#pragma unroll 1
        for (uint32_t o = lane * 16; o < bytes; o += TPR * 16) {
            float v[8];
            load_values(o, v);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                top = max(top, __float_as_uint(v[j]) & 0x7FFFFFFFu);
        }
        top = row_max<TPR>(top, s_red);
    }
    const RowCodes row_codes(__uint_as_float(top));
#pragma unroll 1
    for (uint32_t o = lane * 16; o < bytes; o += TPR * 16) {
        float v[8];
        load_values(o, v);
        if constexpr (Q) {
            uint32_t c[2] = {0, 0};
#pragma unroll
            for (int j = 0; j < 8; ++j)
                c[j >> 2] |= row_codes.code(v[j]) << (8 * (j & 3));
            __builtin_amdgcn_raw_buffer_store_b64(u32x2{c[0], c[1]}, make_rsrc(n.q + at, bytes / 2), o / 2, 0, 0);
        }
        if constexpr (Y)
            __builtin_amdgcn_raw_buffer_store_b128(u32x4{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]),
                                                         bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7])},
                                                   make_rsrc(n.y + at, bytes), o, 0, 0);
    }
    if (Q && lane == 0)
        n.q_scale[row] = row_codes.scale;
}

// TPR threads per row (64: one wave, four rows to a workgroup; else the whole
// workgroup), each with VPT vectors of 8 values at stride TPR.
template <int TPR, int VPT, bool RES, bool NORM, bool Y, bool Q>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void norm_kernel(NormLaunch n)
{
    __shared__ float s_red[TPR / 64];
    constexpr int RPB = TPR < 256 ? 256 / TPR : 1;
    // a row that scaled_row does: behind the stores, which it then overwrites, where its row is still there (a branch
    // before them costs a single row 0.1 us), else instead of them (y in place of x)
    constexpr bool kFirst = Y && !RES;
    const int lane = threadIdx.x % TPR;
    const long long row = (long long)blockIdx.x * RPB + uniform(threadIdx.x / TPR);
    if (row >= (n.rows_dev ? n.rows_dev[0] : n.rows))
        return;                                        // whole workgroups where they meet at barriers
    const size_t at = (size_t)row * n.K;
    const uint32_t bytes = (uint32_t)n.K * 2;          // of a row: past it a load gives 0 and a store goes nowhere
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(n.x + at, bytes);
    u32x4 xv[VPT], rv[RES ? VPT : 1], gv[NORM ? VPT : 1];
    uint32_t off[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        off[i] = (uint32_t)(lane + i * TPR) * 16;
        xv[i] = bload16(rx, off[i], 0);
        if constexpr (RES)
            rv[i] = bload16(make_rsrc(n.residual + at, bytes), off[i], 0);
        __builtin_amdgcn_sched_barrier(0);             // in the order of their use (1 x 7168 2.90 us in another)
    }
    if constexpr (NORM)
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            gv[i] = bload16(make_rsrc(n.weight, bytes), off[i], 0);
    __builtin_amdgcn_sched_barrier(0);                 // all loads on their way before the first is used
    float sq = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        if constexpr (RES) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                xv[i][j] = bf16_pair(bf16_to_f32(xv[i][j] & 0xFFFFu) + bf16_to_f32(rv[i][j] & 0xFFFFu),
                                     bf16_to_f32(xv[i][j] >> 16) + bf16_to_f32(rv[i][j] >> 16));
            __builtin_amdgcn_raw_buffer_store_b128(xv[i], make_rsrc(n.sum + at, bytes), off[i], 0, 0);
        }
        if constexpr (NORM)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float a = bf16_to_f32(xv[i][j] & 0xFFFFu), b = bf16_to_f32(xv[i][j] >> 16);
                sq = __builtin_fmaf(a, a, sq);
                sq = __builtin_fmaf(b, b, sq);
            }
    }
    float ms = 1.0f, rstd = 1.0f;
    if constexpr (NORM) {
        ms = row_sum<TPR>(sq, s_red) / (float)n.K + n.eps;
        if (kFirst && __builtin_expect(out_of_range(ms), 0)) {   // all threads of a row alike
            scaled_row<TPR, RES, Y, Q>(n, row, lane, ms < 0x1p-100f, s_red);
            return;
        }
        rstd = 1.0f / sqrtf(ms);
    }
    auto value = [&](int i, int j) {                   // element j of vector i
        const uint32_t h = j & 1 ? xv[i][j >> 1] >> 16 : xv[i][j >> 1] & 0xFFFFu;
        if constexpr (!NORM)
            return bf16_to_f32(h);
        const uint32_t g = j & 1 ? gv[i][j >> 1] >> 16 : gv[i][j >> 1] & 0xFFFFu;
        return bf16_to_f32(h) * rstd * bf16_to_f32(g);
    };
    if constexpr (Y) {
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            __builtin_amdgcn_raw_buffer_store_b128(
                u32x4{bf16_pair(value(i, 0), value(i, 1)), bf16_pair(value(i, 2), value(i, 3)),
                      bf16_pair(value(i, 4), value(i, 5)), bf16_pair(value(i, 6), value(i, 7))},
                make_rsrc(n.y + at, bytes), off[i], 0, 0);
    }
    if constexpr (Q) {
        uint32_t top = 0;                              // magnitude bits: a NaN or infinity is above every finite one
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t m = __float_as_uint(value(i, j)) & 0x7FFFFFFFu;
                top = m > top ? m : top;
            }
        const float amax = __uint_as_float(row_max<TPR>(top, s_red));
        const RowCodes row_codes(amax);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            uint32_t o[2];
#pragma unroll
            for (int d = 0; d < 2; ++d) {
                o[d] = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    o[d] |= row_codes.code(value(i, 4 * d + j)) << (8 * j);
            }
            __builtin_amdgcn_raw_buffer_store_b64(u32x2{o[0], o[1]}, make_rsrc(n.q + at, bytes / 2), off[i] / 2, 0, 0);
        }
        if (lane == 0)
            n.q_scale[row] = row_codes.scale;
    }
    if (NORM && !kFirst && __builtin_expect(out_of_range(ms), 0))
        scaled_row<TPR, RES, Y, Q>(n, row, lane, ms < 0x1p-100f, s_red);
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
    // A wave per row, which needs no barriers, where that takes at most two vectors a lane (int8 quantizer, wave
    // against workgroup: 1 x 1024 2.1 and 2.1 us, 2048 x 1024 3.0 and 4.0, 16384 x 1024 10.3 and 16.6), or four once
    // there are rows enough to fill the GPU with waves (norm with residual, 1 x 2048 2.5 and 2.2 us; int8 norm, 1024 x
    // 2048 3.6 and 3.8, 16384 x 2048 24 and 29); else a workgroup of 256 (512 threads 1% either way up to 8192
    // values, 1024 threads slower at every number of rows), of 1024 past 64 values a thread.
    if (n.K <= 512)
        return launch_rows<64, 1>(n, st);
    if (n.K <= 1024)
        return launch_rows<64, 2>(n, st);
    if (n.K <= 2048 && n.rows >= 1024)
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
