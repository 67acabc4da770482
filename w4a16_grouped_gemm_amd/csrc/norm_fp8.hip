// norm_fp8.hip -- bf16 rows to FP8 rows (e4m3, a scale for each 128 values), behind
// the RMS norm with the residual's addition or by themselves, and bf16 weights to
// FP8 blocks of 128 x 128.
//
//   h = bf16(x + residual)                 (x itself without a residual)
//   v = h * weight * rstd                  rstd = 1 / sqrt(mean h^2 + eps)
//   q = e4m3(448 v / max|v|), scale = max|v| / 448, for each block of 128
// A block's quotients do not depend on rstd: they go by the products h * weight,
// which binary32 holds exactly. The same codes come out however the sum of squares
// was formed, and values exactly between two codes go to the even one. rstd is a
// power of two, which takes the products to v's magnitude, times m in [1, 2), which
// is in the scale.
#include "fp8.hpp"
#include "gemm_core.hpp"
#include "norm_core.hpp"

namespace moe {

namespace {

__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// The power of two in v (inf for inf and NaN, 0 for a subnormal).
__device__ __forceinline__ float power_of(float v) { return __uint_as_float(__float_as_uint(v) & 0x7F800000u); }

// Eight bf16 values of a row, in binary32.
__device__ __forceinline__ void unpack_row8(u32x4 h, float (&v)[8])
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        v[2 * j] = bf16_to_f32(h[j] & 0xFFFFu);
        v[2 * j + 1] = bf16_to_f32(h[j] >> 16);
    }
}

// Codes of the eight values u of this lane, whose block is its DPP row's, to place o (in values) of the row; the
// block's scale by its first lane. Both through descriptors that hold the row and nothing more.
template <bool POW2>
__device__ __forceinline__ void store_block(const float (&u)[8], float m, __amdgpu_buffer_rsrc_t rq,
                                            __amdgpu_buffer_rsrc_t rs, uint32_t o)
{
    uint32_t top = 0;                                  // magnitude bits: a NaN or infinity is above every finite one
#pragma unroll
    for (int j = 0; j < 8; ++j)
        top = max(top, magnitude(u[j]));
    const BlockCodes block(__uint_as_float(row16_max(top)), m, POW2);
    __builtin_amdgcn_raw_buffer_store_b64(block.codes<POW2>(u), rq, o, 0, 0);
    if (o % 128 == 0)
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(block.scale), rs, o / 32, 0, 0);
}

// A row whose squares leave binary32's range (of finite values, or with a NaN or an infinity): the squares are those
// of the row times a power of two f. Small rows are taken times f, since their rstd may be too large (f times the row
// is exact); of large ones rstd is. Read again from memory, in loops, so that other rows do not pay for it.
template <int TPR, bool RES, bool Y, bool POW2>
__device__ __forceinline__ void scaled_row(const Fp8NormLaunch &n, long long row, int lane, bool small, float *s_red)
{
    const size_t at = (size_t)row * n.K;
    const uint32_t bytes = (uint32_t)n.K * 2;
    // with a residual this thread has just stored h; y may stand in x's place, so it is stored behind each read
    const __amdgpu_buffer_rsrc_t rh = make_rsrc((RES ? n.sum : n.x) + at, bytes), rg = make_rsrc(n.weight, bytes);
    const float f = small ? 0x1p90f : 0x1p-73f;
    float sq = 0.0f;
#pragma unroll 1
    for (uint32_t o = lane * 16; o < bytes; o += TPR * 16) {
        float h[8];
        unpack_row8(bload16(rh, o, 0), h);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            sq = __builtin_fmaf(h[j] * f, h[j] * f, sq);
    }
    const float sum = row_sum<TPR>(sq, s_red);
    const float rs = 1.0f / sqrtf(sum / (float)n.K + n.eps * f * f);
    const float rstd = small ? rs : rs * f, hf = small ? f : 1.0f;
    const float p2 = small ? power_of(rs) : power_of(rs) * f;
    // an infinite eps makes rs 0, and finite rows zeros; a row with an infinity is NaN
    const float m = rs == 0.0f && __builtin_isfinite(sum) ? 1.0f : rs / power_of(rs);
#pragma unroll 1
    for (uint32_t o = lane * 16; o < bytes; o += TPR * 16) {
        float h[8], g[8], u[8];
        unpack_row8(bload16(rh, o, 0), h);
        unpack_row8(bload16(rg, o, 0), g);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            u[j] = h[j] * hf * p2 * g[j];
        store_block<POW2>(u, m, make_rsrc(n.q + at, bytes / 2),
                          make_rsrc(n.q_scale + (size_t)row * (n.K / 128), bytes / 64), o / 2);
        if constexpr (Y) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                u[j] = h[j] * hf * rstd * g[j];
            __builtin_amdgcn_raw_buffer_store_b128(u32x4{bf16_pair(u[0], u[1]), bf16_pair(u[2], u[3]),
                                                         bf16_pair(u[4], u[5]), bf16_pair(u[6], u[7])},
                                                   make_rsrc(n.y + at, bytes), o, 0, 0);
        }
    }
}

// TPR threads per row (64: one wave, four rows to a workgroup; else the whole
// workgroup), each with VPT vectors of 8 values at stride TPR: 16 neighbouring
// lanes hold a block. One pass over memory, which bounds it: 8192 x 7168 with the
// residual 73 us, 5.6 TB/s of what is read and written; 1 x 2048 2.6 us.
template <int TPR, int VPT, bool RES, bool NORM, bool Y, bool POW2>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void norm_fp8_kernel(Fp8NormLaunch n)
{
    __shared__ float s_red[TPR / 64];
    constexpr int RPB = TPR < 256 ? 256 / TPR : 1;
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
        __builtin_amdgcn_sched_barrier(0);             // in the order of their use
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
        if constexpr (NORM) {
            float h[8];
            unpack_row8(xv[i], h);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                sq = __builtin_fmaf(h[j], h[j], sq);
        }
    }
    float rstd = 1.0f, p2 = 1.0f, m = 1.0f;
    if constexpr (NORM) {
        const float ms = row_sum<TPR>(sq, s_red) / (float)n.K + n.eps;
        if (__builtin_expect(out_of_range(ms), 0)) {   // all threads of a row alike
            scaled_row<TPR, RES, Y, POW2>(n, row, lane, ms < 0x1p-100f, s_red);
            return;
        }
        rstd = 1.0f / sqrtf(ms);
        p2 = power_of(rstd);
        m = rstd / p2;
    }
    const __amdgpu_buffer_rsrc_t rq = make_rsrc(n.q + at, bytes / 2),
                                 rs = make_rsrc(n.q_scale + (size_t)row * (n.K / 128), bytes / 64);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        float h[8], u[8];
        unpack_row8(xv[i], h);
        if constexpr (NORM) {
            float g[8];
            unpack_row8(gv[i], g);
            if constexpr (Y) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    u[j] = h[j] * rstd * g[j];
                __builtin_amdgcn_raw_buffer_store_b128(u32x4{bf16_pair(u[0], u[1]), bf16_pair(u[2], u[3]),
                                                             bf16_pair(u[4], u[5]), bf16_pair(u[6], u[7])},
                                                       make_rsrc(n.y + at, bytes), off[i], 0, 0);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j)
                u[j] = h[j] * p2 * g[j];
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                u[j] = h[j];
        }
        store_block<POW2>(u, m, rq, rs, off[i] / 2);
    }
}

template <int TPR, int VPT, bool POW2>
hipError_t launch_rows(const Fp8NormLaunch &n, hipStream_t st)
{
    constexpr int RPB = TPR < 256 ? 256 / TPR : 1;
    const dim3 grid((unsigned)((n.rows + RPB - 1) / RPB)), block(TPR < 256 ? 256 : TPR);
    if (!n.weight)
        hipLaunchKernelGGL((norm_fp8_kernel<TPR, VPT, false, false, false, POW2>), grid, block, 0, st, n);
    else if (n.residual && n.y)
        hipLaunchKernelGGL((norm_fp8_kernel<TPR, VPT, true, true, true, POW2>), grid, block, 0, st, n);
    else if (n.residual)
        hipLaunchKernelGGL((norm_fp8_kernel<TPR, VPT, true, true, false, POW2>), grid, block, 0, st, n);
    else if (n.y)
        hipLaunchKernelGGL((norm_fp8_kernel<TPR, VPT, false, true, true, POW2>), grid, block, 0, st, n);
    else
        hipLaunchKernelGGL((norm_fp8_kernel<TPR, VPT, false, true, false, POW2>), grid, block, 0, st, n);
    return hipGetLastError();
}

template <bool POW2>
hipError_t launch_rows_of(const Fp8NormLaunch &n, hipStream_t st)
{
    if (n.K <= 512)
        return launch_rows<64, 1, POW2>(n, st);
    if (n.K <= 1024)
        return launch_rows<64, 2, POW2>(n, st);
    if (n.K <= 2048 && n.rows >= 1024)
        return launch_rows<64, 4, POW2>(n, st);
    if (n.K <= 2048)
        return launch_rows<256, 1, POW2>(n, st);
    if (n.K <= 4096)
        return launch_rows<256, 2, POW2>(n, st);
    if (n.K <= 8192)
        return launch_rows<256, 4, POW2>(n, st);
    if (n.K <= 16384)
        return launch_rows<256, 8, POW2>(n, st);
    return launch_rows<1024, 8, POW2>(n, st);
}

// One block of 128 x 128 weights to a workgroup of 256 threads: 16 lanes to a
// row's 256 bytes, eight rows to a thread. Bound by memory, 3 bytes a value: 32 x
// 4096 x 7168 525 us (5.4 TB/s), 2112 x 7168 9.5 us (4.8).
template <bool POW2>
__global__ __launch_bounds__(256) void fp8_weights_kernel(int N, int K, const uint16_t *w, uint8_t *q, float *scale)
{
    __shared__ uint32_t s_top[4];
    const int G = K / 128, B = (N + 127) / 128;
    const int g = blockIdx.x % G, rest = blockIdx.x / G, b = rest % B, e = rest / B;
    const size_t base = ((size_t)e * N + (size_t)b * 128) * K;
    const int rows = N - b * 128 < 128 ? N - b * 128 : 128;
    // descriptors that end behind the block's last row: past them a load gives 0, which changes no maximum
    const __amdgpu_buffer_rsrc_t rw = make_rsrc(w + base, (uint32_t)rows * K * 2),
                                 rq = make_rsrc(q + base, (uint32_t)rows * K);
    u32x4 v[8];
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        o[i] = (uint32_t)(threadIdx.x / 16 + 16 * i) * K + g * 128 + threadIdx.x % 16 * 8;
        v[i] = bload16(rw, o[i] * 2, 0);
    }
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float u[8];
        unpack_row8(v[i], u);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            top = max(top, magnitude(u[j]));
    }
    top = wave_reduce(top, [](uint32_t a, uint32_t b) { return b > a ? b : a; });
    if (threadIdx.x % 64 == 0)
        s_top[threadIdx.x / 64] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i)
        top = max(top, s_top[i]);
    const BlockCodes block(__uint_as_float(top), 1.0f, POW2);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float u[8];
        unpack_row8(v[i], u);
        __builtin_amdgcn_raw_buffer_store_b64(block.codes<POW2>(u), rq, o[i], 0, 0);
    }
    if (threadIdx.x == 0)
        scale[blockIdx.x] = block.scale;
}

}  // namespace

hipError_t launch_norm_fp8(const Fp8NormLaunch &n, hipStream_t st)
{
    return n.pow2 ? launch_rows_of<true>(n, st) : launch_rows_of<false>(n, st);
}

hipError_t launch_fp8_weights(int E, int N, int K, const uint16_t *w, bool pow2, uint8_t *q, float *scale,
                              hipStream_t st)
{
    const dim3 grid((unsigned)((long long)E * ((N + 127) / 128) * (K / 128)));
    if (pow2)
        hipLaunchKernelGGL((fp8_weights_kernel<true>), grid, dim3(256), 0, st, N, K, w, q, scale);
    else
        hipLaunchKernelGGL((fp8_weights_kernel<false>), grid, dim3(256), 0, st, N, K, w, q, scale);
    return hipGetLastError();
}

}  // namespace moe
