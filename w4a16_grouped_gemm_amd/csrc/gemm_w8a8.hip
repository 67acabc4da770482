// gemm_w8a8.hip -- products of int8 rows: dense, and grouped over the experts'
// segments with the SwiGLU epilogue.
//
//   acc[r][n] = sum_k a[r][k] w[n][k]          exact, binary integer
//   c[r][n]   = float(acc) * as[r] * ws[n]     (binary32)
//
// MFMA: v_mfma_i32_16x16x64_i8, the weight rows as operand A and the tokens as
// operand B, so that a result lane holds four consecutive outputs of one token.
// Both operands take the same permutation of K, which leaves the sums as they are.
#include "gemm_core.hpp"
#include "w8a8.hpp"

namespace moe {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ i32x4 mfma_i8(u32x4 w, u32x4 x, i32x4 c)
{
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, w), __builtin_bit_cast(i32x4, x), c, 0, 0, 0);
}

struct W8Args {
    const int8_t *a;
    const float *as;
    const int32_t *a_row_index;
    int top_k;
    const int32_t *offsets;
    int max_rows;                // rows of c; all of them with offsets NULL
    int E;
    const int8_t *wq;
    const float *ws;
    void *c;
    int K, N;
};

// Activation row of result row r: what the index holds is kept inside the array.
__device__ __forceinline__ int act_row(const W8Args &p, int r)
{
    if (!p.a_row_index)
        return r;
    const int i = p.a_row_index[r];
    return (i < 0 ? 0 : (i < p.max_rows ? i : p.max_rows - 1)) / p.top_k;
}

// Chunk `chunk` of at most CS rows of one expert, found by one wave from the
// row offsets: false past the last chunk. Every lane gets the result.
__device__ __forceinline__ bool find_chunk(const W8Args &p, int CS, int chunk, int lane, int &e, int &r0, int &rows)
{
    if (!p.offsets) {
        e = 0;
        r0 = chunk * CS;
        rows = p.max_rows - r0;
        rows = rows < CS ? rows : CS;
        return rows > 0;
    }
    int before = 0;
    for (int e0 = 0; e0 < p.E; e0 += 64) {
        const int ee = e0 + lane < p.E ? e0 + lane : p.E - 1;
        const int o0 = p.offsets[ee], o1 = p.offsets[ee + 1];
        const int n = e0 + lane < p.E ? (o1 - o0 + CS - 1) / CS : 0;
        int total;
        const int first = before + wave_exclusive_scan(n, total);
        const uint64_t at = __ballot(first <= chunk && chunk < first + n);
        if (at) {
            const int l = __builtin_ctzll(at);
            e = e0 + l;
            const int c = chunk - __builtin_amdgcn_readlane(first, l);
            r0 = __builtin_amdgcn_readlane(o0, l) + c * CS;
            const int end = __builtin_amdgcn_readlane(o1, l);
            rows = (end < p.max_rows ? end : p.max_rows) - r0;
            rows = rows < CS ? rows : CS;
            return rows > 0 && r0 >= 0;
        }
        before += total;
    }
    return false;
}

// Few rows per expert: each wave streams its own weight rows from memory to
// registers and multiplies them with NSUB subtiles of 16 tokens; no LDS, no
// barrier. The weights are what such a call has to read, once.
template <int KIND, bool F32, int NSUB, int TPW>
__global__ __launch_bounds__(256) void w8_stream_kernel(W8Args p, int blocks)
{
    constexpr bool SW = KIND == MOE_GEMM_W13_SWIGLU;
    constexpr int TG = SW ? TPW / 2 : TPW;              // tiles side by side: a lane's outputs are 4 TG consecutive ones
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int m = lane & 15, q = lane >> 4;
    const int chunk = blockIdx.x / blocks;
    const int block = blockIdx.x - chunk * blocks;
    int e, r0, rows;
    if (!find_chunk(p, 16 * NSUB, chunk, lane, e, r0, rows))
        return;
    const int cols = SW ? p.N / 2 : p.N;                // outputs per row
    const int n0 = (block * 4 + wave) * 16 * TG;
    if (n0 >= cols)
        return;
    // weight row of lane row m in tile t: outputs n0 + (m / 4) 4 TG + 4 t + m % 4 (gate), the same + N / 2 (up)
    const int8_t *wrow[TPW];
#pragma unroll
    for (int t = 0; t < TPW; ++t) {
        int n = n0 + (m >> 2) * 4 * TG + (t % TG) * 4 + (m & 3);
        n = n < cols ? n : cols - 1;
        if (SW && t >= TG)
            n += cols;
        wrow[t] = p.wq + ((size_t)e * p.N + n) * p.K + q * 32;
    }
    const int8_t *xrow[NSUB];
    int arow[NSUB];
#pragma unroll
    for (int s = 0; s < NSUB; ++s) {
        const int r = r0 + (16 * s + m < rows ? 16 * s + m : rows - 1);
        arow[s] = act_row(p, r);
        xrow[s] = p.a + (size_t)arow[s] * p.K + q * 32;
    }
    i32x4 acc[NSUB][TPW];
#pragma unroll
    for (int s = 0; s < NSUB; ++s)
#pragma unroll
        for (int t = 0; t < TPW; ++t)
            acc[s][t] = i32x4{0, 0, 0, 0};
    for (int k = 0; k < p.K; k += 128) {
        u32x4 w[TPW][2], x[NSUB][2];
#pragma unroll
        for (int t = 0; t < TPW; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                w[t][h] = *reinterpret_cast<const u32x4 *>(wrow[t] + k + 16 * h);
#pragma unroll
        for (int s = 0; s < NSUB; ++s)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                x[s][h] = *reinterpret_cast<const u32x4 *>(xrow[s] + k + 16 * h);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int s = 0; s < NSUB; ++s)
#pragma unroll
                for (int t = 0; t < TPW; ++t)
                    acc[s][t] = mfma_i8(w[t][h], x[s][h], acc[s][t]);
    }
    const int nq = n0 + q * 4 * TG;
#pragma unroll
    for (int s = 0; s < NSUB; ++s) {
        if (16 * s + m >= rows)
            continue;
        const float as = p.as[arow[s]];
        const size_t crow = (size_t)(r0 + 16 * s + m) * cols;
#pragma unroll
        for (int t = 0; t < TG; ++t) {
            const int n = nq + 4 * t;
            if (n >= cols)
                continue;
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float *ws = p.ws + (size_t)e * p.N + n + i;
                v[i] = (float)acc[s][t][i] * as * ws[0];
                if constexpr (SW)
                    v[i] = silu_fast(v[i]) * ((float)acc[s][t + TG][i] * as * ws[cols]);
            }
            if constexpr (F32)
                *reinterpret_cast<floatx4 *>(static_cast<float *>(p.c) + crow + n) = floatx4{v[0], v[1], v[2], v[3]};
            else
                *reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(p.c) + crow + n) =
                    u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        }
    }
}

template <int KIND, bool F32>
hipError_t launch_stream(const W8GemmLaunch &g, const W8Args &p, hipStream_t st)
{
    constexpr int TPW = 4, NSUB = 2;
    constexpr int TG = KIND == MOE_GEMM_W13_SWIGLU ? TPW / 2 : TPW;
    const int cols = KIND == MOE_GEMM_W13_SWIGLU ? g.N / 2 : g.N;
    const int blocks = (cols + 64 * TG - 1) / (64 * TG);
    // at most one part-filled chunk per expert with rows, and the full ones
    const int full = g.max_rows / (16 * NSUB);
    const long long chunks = g.offsets ? (long long)full + (g.num_experts < g.max_rows ? g.num_experts : g.max_rows)
                                       : (g.max_rows + 16 * NSUB - 1) / (16 * NSUB);
    hipLaunchKernelGGL((w8_stream_kernel<KIND, F32, NSUB, TPW>), dim3((unsigned)(chunks * blocks)), dim3(256), 0, st, p,
                       blocks);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_w8_gemm(const W8GemmLaunch &g, hipStream_t st)
{
    const W8Args p{g.a, g.as, g.a_row_index, g.top_k, g.offsets, g.max_rows, g.num_experts, g.wq, g.ws, g.c, g.K, g.N};
    if (g.kind == MOE_GEMM_W13_SWIGLU)
        return launch_stream<MOE_GEMM_W13_SWIGLU, false>(g, p, st);
    if (g.c_f32)
        return launch_stream<MOE_GEMM_W2, true>(g, p, st);
    return launch_stream<MOE_GEMM_W2, false>(g, p, st);
}

}  // namespace moe
