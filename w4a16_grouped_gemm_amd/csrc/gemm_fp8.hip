// gemm_fp8.hip -- products of FP8 rows (e4m3) with a scale for each 128 values of K:
// dense, and grouped over the experts' segments with the SwiGLU epilogue.
//
//   c[r][n] = sum_g as[r][g] ws[n / 128][g] sum_{k in group g} a[r][k] w[n][k]
//
// A group's sum comes from the matrix unit (from zero, binary32), times the product
// of its two scales and onto the total by one fused multiply-add. MFMA:
// v_mfma_f32_16x16x128_f8f6f4, the weight rows as operand A and the tokens as
// operand B, so that a result lane holds four consecutive outputs of one token and
// a group is one instruction. Both operands take the same permutation of K.
//
// The matrix unit aligns the products of each run of eight e4m3 pairs to the
// largest and keeps 13 bits below it (measured, every FP8 instruction alike). A
// group's sum of normal values is off by 1.5e-5 of itself, and where the products
// of a run cancel, what is below 2^-13 of them is lost whatever the result's type.
// v_mfma_f32_16x16x32_bf16 on the widened codes adds in binary32, at half the rate
// and with the widening in the vector unit. It is taken for binary32 results, and
// for bf16 results where memory bounds the product: in the ring kernel's tiles of up
// to 32 rows (kWide), which grouped products of up to 10 expected rows take. us with
// the FP8 and the bf16 instruction: 1 x 14336 x 4096 11.3 and 11.5, 32 x 4096 x 4096
// 7.3 and 7.5, 128 x 4096 x 4096 10.9 and 11.1, 4 rows for each of 128 experts 2048 ->
// 2 x 768 65.2 and 65.4. Elsewhere bf16 results take the FP8 instruction, since the
// other one costs: 256 x 4096 x 4096 14.6 and 16.1, 300 x 4096 x 4096 16.4 and 19.5;
// in tiles of 128 x 64 16 rows for each of 128 experts 2048 -> 2 x 768 71 and 81; 64
// rows for each of 32 7168 -> 2 x 2048 178 and 252 (in tiles of 256 x 64, 256 x 128 has
// no registers for it); 4096 x 4096 x 7168 116 and 230.
#include <mutex>

#include "expert_chunks.hpp"
#include "fp8.hpp"
#include "gemm_core.hpp"
#include "lds_copy.hpp"

namespace moe {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

struct Fp8Args {
    const uint8_t *a;
    uint32_t a_bytes;
    const float *as;
    const int32_t *a_row_index;
    int top_k;
    const int32_t *offsets;
    int max_rows;                // rows of c; all of them with offsets NULL
    int E;
    const uint8_t *wq;
    const float *ws;
    void *c;
    int K, N;
};

// A lane's 32 codes of a 16 x 128 fragment: 16-byte chunks q and q + 4 of its row.
struct Frag {
    u32x4 lo, hi;
};

// Sixteen codes -> two operands of eight bf16 values.
__device__ __forceinline__ void widen(u32x4 c, bf16x8 (&o)[2])
{
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const b2 l = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[i], 1.0f, false);
        const b2 h = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[i], 1.0f, true);
        o[i >> 1][4 * (i & 1)] = l[0];
        o[i >> 1][4 * (i & 1) + 1] = l[1];
        o[i >> 1][4 * (i & 1) + 2] = h[0];
        o[i >> 1][4 * (i & 1) + 3] = h[1];
    }
}

// A fragment as the matrix unit takes it: codes, or bf16 values (WIDE).
template <bool WIDE>
struct Operand;

template <>
struct Operand<false> {
    i32x8 v;
    __device__ __forceinline__ explicit Operand(const Frag &f)
    {
        v = __builtin_bit_cast(i32x8, f);
    }
};

template <>
struct Operand<true> {
    bf16x8 v[4];
    __device__ __forceinline__ explicit Operand(const Frag &f)
    {
        bf16x8 t[2];
        widen(f.lo, t);
        v[0] = t[0];
        v[1] = t[1];
        widen(f.hi, t);
        v[2] = t[0];
        v[3] = t[1];
    }
};

// The sum over a group: 16 weight rows x 16 tokens.
__device__ __forceinline__ floatx4 group_sum(const Operand<false> &w, const Operand<false> &x)
{
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w.v, x.v, floatx4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}

__device__ __forceinline__ floatx4 group_sum(const Operand<true> &w, const Operand<true> &x)
{
    floatx4 c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.v[i], x.v[i], c, 0, 0, 0);
    return c;
}

__device__ __forceinline__ void add_scaled(floatx4 &tot, float s, floatx4 c)
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        tot[i] = __builtin_fmaf(s, c[i], tot[i]);
}

// v is in vector registers here, as if it were read.
__device__ __forceinline__ void keep(floatx4 v) { asm volatile("" ::"v"(v[0]), "v"(v[1]), "v"(v[2]), "v"(v[3])); }

__device__ __forceinline__ float load_f32(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff)
{
    return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, voff, soff, 0));
}

// The scales of expert e's weights: a row of K / 128 for each 128 weight rows.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t scale_rsrc(const Fp8Args &p, int e)
{
    const int B = (p.N + 127) / 128, G = p.K / 128;
    return make_rsrc(p.ws + (size_t)e * B * G, (uint32_t)B * G * 4);
}

// ---------------------------------------------------------------------------
// Few rows or few workgroups: the weights are what such a call has to read, once.
// Each wave streams its own weight rows, TPW tiles of 16, and its chunk's NSUB
// subtiles of 16 tokens through a part of LDS that no other wave sees, D groups of K
// ahead: copies straight from memory, eight lanes to a row's 128 bytes, waited for by
// count, and no meeting of the waves. WK waves of a workgroup share a set of weight
// rows, each with its part of K, and add their sums in the waves' order in the end.
//
// Loads to the registers of the lanes that multiply them take 16 bytes of a row
// each and pass the cache one lane at a time: 16 x 14336 x 4096 17.1 us that way and
// 14.2 here, 64 x 4096 x 4096 12.1 and 8.7. Weights that are read once (ONCE) come
// non-temporally, which leaves the caches to the tokens: 16 x 14336 x 4096 13.2, 1 x
// 14336 x 4096 11.2 (5.2 TB/s) instead of 12.4; 333 x 2112 x 7168, six chunks to a weight,
// would take 20.6 instead of 18.0. Experts with a few rows each, more workgroups than
// run at a time: a wave takes all of K. 128 experts with 4 rows each, 2048 -> 2 x 768, 64 us (6.2
// TB/s), in registers 76, there non-temporally 89 (the two halves of a line are fetched
// apart and the second finds it gone); 4096 -> 2048 172 (6.1 TB/s) and 188. Of these an
// expert with several chunks has its weights read by each of them, so by way of the
// caches: 64 and 100 tokens on 128 experts by Zipf's law (up to 64 and 99 rows for one)
// 57.3 us instead of 58.9, 65.8 instead of 68.9, 32 tokens on 32 experts of 7168 -> 2 x 2048
// 158 instead of 175, 2048 -> 7168 75 instead of 83, but 768 -> 2048 34.4 instead of 34.1
// and 41.8 instead of 40.2. Two loops, since a choice at each copy took 1 us of 50.
//
// Chunks of a dense product side by side on an XCD: 333 x 2112 x 7168 (33 column
// blocks, which wander over the XCDs else) 22.1 -> 19.7 us; with the multiply-adds
// three products behind their sums 19.5, binary32 results 24.4 -> 23.3, 256 x 4096 x
// 4096 15.1 -> 14.8. What bounds it there is the way of the copies into LDS, 128 KiB
// under way in each CU: weights that were touched ahead into L2 did not help.
// ---------------------------------------------------------------------------
// Copies and loads of a wave that went out behind those of a quad's group j when its turn comes: the groups after it,
// and the next quads' scales in between.
constexpr int stream_behind(int D, int j, int copies, int scales)
{
    return (D - 1) * copies + (D == 4 || j == 1 || j == 2 ? scales : 0);
}

template <int KIND, bool F32, int NSUB, int TPW, int WK, int D, bool ONCE>
__global__ __launch_bounds__(256, NSUB * TPW > 8 ? 1 : 2) void fp8_ring_kernel(Fp8Args p, int blocks)
{
    constexpr bool SW = KIND == MOE_GEMM_W13_SWIGLU;
    constexpr bool kWide = F32 || NSUB <= 2;            // sums in binary32
    constexpr int TG = SW ? TPW / 2 : TPW;              // tiles side by side: a lane's outputs are 4 TG consecutive ones
    constexpr int WN = 4 / WK, H = SW ? 2 : 1;
    constexpr int C = 2 * (TPW + NSUB), kScales = NSUB + H;   // copies of a group, loads of a quad's scales
    constexpr int kSlot = C * 1024, kWave = D * kSlot;
    static_assert(D == 2 || D == 4, "groups of a quad");
    extern __shared__ __align__(16) unsigned char s_dyn[];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int m = lane & 15, q = lane >> 4;
    const int wn = wave / WK, wk = wave % WK;
    int chunk = blockIdx.x / blocks;
    int block = blockIdx.x - chunk * blocks;
    if (!p.offsets) {                                   // the chunks beside each other on one XCD, whose L2 keeps their weights
        const int chunks = gridDim.x / blocks, i = xcd_share(gridDim.x, blockIdx.x);
        block = i / chunks;
        chunk = i - block * chunks;
    }
    int e, r0, rows;
    bool once = ONCE;                                   // the weights come non-temporally: where the expert has one chunk
    if (!find_chunk<false>(p, 16 * NSUB, chunk, lane, e, r0, rows, ONCE && WK == 1 ? &once : nullptr))
        return;
    e = uniform(e);
    const int cols = SW ? p.N / 2 : p.N;                // outputs per row
    const int n0 = (block * WN + wn) * 16 * TG;
    if (WK == 1 && n0 >= cols)
        return;
    const int G = p.K / 128;
    const __amdgpu_buffer_rsrc_t ri = index_rsrc(p), rxs = make_rsrc(p.as, p.a_bytes / 32), rws = scale_rsrc(p, e);
    const uint8_t *wbase = p.wq + (size_t)e * p.N * p.K;
    // rows whose chunk this lane copies, 8 rows to a copy; place l of a row's eight 16-byte chunks holds chunk l ^ (row / 2)
    const uint32_t place = (uint32_t)((lane & 7) ^ ((lane >> 4) & 3)) * 16;
    int row[2 * NSUB], idx[2 * NSUB], srow[NSUB], sidx[NSUB];
#pragma unroll
    for (int j = 0; j < 2 * NSUB; ++j) {
        const int r = 8 * j + (lane >> 3);
        row[j] = r0 + (r < rows ? r : rows - 1);
        idx[j] = load_index(ri, row[j]);
    }
#pragma unroll
    for (int s = 0; s < NSUB; ++s) {
        srow[s] = r0 + (16 * s + m < rows ? 16 * s + m : rows - 1);
        sidx[s] = load_index(ri, srow[s]);
    }
    // weight row of lane row m in tile t: outputs n0 + (m / 4) 4 TG + 4 t + m % 4 (gate), the same + N / 2 (up)
    uint32_t wo[2 * TPW], xo[2 * NSUB], so[NSUB];
#pragma unroll
    for (int j = 0; j < 2 * TPW; ++j) {
        const int t = j / 2, r = (j & 1) * 8 + (lane >> 3);
        int n = n0 + (r >> 2) * 4 * TG + (t % TG) * 4 + (r & 3);
        n = n < cols ? n : cols - 1;
        wo[j] = (uint32_t)(n + (SW && t >= TG ? cols : 0)) * p.K + (place ^ (uint32_t)(j & 1) * 64);
    }
    // 16 TG columns from a multiple of 16 TG on are all of one block of 128
    const uint32_t ws0 = (uint32_t)(n0 < cols ? n0 : cols - 1) / 128 * G * 4, ws1 = ws0 + (uint32_t)(cols / 128) * G * 4;
    // groups [g, end) are this wave's; those past them are copied from arrays of no bytes, to keep the count
    int g = wk * G / WK;
    const int end = (wk + 1) * G / WK;
    lds_byte *lds = (lds_byte *)s_dyn + wave * kWave;
    auto copy_w = [&](auto nt, int k, int slot) {
        const __amdgpu_buffer_rsrc_t rw = make_rsrc(wbase, k < end ? (uint32_t)p.N * p.K : 0u);
#pragma unroll
        for (int j = 0; j < 2 * TPW; ++j)
            copy16<decltype(nt)::value>(rw, lds + slot * kSlot + j * 1024, wo[j], k < end ? k * 128 : 0);
    };
    auto copy_x = [&](int k, int slot) {
        const __amdgpu_buffer_rsrc_t rx = make_rsrc(p.a, k < end ? p.a_bytes : 0u);
#pragma unroll
        for (int j = 0; j < 2 * NSUB; ++j)
            copy16(rx, lds + slot * kSlot + (2 * TPW + j) * 1024, xo[j], k < end ? k * 128 : 0);
    };
    struct Scales {                                     // of four groups
        floatx4 x[NSUB], w[H];
    };
    auto load_scales = [&](Scales &s, int k) {
#pragma unroll
        for (int i = 0; i < NSUB; ++i)
            s.x[i] = __builtin_bit_cast(floatx4, bload16(rxs, so[i] + k * 4, 0));
        s.w[0] = __builtin_bit_cast(floatx4, bload16(rws, ws0 + k * 4, 0));
        if constexpr (SW)
            s.w[1] = __builtin_bit_cast(floatx4, bload16(rws, ws1 + k * 4, 0));
    };
    // the first weights set out before the tokens' rows are known
    const std::integral_constant<bool, ONCE> first{};   // these non-temporally in any case
    copy_w(first, g, 0);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < 2 * NSUB; ++j)
        xo[j] = (uint32_t)act_row(p, row[j], idx[j]) * p.K + (place ^ (uint32_t)(j & 1) * 64);
#pragma unroll
    for (int s = 0; s < NSUB; ++s)
        so[s] = (uint32_t)act_row(p, srow[s], sidx[s]) * G * 4;
    Scales sc, sn, sl;                                  // the quad's, the next one's, those under way
    load_scales(sc, g);
    if constexpr (D == 2)
        load_scales(sn, g + 4);
    __builtin_amdgcn_sched_barrier(0);
    copy_x(g, 0);
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (D == 4)
        load_scales(sn, g + 4);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 1; j < D; ++j) {
        copy_w(first, g + j, j);
        copy_x(g + j, j);
    }
    floatx4 acc[NSUB][TPW];
#pragma unroll
    for (int s = 0; s < NSUB; ++s)
#pragma unroll
        for (int t = 0; t < TPW; ++t)
            acc[s][t] = floatx4{0.f, 0.f, 0.f, 0.f};
    // fragment reads: lane l holds chunks l / 16 and l / 16 + 4 of row l % 16
    const uint32_t f0 = (uint32_t)(wave * kWave + m * 128 + ((q ^ (m >> 1)) & 7) * 16);
    auto fragment = [&](int slot, int i) {
        Frag f;
        f.lo = *reinterpret_cast<const u32x4 *>(s_dyn + f0 + slot * kSlot + i * 2048);
        f.hi = *reinterpret_cast<const u32x4 *>(s_dyn + (f0 ^ 64u) + slot * kSlot + i * 2048);
        return f;
    };
    auto turn = [&](auto nt, auto turn_of) {
        constexpr int J = decltype(turn_of)::value, SLOT = J % D;
        wait_for<stream_behind(D, J, C, kScales)>();
        if (g + J < end) {
            Frag w[TPW];
#pragma unroll
            for (int t = 0; t < TPW; ++t)
                w[t] = fragment(SLOT, t);
            constexpr int kLag = NSUB * TPW > 3 ? 3 : NSUB * TPW - 1;   // products between a group's sum and its use
            floatx4 c[kLag + 1];
            auto add = [&](int i) {
                const int s = i / TPW, t = i % TPW;
                add_scaled(acc[s][t], sc.x[s][J] * sc.w[SW && t >= TG ? 1 : 0][J], c[i % (kLag + 1)]);
                keep(acc[s][t]);
            };
#pragma unroll
            for (int s = 0; s < NSUB; ++s) {
                const Operand<kWide> xv(fragment(SLOT, TPW + s));
#pragma unroll
                for (int t = 0; t < TPW; ++t) {
                    const int i = s * TPW + t;
                    c[i % (kLag + 1)] = group_sum(Operand<kWide>(w[t]), xv);
                    if (i >= kLag)
                        add(i - kLag);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
#pragma unroll
            for (int i = NSUB * TPW - kLag; i < NSUB * TPW; ++i)
                add(i);
        }
        // every fragment has left LDS
        __builtin_amdgcn_sched_barrier(0);
        copy_w(nt, g + J + D, SLOT);
        copy_x(g + J + D, SLOT);
        __builtin_amdgcn_sched_barrier(0);
    };
    auto groups = [&](auto nt) {
        for (; g < end; g += 4) {
            turn(nt, std::integral_constant<int, 0>());
            load_scales(sl, g + 8);
            __builtin_amdgcn_sched_barrier(0);
            turn(nt, std::integral_constant<int, 1>());
            turn(nt, std::integral_constant<int, 2>());
            turn(nt, std::integral_constant<int, 3>());
            sc = sn;
            sn = sl;
        }
    };
    if (once)
        groups(std::true_type());
    else
        groups(std::false_type());
    wait_for<0>();                                      // copies past the last group write to LDS too
    if constexpr (WK > 1) {
        floatx4 *part = reinterpret_cast<floatx4 *>(s_dyn);   // [WN][WK - 1][NSUB TPW][64]
        __syncthreads();
#pragma unroll
        for (int s = 0; s < NSUB; ++s)
#pragma unroll
            for (int t = 0; t < TPW; ++t)
                if (wk > 0)
                    part[((wn * (WK - 1) + wk - 1) * NSUB * TPW + s * TPW + t) * 64 + lane] = acc[s][t];
        __syncthreads();
        if (wk > 0)
            return;
#pragma unroll
        for (int i = 0; i < WK - 1; ++i)
#pragma unroll
            for (int s = 0; s < NSUB; ++s)
#pragma unroll
                for (int t = 0; t < TPW; ++t)
                    acc[s][t] += part[((wn * (WK - 1) + i) * NSUB * TPW + s * TPW + t) * 64 + lane];
    }
    const int nq = n0 + q * 4 * TG;
#pragma unroll
    for (int s = 0; s < NSUB; ++s) {
        if (16 * s + m >= rows)
            continue;
        const size_t crow = (size_t)(r0 + 16 * s + m) * cols;
#pragma unroll
        for (int t = 0; t < TG; ++t) {
            const int n = nq + 4 * t;
            if (n >= cols)
                continue;
            floatx4 v = acc[s][t];
            if constexpr (SW)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    v[i] = silu_fast(v[i]) * acc[s][t + TG][i];
            if constexpr (F32)
                *reinterpret_cast<floatx4 *>(static_cast<float *>(p.c) + crow + n) = v;
            else
                *reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(p.c) + crow + n) =
                    u32x2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
        }
    }
}

// A kernel's LDS limit is raised once on each device that launches it.
template <class Kernel, Kernel *kernel, int BYTES>
void allow_lds()
{
    constexpr int kMaxDevices = 64;
    static std::once_flag once[kMaxDevices];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices)
        return;
    std::call_once(once[dev], [] {
        (void)hipFuncSetAttribute(reinterpret_cast<const void *>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, BYTES);
    });
}

template <int KIND, bool F32, int NSUB, int TPW, int WK, int D, bool ONCE = false>
hipError_t launch_ring(const Fp8GemmLaunch &g, const Fp8Args &p, hipStream_t st)
{
    constexpr int TG = KIND == MOE_GEMM_W13_SWIGLU ? TPW / 2 : TPW;
    const int cols = KIND == MOE_GEMM_W13_SWIGLU ? g.N / 2 : g.N;
    constexpr int BC = 16 * TG * (4 / WK), kBytes = 4 * D * 2 * (TPW + NSUB) * 1024;
    static_assert(kBytes >= 4 * NSUB * TPW * 1024, "the waves' sums fit");
    const int blocks = (cols + BC - 1) / BC;
    allow_lds<decltype(fp8_ring_kernel<KIND, F32, NSUB, TPW, WK, D, ONCE>), fp8_ring_kernel<KIND, F32, NSUB, TPW, WK, D, ONCE>,
              kBytes>();
    hipLaunchKernelGGL((fp8_ring_kernel<KIND, F32, NSUB, TPW, WK, D, ONCE>),
                       dim3((unsigned)(chunks_at_most(g, 16 * NSUB) * blocks)), dim3(256), kBytes, st, p, blocks);
    return hipGetLastError();
}

// Tiles of 16 rows; of up to 16 rows in all, the weights are read once.
template <int KIND, bool F32, int TPW, int WK, int D>
hipError_t launch_ring_16(const Fp8GemmLaunch &g, const Fp8Args &p, hipStream_t st)
{
    if constexpr (KIND == MOE_GEMM_W2)
        if (!g.offsets && g.max_rows <= 16)
            return launch_ring<KIND, F32, 1, TPW, WK, D, true>(g, p, st);
    return launch_ring<KIND, F32, 1, TPW, WK, D>(g, p, st);
}

// ---------------------------------------------------------------------------
// Many rows per expert: a workgroup computes 64 TN weight rows x 16 TM tokens.
// Four of its eight waves multiply, 16 TN rows by all the tokens each; the other
// four copy both from memory straight to LDS, a group of K (128 bytes) to a stage
// and kStages stages deep, and wait for the copies. A wave that multiplies issues
// no copy: where it did, it stood behind the other waves' at the address unit (16
// cycles a copy) while its matrix unit ran dry.
//
// The tokens' fragments are read from LDS as they are needed, the weights' a stage
// ahead into registers, which leaves their place to the group after the next two.
// Scales come 16 bytes (four groups) at a time. Weights that are read once, of experts
// with one chunk of rows, come non-temporally.
//
// A workgroup takes tile after tile, and the copies of the next one's first stages
// go out under the last products of this one: neither the way from memory to the
// first product nor the stores behind the last leave the memory or the matrix unit
// idle between two tiles.
//
// A stage's rows are 128 bytes, eight 16-byte chunks each; row r keeps chunk c at
// place c ^ ((r >> 1) & 7), so that the 64 lanes of a fragment read (16 rows x 4
// chunks) meet no bank conflict. Eight lanes copy a row's 128 bytes: weights loaded
// by the lanes that multiply them, each from a row of its own, come at 16 bytes a
// cycle and CU, a quarter of this.
//
// A group's sums come out of the matrix unit kDelay instructions before their
// multiply-adds onto the totals, which so run beside the next products: with one
// instead of three 4096 x 4096 x 7168 takes 131 us instead of 115.
//
// us, tiles of 256 x 128: 4096 x 4096 x 7168 115 (2.1 PFLOP/s), 8192 x 8192 x 8192
// 482 (2.3), 8192 x 14336 x 4096 452, with a tile to a workgroup 465; 2048 rows on 32
// experts, 7168 -> 2 x 2048, 168 (940 MB of weights at 5.6 TB/s), 2048 -> 7168 100,
// with weights by way of the caches 180 and 108, and with a tile to a workgroup 186 and
// 111 then. The large ones are bound by the copies:
// without them (the operands of the first three groups over and over) the first
// three take 91, 374 and 364, at the clock that the matrix unit holds; all copies
// from L2 instead of memory gain 6%.
// ---------------------------------------------------------------------------
constexpr int kDelay = 3;                             // MFMAs between a group's sum and its use
constexpr int kStages = 3;                            // places for tokens and for weights
constexpr int kTilesAhead = 4;                        // groups that K must have where a workgroup takes several tiles

template <int TN, int TM>
struct TileLds {                                      // where things are, in bytes
    static constexpr int kTokens = 16 * TM * 128, kWeights = 64 * TN * 128;   // of a stage
    static constexpr int kW = kStages * kTokens, kScale = kW + kStages * kWeights;
    // scales of four groups: 1 KiB for 64 tokens each, 1 KiB for the weights; three places, as a tile's last may serve one stage
    static constexpr int kScaleCopies = (16 * TM + 63) / 64, kScales = (kScaleCopies + 1) * 1024;
    static constexpr int kTile = kScale + 3 * kScales, kBytes = kTile + 2 * 16;
};

// The meeting of all waves: stores to LDS before it are seen behind it.
__device__ __forceinline__ void meet()
{
    __builtin_amdgcn_sched_barrier(0);
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_s_barrier();
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_sched_barrier(0);
}

// Whether expert e's rows are all in one chunk of CS: its weights are read once then.
__device__ __forceinline__ bool read_once(const Fp8Args &p, int CS, int e)
{
    const uint32_t rows = p.offsets ? (uint32_t)p.offsets[e + 1] - (uint32_t)p.offsets[e] : (uint32_t)p.max_rows;
    return uniform(rows <= (uint32_t)CS);
}

template <int KIND, bool F32, int TN, int TM>
__global__ __launch_bounds__(512, TN > 2 ? 2 : 4) void fp8_tile_kernel(Fp8Args p, int tn)
{
    using S = TileLds<TN, TM>;
    constexpr bool SW = KIND == MOE_GEMM_W13_SWIGLU;
    constexpr int TG = SW ? TN / 2 : TN, H = SW ? 2 : 1;
    constexpr int BM = 16 * TM, BC = 64 * TG;           // tokens, output columns
    extern __shared__ __align__(16) unsigned char s_dyn[];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int wn = wave & 3;
    const int cols = SW ? p.N / 2 : p.N;
    const int G = p.K / 128;
    // Tile i of this workgroup for the waves that multiply: first row, rows, column tile, whether another follows
    struct Tile {
        int r0, rows, nt, more;
    };
    Tile *s_tile = reinterpret_cast<Tile *>(s_dyn + S::kTile);      // tile i in place i % 2
    // Stage s, counted over all tiles, takes place s % kStages. The waves meet before the first stage and in the middle of
    // each stage s: then stage s + 1 is whole, every wave has read all tokens of stage s - 1, whose place takes those of
    // stage s + 2, and has the weights of stage s in registers, whose place takes those of stage s + 3.
    if (wave >= 4) {
        constexpr int L = TM / 2, LW = 2 * TN;          // copies of a wave per stage: tokens, weights
        const uint32_t K = (uint32_t)p.K;
        const __amdgpu_buffer_rsrc_t ri = index_rsrc(p);
        lds_byte *lds = (lds_byte *)s_dyn;
        Chunks chunks;
        const int tm = uniform(min(count_chunks(p, BM, lane, chunks), most_chunks(p, BM)));
        // where a tile's copies read from: this lane's rows of weights and tokens, a chunk of each, and of scales
        struct From {
            int e;
            bool once;
            uint32_t w[LW], x[L], ws, xs;
        };
        const uint32_t chunk = (uint32_t)((lane & 7) ^ ((lane >> 4) & 3)) * 16;   // of this lane's row in copies of rows 0 .. 7 of 16
        int xrow[L + 1], xidx[L + 1];                   // rows whose tokens this lane copies; whose scales
        auto find = [&](int b, Tile &t, From &f) {      // tile b: what follows from its place alone, and the index on its way
            int mt = 0, nt = 0, e, r0, rows, next_m, next_n;
            t = Tile{0, 0, -1, 0};
            if (!have_tile(tm, tn, b, mt, nt))
                return false;
            if (!rows_of_tile(p, BM, mt, lane, chunks, e, r0, rows))
                e = r0 = rows = 0;                      // not reached: offsets are clamped; would compute and store nothing
            f.e = uniform(e);
            f.once = read_once(p, BM, f.e);
            t.r0 = uniform(r0);
            t.rows = uniform(rows);
            t.nt = nt;
            const int row1 = t.rows > 1 ? t.rows - 1 : 0;
            t.more = have_tile(tm, tn, b + (int)gridDim.x, next_m, next_n) ? 1 : 0;
#pragma unroll
            for (int j = 0; j <= L; ++j) {
                const int row = j < L ? (wn * L + j) * 8 + (lane >> 3) : wn * 64 + lane;
                xrow[j] = t.r0 + (row < row1 ? row : row1);
                xidx[j] = load_index(ri, xrow[j]);
            }
            // row m of a multiplying wave's tile a is output (m / 4) 4 TG + 4 a + m % 4
            const int nw = nt * BC + wn * 16 * TG;
#pragma unroll
            for (int j = 0; j < LW; ++j) {
                const int a = j / 2, r = (j & 1) * 8 + (lane >> 3);
                int n = nw + (r >> 2) * 4 * TG + (a % TG) * 4 + (r & 3);
                n = n < cols ? n : cols - 1;
                f.w[j] = (uint32_t)(n + (SW && a >= TG ? cols : 0)) * K + (chunk ^ (uint32_t)(j & 1) * 64);
            }
            // the (up to) two blocks of 128 weight rows that the tile's columns are in, one to the even lanes, one to the odd
            const int last = (cols - 1) / 128, b0 = nt * BC / 128;
            const int b1 = SW ? b0 + cols / 128 : (b0 + 1 < last ? b0 + 1 : last);
            f.ws = (uint32_t)((lane & 1 ? b1 : b0) * G) * 4;
            return true;
        };
        auto find_rows = [&](From &f) {                 // the rest, of the index
#pragma unroll
            for (int j = 0; j < L; ++j)
                f.x[j] = (uint32_t)act_row(p, xrow[j], xidx[j]) * K + (chunk ^ (uint32_t)((wn * L + j) & 1) * 64);
            f.xs = (uint32_t)act_row(p, xrow[L], xidx[L]) * G * 4;
        };
        const __amdgpu_buffer_rsrc_t rx = make_rsrc(p.a, p.a_bytes), rxs = make_rsrc(p.as, p.a_bytes / 32);
        auto copy_w = [&](const From &f, int g, int at) {
            const __amdgpu_buffer_rsrc_t rw = make_rsrc(p.wq + (size_t)f.e * p.N * K, (uint32_t)p.N * K);
            auto copies = [&](auto nt) {
#pragma unroll
                for (int j = 0; j < LW; ++j)
                    copy16<decltype(nt)::value>(rw, lds + S::kW + at * S::kWeights + (wn * LW + j) * 1024, f.w[j], g * 128);
            };
            if (f.once)
                copies(std::true_type());
            else
                copies(std::false_type());
        };
        int scale_at = 2 * S::kScales;                  // the last place that scales went to
        auto copy_x = [&](const From &f, int g, int at) {   // and the scales of groups g .. g + 3
            if ((g & 3) == 0) {
                scale_at = scale_at == 2 * S::kScales ? 0 : scale_at + S::kScales;
                if (wn < S::kScaleCopies)
                    copy16(rxs, lds + S::kScale + scale_at + wn * 1024, f.xs + g * 4, 0);
                else if (wn == 3)
                    copy16(scale_rsrc(p, f.e), lds + S::kScale + scale_at + S::kScaleCopies * 1024, f.ws + g * 4, 0);
            }
#pragma unroll
            for (int j = 0; j < L; ++j)
                copy16(rx, lds + at * S::kTokens + (wn * L + j) * 1024, f.x[j], g * 128);
        };
        Tile tile;
        From from, next;
        int b = blockIdx.x;
        const bool any = find(b, tile, from);
        if (wave == 4)
            s_tile[0] = tile;
        if (!any) {
            __builtin_amdgcn_s_waitcnt(vmcnt_imm(63) & ~(15u << 8));
            meet();
            return;
        }
        // the weights set out before the tokens' rows are known
        copy_w(from, 0, 0);
        find_rows(from);
        copy_x(from, 0, 0);
        if (G > 1) {
            copy_w(from, 1, 1);
            copy_x(from, 1, 1);
        }
        if (G > 2)
            copy_w(from, 2, 2);
        // In flight behind what a meeting needs: at the first one stage 1 and the weights of stage 2, later the weights of
        // stage s + 2. Where the stages end, fewer are, and all are waited for.
        __builtin_amdgcn_s_waitcnt(vmcnt_imm(63) & ~(15u << 8));
        if (G > 2)
            wait_for<L + 2 * LW>();
        else
            wait_for<0>();
        meet();
        int at = 0;                                     // place of stage s
        for (int i = 1;; ++i) {
            const bool more = tile.more;
            for (int g = 0; g < G; ++g) {
                if (g + 2 < G || more)
                    wait_for<LW>();
                else
                    wait_for<0>();
                meet();
                if (more) {                             // then G >= kTilesAhead: both steps come before the next tile's first copy
                    if (g == 0) {
                        b += gridDim.x;
                        find(b, tile, next);
                        if (wave == 4)
                            s_tile[i & 1] = tile;
                        __builtin_amdgcn_s_waitcnt(vmcnt_imm(63) & ~(15u << 8));
                    }
                    if (g == 1)
                        find_rows(next);
                }
                const int at2 = at == 0 ? 2 : at - 1;
                if (g + 2 < G)
                    copy_x(from, g + 2, at2);
                else if (more)
                    copy_x(next, g + 2 - G, at2);
                if (g + 3 < G)
                    copy_w(from, g + 3, at);
                else if (more)
                    copy_w(next, g + 3 - G, at);
                at = at == 2 ? 0 : at + 1;
            }
            if (!more)
                return;
            from = next;
        }
    }

    constexpr int XR = TM % 8 == 0 ? 4 : 2;             // token fragments in registers
    constexpr int M = TN * TM / 2;                      // MFMAs of half a stage
    static_assert(TM % XR == 0 && M % (kDelay + 1) == 0 && TN * XR > kDelay, "rings");
    static_assert(XR - 1 <= TM / 2, "the next stage's fragments are read in a stage's second half only");
    const int m = lane & 15, q = lane >> 4;
    // fragment reads: lane l holds chunks l / 16 and l / 16 + 4 of row l % 16
    const uint32_t f0 = (uint32_t)(m * 128 + ((q ^ (m >> 1)) & 7) * 16);
    const uint32_t f1 = f0 ^ 64u;
    Frag x[XR];
    float xs[XR], sc[XR][H];
    Frag w[2][TN];
    // one of the 2 TN reads of a group's weight fragments
    auto read_w = [&](Frag (&f)[TN], int j, uint32_t at) {
        const unsigned char *src = s_dyn + S::kW + at + wn * (2048 * TN) + j / 2 * 2048;
        if (j & 1)
            f[j / 2].hi = *reinterpret_cast<const u32x4 *>(src + f1);
        else
            f[j / 2].lo = *reinterpret_cast<const u32x4 *>(src + f0);
    };
    // one of the three reads of token fragment b: its two chunks, its scales
    auto read_x = [&](int j, int b, uint32_t at, uint32_t scale_at) {
        if (j == 0)
            x[b % XR].lo = *reinterpret_cast<const u32x4 *>(s_dyn + at + f0 + b * 2048);
        else if (j == 1)
            x[b % XR].hi = *reinterpret_cast<const u32x4 *>(s_dyn + at + f1 + b * 2048);
        else
            xs[b % XR] = *reinterpret_cast<const float *>(s_dyn + scale_at + m * 16 + b * 256);
    };
    floatx4 tot[TN][TM], c[kDelay + 1];
    auto add = [&](int i) {                             // product i of a stage onto its total, here and not where that is used
        const int a = i % TN, b = i / TN;
        add_scaled(tot[a][b], sc[b % XR][SW && a >= TG ? 1 : 0], c[i % (kDelay + 1)]);
        keep(tot[a][b]);
    };
    float wsv[H];
    uint32_t cur = 0, wcur = 0, scur = S::kScale;       // places of stage g, and of its scales
    auto read_ws = [&](float (&v)[H], int wsb, uint32_t scale_at) {
#pragma unroll
        for (int h = 0; h < H; ++h)
            v[h] = *reinterpret_cast<const float *>(s_dyn + S::kScaleCopies * 1024 + scale_at + (SW ? h : wsb) * 16);
    };
    // Half a stage: products of token fragments [HALF TM / 2, ...), XR - 1 fragments read ahead (those of stage g + 1,
    // at `nxt`, behind the last). Between two products stand the multiply-adds of an earlier one and what there is to
    // read, in this order: the compiler's own is full of waits.
    auto half_stage = [&](auto half, const Frag (&f)[TN], uint32_t nxt, uint32_t snxt, auto read, auto reads) {
        constexpr int HALF = decltype(half)::value, READS = decltype(reads)::value;
#pragma unroll
        for (int k = 0; k < TM / 2; ++k) {
            const int b = HALF * TM / 2 + k, ahead = b + XR - 1;
            const Operand<F32> xv(x[b % XR]);
#pragma unroll
            for (int a = 0; a < TN; ++a) {
                const int i = b * TN + a, at = k * TN + a;
                c[i % (kDelay + 1)] = group_sum(Operand<F32>(f[a]), xv);
#pragma unroll
                for (int j = spread_to(a, 3, TN); j < spread_to(a + 1, 3, TN); ++j)
                    read_x(j, ahead % TM, ahead < TM ? cur : nxt, ahead < TM ? scur : snxt);
#pragma unroll
                for (int j = spread_to(at, READS, M); j < spread_to(at + 1, READS, M); ++j)
                    read(j);
                add((i + TN * TM - kDelay) % (TN * TM));
                if (a == 0) {
#pragma unroll
                    for (int h = 0; h < H; ++h)
                        sc[b % XR][h] = xs[b % XR] * wsv[h];
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    };
    using Half0 = std::integral_constant<int, 0>;
    using Half1 = std::integral_constant<int, 1>;
    int wsb, wsb_next;                                  // which of the tile's two blocks of weight rows the wave's are in
    auto block_of = [&](int nt) {
        const int n0 = nt * BC, nw = n0 + wn * 16 * TG;
        return SW || nw >= cols ? 0 : nw / 128 - n0 / 128;
    };
    // the last stage of a tile reads ahead of the next one's first
    auto stage = [&](const Frag (&f)[TN], Frag (&fn)[TN], int g) {
        const uint32_t nxt = cur == 2 * S::kTokens ? 0u : cur + S::kTokens, wnxt = wcur == 2 * S::kWeights ? 0u : wcur + S::kWeights;
        const bool turn = ((g + 1) & 3) == 0 || g + 1 == G;
        const uint32_t s0 = scur - (uint32_t)(g & 3) * 4;
        const uint32_t snxt = !turn ? scur + 4 : s0 == S::kScale + 2 * S::kScales ? (uint32_t)S::kScale : s0 + S::kScales;
        half_stage(Half0(), f, nxt, snxt, [](int) {}, std::integral_constant<int, 0>());
        meet();
        float wsn[H];
        read_ws(wsn, g + 1 == G ? wsb_next : wsb, snxt);
        half_stage(Half1(), f, nxt, snxt, [&](int j) { read_w(fn, j, wnxt); }, std::integral_constant<int, 2 * TN>());
        cur = nxt;
        wcur = wnxt;
        scur = snxt;
#pragma unroll
        for (int h = 0; h < H; ++h)
            wsv[h] = wsn[h];
    };
    __builtin_amdgcn_sched_barrier(0);
    meet();
    if (uniform(s_tile[0].nt) < 0)
        return;
    wsb = block_of(uniform(s_tile[0].nt));
#pragma unroll
    for (int j = 0; j < 2 * TN; ++j)
        read_w(w[0], j, 0);
#pragma unroll
    for (int b = 0; b < XR - 1; ++b)
#pragma unroll
        for (int j = 0; j < 3; ++j)
            read_x(j, b, 0, S::kScale);
    read_ws(wsv, wsb, S::kScale);
    for (int ti = 0;; ++ti) {
        const int r0 = uniform(s_tile[ti & 1].r0), rows = uniform(s_tile[ti & 1].rows), nt = uniform(s_tile[ti & 1].nt),
                  more = uniform(s_tile[ti & 1].more);
        const int nw = nt * BC + wn * 16 * TG;          // the wave's first column
        wsb = wsb_next = block_of(nt);
#pragma unroll
        for (int a = 0; a < TN; ++a)
#pragma unroll
            for (int b = 0; b < TM; ++b)
                tot[a][b] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i <= kDelay; ++i)
            c[i] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int b = 0; b < XR; ++b)
#pragma unroll
            for (int h = 0; h < H; ++h)
                sc[b][h] = 0.f;
        // stages in pairs, an odd one first: one way out of the loop, else the compiler holds the totals twice
        int g = 0;
        if (G & 1) {
#pragma unroll
            for (int t = 0; t < TN; ++t)
                w[1][t] = w[0][t];
            stage(w[1], w[0], g++);
        }
        for (; g < G; g += 2) {
            stage(w[0], w[1], g);
            if (g + 2 == G && more)                     // written two stages ago or before
                wsb_next = block_of(uniform(s_tile[(ti + 1) & 1].nt));
            stage(w[1], w[0], g + 1);
        }
#pragma unroll
        for (int i = TN * TM - kDelay; i < TN * TM; ++i)
            add(i);

        // a lane's 4 TG outputs of a token are consecutive, four lanes make a run of 16 TG
        int me = m;
        asm volatile("" : "+v"(me));                    // else the rows' numbers are held in registers through the loop
#pragma unroll
        for (int b = 0; b < TM; ++b) {
            const int t = b * 16 + me, n = nw + q * 4 * TG;
            if (t >= rows || n >= cols)
                continue;
            const size_t at = (size_t)(r0 + t) * cols + n;
            float v[4 * TG];
#pragma unroll
            for (int a = 0; a < TG; ++a)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[4 * a + i] = tot[a][b][i];
                    if constexpr (SW)
                        v[4 * a + i] = silu_fast(v[4 * a + i]) * tot[a + TG][b][i];
                }
            // N is a multiple of 16: where the first of a lane's 4 TG <= 16 outputs exists, all do
#pragma unroll
            for (int a = 0; a < 4 * TG; a += F32 ? 4 : 8) {
                if constexpr (F32)
                    *reinterpret_cast<floatx4 *>(static_cast<float *>(p.c) + at + a) = floatx4{v[a], v[a + 1], v[a + 2], v[a + 3]};
                else if constexpr (4 * TG >= 8)
                    *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(p.c) + at + a) =
                        u32x4{bf16_pair(v[a], v[a + 1]), bf16_pair(v[a + 2], v[a + 3]), bf16_pair(v[a + 4], v[a + 5]),
                              bf16_pair(v[a + 6], v[a + 7])};
                else
                    *reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(p.c) + at + a) =
                        u32x2{bf16_pair(v[a], v[a + 1]), bf16_pair(v[a + 2], v[a + 3])};
            }
        }
        if (!more)
            return;
    }
}

template <int KIND, bool F32, int TN, int TM>
hipError_t launch_tile(const Fp8GemmLaunch &g, const Fp8Args &p, hipStream_t st)
{
    constexpr bool SW = KIND == MOE_GEMM_W13_SWIGLU;
    constexpr int BM = 16 * TM, BC = 64 * (SW ? TN / 2 : TN), kBytes = TileLds<TN, TM>::kBytes;
    const int cols = SW ? g.N / 2 : g.N;
    const int tn = (cols + BC - 1) / BC;
    // as many workgroups as run at one time (a multiple of the XCDs), each with its share of the tiles
    constexpr long long kAtOnce = 256 * (kBytes * 2 <= 160 * 1024 ? 2 : 1);
    const long long all = chunks_at_most(g, BM) * tn;
    const long long grid = g.K >= kTilesAhead * 128 && all > kAtOnce ? kAtOnce : all;
    allow_lds<decltype(fp8_tile_kernel<KIND, F32, TN, TM>), fp8_tile_kernel<KIND, F32, TN, TM>, kBytes>();
    hipLaunchKernelGGL((fp8_tile_kernel<KIND, F32, TN, TM>), dim3((unsigned)grid), dim3(512), kBytes, st, p, tn);
    return hipGetLastError();
}

// Which kernel, from the expected rows R' of an expert that has any and the workgroups (items) that each would have; us
// on MI355X in graphs of calls, operands rotating through more than the 256 MB memory-side cache:
//   The ring kernel where one of its forms has at most a workgroup for each CU: of those the one that copies least
//     beside a CU's share of the weights, the larger tile where two do alike. M x N x K: 1 x 4096 x 4096 5.5 with 16 x
//     16 outputs to a workgroup, 6.6 with 16 x 32; 64 x 4096 x 4096 8.6 with 32 x 32, 11.0 with 32 x 64; 256 x 4096 x
//     4096 14.7 with 64 x 64, 18.1 with 32 x 64; 350 x 4096 x 4096 17.6 with 48 x 128, 20.2 with 64 x 128; 450 x 2560 x 4096
//     15.7 with 80 x 64, 17.1 with 48 x 128; 512 x 4096 x 4096 21.0 with 64 x 128, 26.1 with 64 x 64 and 24.5 in the
//     tile kernel; 333 x 2112 x 7168 18.0 with 48 x 64, 19.3 with 64 x 64 and 41 in the tile kernel. 80 rows of binary32
//     results spill. From 17 rows on, half of K to a wave instead of a quarter where K is short: 64 x 4096 x 512, 1024, 1280
//     and 1920 4.0, 4.4, 5.2 and 6.1 against 4.7, 4.8, 5.0 and 5.7, 256 x 4096 x the same 6.2, 6.6, 8.6 and 9.9 against 7.7,
//     8.0, 8.4 and 9.4, 333 x 2112 x 512, 1024 and 1280 6.0, 6.5 and 8.4 against 6.5, 6.8 and 7.2. (Up to 16 rows
//     a quarter is better at any K: 1 x 4096 x 512, 1024 and 1920 3.7, 3.8 and 4.1 against 3.9, 4.5 and 6.3.)
//     With up to 16 rows of a dense product at any number of columns.
//   experts with R' <= 10: the ring kernel with 16 x 32 weight rows to a wave, all of K, whose sums are binary32's too (TB/s of
//     all that is read and written, here and in tiles of 128 x 64): 2048 -> 2 x 768 with 1, 4, 8 and 16 rows for each of 128
//     experts 5.8 and 5.4, 6.0 and 5.8, 6.1 and 5.8, 4.5 and 5.6; 2048 -> 2048 with 4 rows 6.3 and 6.0, 1024 -> 2048 5.9 and
//     5.7. Shorter K, us: 128, 256, 512 and 1024 -> 2 x 768 with 8 rows 16.1 and 15.0, 17.5 and 19.4, 22.2 and 22.3, 36.4 and
//     38.1, with 10 rows 17.3 and 15.2, 19.0 and 19.6, 23.1 and 21.6, 38.6 and 37.7; 768 -> 2048 with 1, 4 and 8 rows 28.2
//     and 27.4, 38.8 and 36.4, 41.2 and 37.1; 512 -> 2048 with 4 and 8 26.9 and 26.9, 28.4 and 26.9; 256 -> 2048 with 4 22.1
//     and 24.0, 256 -> 7168 of 256 experts with 1 46.7 and 54.3
//   R' <= 28: tiles of 128 x 64 (weight rows x tokens): 25 and 32 rows for each of 128 experts, 2048 -> 2 x 768, 72.7 and
//     75.4; 74.5 and 73.6 with 256 x 64; 80.1 and 78.1 with 256 x 128
//   above: 256 x 128, but 256 x 64 where that takes no more rounds of the CUs: 1024 x 4096 x 4096 27.4, with 256 x 128 32;
//     1536 x 4096 x 4096 43.3 and, with 256 x 128, 34.1; 50 rows for each of 128 experts 87.1 and 81.7, where the few
//     experts with more than 64 make a round of their own: the rounds are those of R' and two standard deviations.
//     binary32 results, whose widened codes need the registers, always 256 x 64: 4096 x 4096 x 4096 141, with 128 x 64 147.
template <int KIND, bool F32>
hipError_t launch_kind(const Fp8GemmLaunch &g, const Fp8Args &p, hipStream_t st)
{
    constexpr bool SW = KIND == MOE_GEMM_W13_SWIGLU;
    constexpr double kCus = 256.0;
    const Load load(g);
    const double per = load.per;
    auto rounds = [&](int BN, int BM) { return ceil(load.items(BN, BM) / kCus); };
    // the ring kernel's forms, larger tiles first: rows, weight rows, waves along the weights
    struct Ring {
        int rows, weights, wn;
    };
    constexpr Ring kRing[] = {{64, 128, 2}, {48, 128, 2}, {80, 64, 1}, {64, 64, 1}, {48, 64, 1}, {32, 128, 2},
                              {32, 64, 1}, {32, 32, 1}, {16, 128, 2}, {16, 64, 2}, {16, 32, 1}, {16, 16, 1}};
    const bool short_k = g.K <= 1024;
    int best = -1;
    double least = 0.0;
    for (int i = 0; i < (SW ? 11 : 12); ++i) {
        const Ring &r = kRing[i];
        if ((r.rows > 16 && (per <= r.rows / 2 || (short_k && r.wn == 1))) || (F32 && r.rows > 64))
            continue;
        const double n = rounds(r.weights, r.rows), cost = n * (r.weights + r.rows * r.wn);
        if ((n <= 1.0 || (!g.offsets && per <= 16.0)) && (best < 0 || cost < least)) {
            best = i;
            least = cost;
        }
    }
    switch (best) {
    case 0: return launch_ring<KIND, F32, 4, 4, 2, 2>(g, p, st);
    case 1: return launch_ring<KIND, F32, 3, 4, 2, 2>(g, p, st);
    case 2:
        if constexpr (!F32)
            return launch_ring<KIND, F32, 5, 4, 4, 2>(g, p, st);
        break;
    case 3: return launch_ring<KIND, F32, 4, 4, 4, 2>(g, p, st);
    case 4: return launch_ring<KIND, F32, 3, 4, 4, 2>(g, p, st);
    case 5: return launch_ring<KIND, F32, 2, 4, 2, 2>(g, p, st);
    case 6: return launch_ring<KIND, F32, 2, 4, 4, 2>(g, p, st);
    case 7: return launch_ring<KIND, F32, 2, 2, 4, 2>(g, p, st);
    case 8: return launch_ring_16<KIND, F32, 4, 2, 2>(g, p, st);
    case 9: return launch_ring_16<KIND, F32, 2, 2, 2>(g, p, st);
    case 10: return launch_ring_16<KIND, F32, 2, 4, 2>(g, p, st);
    case 11:
        if constexpr (!SW)
            return launch_ring_16<KIND, F32, 1, 4, 4>(g, p, st);
    }
    if (g.offsets && per <= 10.0)
        return launch_ring<KIND, F32, 1, 2, 1, 2, true>(g, p, st);
    if (per <= 28.0)
        return launch_tile<KIND, F32, 2, 4>(g, p, st);
    const double rows = g.offsets ? per + 2.0 * sqrt(per) : per, columns = load.items(256, 1) / ceil(per);
    auto tall = [&](int BM) { return ceil(columns * ceil(rows / BM) / kCus); };
    if constexpr (!F32)
        if (tall(128) < tall(64))
            return launch_tile<KIND, F32, 4, 8>(g, p, st);
    return launch_tile<KIND, F32, 4, 4>(g, p, st);
}

}  // namespace

hipError_t launch_fp8_gemm(const Fp8GemmLaunch &g, hipStream_t st)
{
    const Fp8Args p{g.a, (uint32_t)((size_t)(g.a_row_index ? g.max_rows / g.top_k : g.max_rows) * g.K), g.as, g.a_row_index,
                    g.top_k, g.offsets, g.max_rows, g.num_experts, g.wq, g.ws, g.c, g.K, g.N};
    if (g.kind == MOE_GEMM_W13_SWIGLU)
        return launch_kind<MOE_GEMM_W13_SWIGLU, false>(g, p, st);
    if (g.c_f32)
        return launch_kind<MOE_GEMM_W2, true>(g, p, st);
    return launch_kind<MOE_GEMM_W2, false>(g, p, st);
}

}  // namespace moe
