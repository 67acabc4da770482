// gemm_w8a8.hip -- products of int8 rows: dense, and grouped over the experts'
// segments with the SwiGLU epilogue.
//
//   acc[r][n] = sum_k a[r][k] w[n][k]          exact, binary integer
//   c[r][n]   = float(acc) * as[r] * ws[n]     (binary32)
//
// MFMA: v_mfma_i32_16x16x64_i8, the weight rows as operand A and the tokens as
// operand B, so that a result lane holds four consecutive outputs of one token.
// Both operands take the same permutation of K, which leaves the sums as they are.
#include <mutex>

#include "gemm_core.hpp"
#include "w8a8.hpp"

namespace moe {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ i32x4 mfma_i8(u32x4 w, u32x4 x, i32x4 c)
{
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, w), __builtin_bit_cast(i32x4, x), c, 0, 0, 0);
}

// fp32 pair -> bf16 pair, round to nearest even
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi)
{
    typedef float f2 __attribute__((ext_vector_type(2)));
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2{lo, hi}), b2));
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

// ---------------------------------------------------------------------------
// Many rows per expert: a workgroup of four waves computes BN weight rows x BM
// tokens, a wave 32 TN x 32 TM of them with v_mfma_i32_32x32x32_i8. Both
// operands pass through LDS, kStageK bytes of K to a stage, five stages deep.
//
// A stage holds BN + BM rows of 64 bytes, four 16-byte chunks each; row r keeps
// chunk c at place c ^ ((r >> 2) & 3), so that the 64 lanes of a fragment read
// (32 rows x 2 chunks) meet no bank conflict. The copies go from memory straight
// to LDS (buffer_load ... lds, 16 bytes a lane, lane l to place l of 16 rows);
// each lane asks for the chunk that belongs to its place, so four lanes still
// read 64 contiguous bytes.
//
// A weight row's place decides which output a result register is: tile t's row
// r holds output ((r >> 2) & 1) 16 TG + 16 t + 4 (r >> 3) + (r & 3) of the
// wave's columns, which makes a lane's sixteen results of a tile consecutive.
// ---------------------------------------------------------------------------
constexpr int kStageK = 64;
constexpr int kStages = 5;

typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) unsigned char lds_byte;

constexpr uint32_t vmcnt_imm(int n)                   // s_waitcnt vmcnt(n), other counters untouched
{
    return (uint32_t)((n & 15) | ((n >> 4) << 14) | (7 << 4) | (15 << 8));
}

// 16 bytes per lane from memory to LDS: lane l's to dst + 16 l
__device__ __forceinline__ void copy16(__amdgpu_buffer_rsrc_t r, lds_byte *dst, uint32_t voff, uint32_t soff)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, dst, 16, voff, soff, 0, 0);
}

template <int N>
__device__ __forceinline__ void wait_barrier()
{
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(N));
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_s_barrier();
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_sched_barrier(0);
}

// Tile (row tile, column tile) of linear index i: column tiles in groups of
// eight row tiles, so that the workgroups running at one time share both operands.
__device__ __forceinline__ void tile_of(int i, int tm, int tn, int &m, int &n)
{
    constexpr int G = 8;
    const int g = i / (G * tn), rest = i - g * G * tn;
    const int gm = tm - g * G < G ? tm - g * G : G;
    m = g * G + rest % gm;
    n = rest / gm;
}

// How many of n things spread evenly over m places come before place i.
constexpr int spread_to(int i, int n, int m) { return i * n / m; }

// The order of a half step's instructions: its LDS reads and its copies to LDS
// spread evenly behind the MFMAs, so that none of them holds the matrix unit's
// next instruction back. (The half step issues them in this order already.)
template <int MFMAS, int READS, int COPIES>
__device__ __forceinline__ void spread()
{
#pragma unroll
    for (int i = 0; i < MFMAS; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
#pragma unroll
        for (int j = spread_to(i, READS, MFMAS); j < spread_to(i + 1, READS, MFMAS); ++j)
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
#pragma unroll
        for (int j = spread_to(i, COPIES, MFMAS); j < spread_to(i + 1, COPIES, MFMAS); ++j)
            __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
    }
}

template <int TN, int TM>
struct Frags {
    u32x4 w[TN], x[TM];
};

template <int KIND, bool F32, int TN, int TM, int NWN, int NWM>
__global__ __launch_bounds__(256, 1) void w8_tile_kernel(W8Args p, int tm, int tn)
{
    constexpr bool SW = KIND == MOE_GEMM_W13_SWIGLU;
    constexpr int TG = SW ? TN / 2 : TN;
    constexpr int BN = 32 * TN * NWN, BM = 32 * TM * NWM;
    constexpr int BC = SW ? BN / 2 : BN;                // output columns of the workgroup
    constexpr int LN = BN / 64, LM = BM / 64;           // copies of a wave per stage
    constexpr int L = LN + LM;
    constexpr int kStageBytes = (BN + BM) * kStageK;
    extern __shared__ __align__(16) unsigned char s_dyn[];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int wn = wave / NWM, wm = wave % NWM;
    // XCD x (workgroups x, x + 8, ...) takes the x-th share of the tiles
    const int total = gridDim.x, per = total / kXcds, extra = total % kXcds;
    const int x = blockIdx.x % kXcds;
    const int item = x * per + (x < extra ? x : extra) + blockIdx.x / kXcds;
    int mt, nt;
    tile_of(item, tm, tn, mt, nt);
    int e, r0, rows;
    if (!find_chunk(p, BM, mt, lane, e, r0, rows))
        return;
    e = uniform(e);
    const int cols = SW ? p.N / 2 : p.N;
    const int n0 = nt * BC;
    const uint32_t K = (uint32_t)p.K;

    // this lane's place in a copy of 16 rows, and the chunk that belongs there
    const int prow = lane >> 2;
    auto chunk_at = [&](int row) { return (uint32_t)(((lane & 3) ^ ((row >> 2) & 3)) * 16); };
    uint32_t wo[LN], xo[LM];
#pragma unroll
    for (int j = 0; j < LN; ++j) {
        const int row = (wave * LN + j) * 16 + prow;    // row of the stage: wave's columns, tile, row of the tile
        const int w = row / (32 * TN), t = row / 32 % TN, r = row % 32;
        int n = n0 + w * 32 * TG + ((r >> 2) & 1) * 16 * TG + (t % TG) * 16 + (r >> 3) * 4 + (r & 3);
        n = n < cols ? n : cols - 1;
        wo[j] = (uint32_t)(n + (SW && t >= TG ? cols : 0)) * K + chunk_at(row);
    }
#pragma unroll
    for (int j = 0; j < LM; ++j) {
        const int row = (wave * LM + j) * 16 + prow;
        xo[j] = (uint32_t)act_row(p, r0 + (row < rows ? row : rows - 1)) * K + chunk_at(row);
    }
    const __amdgpu_buffer_rsrc_t rw = make_rsrc(p.wq + (size_t)e * p.N * K, (uint32_t)p.N * K);
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(p.a, 0xFFFFFFFFu);
    lds_byte *lds = (lds_byte *)s_dyn;
    // one of a wave's L copies of a stage: K bytes [k, k + 64) to the stage at byte `at` of LDS
    auto copy_one = [&](int j, uint32_t at, uint32_t k) {
        lds_byte *dst = lds + at;
        if (j < LN)
            copy16(rw, dst + (wave * LN + j) * 1024, wo[j < LN ? j : 0], k);
        else
            copy16(rx, dst + BN * kStageK + (wave * LM + j - LN) * 1024, xo[j < LN ? 0 : j - LN], k);
    };
    auto copy = [&](int s) {
#pragma unroll
        for (int j = 0; j < L; ++j)
            copy_one(j, (uint32_t)(s % kStages) * kStageBytes, (uint32_t)s * kStageK);
    };
    // fragment reads: lane l holds chunk 2 kk + l / 32 of row l % 32
    const int fr = lane & 31;
    const uint32_t f0 = (uint32_t)(fr * 64 + (((lane >> 5) ^ ((fr >> 2) & 3)) * 16));
    const uint32_t f1 = f0 ^ 32u;
    using Fr = Frags<TN, TM>;
    // one of a half step's TN + TM fragments (tokens and the first weights first: what the MFMAs need first)
    auto read_one = [&](int j, const unsigned char *src, Fr &d) {
        if (j < TM)
            d.x[j < TM ? j : 0] = *reinterpret_cast<const u32x4 *>(src + BN * kStageK + (wm * TM + j) * 2048);
        else
            d.w[j < TM ? 0 : j - TM] = *reinterpret_cast<const u32x4 *>(src + (wn * TN + j - TM) * 2048);
    };
    i32x16 acc[TN][TM];
#pragma unroll
    for (int a = 0; a < TN; ++a)
#pragma unroll
        for (int b = 0; b < TM; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                acc[a][b][i] = 0;
    // Half a step: multiplies d while the fragments at byte `from` of LDS go to
    // dn and copies [C0, C1) of the stage at byte `to` go out.
    auto half_step = [&](const Fr &d, Fr &dn, uint32_t from, auto c0, auto c1, uint32_t to, uint32_t k) {
        constexpr int M = TN * TM, R = TN + TM, C0 = decltype(c0)::value, C = decltype(c1)::value - C0;
        const unsigned char *src = s_dyn + from;
#pragma unroll
        for (int i = 0; i < M; ++i) {
#pragma unroll
            for (int j = spread_to(i, R, M); j < spread_to(i + 1, R, M); ++j)
                read_one(j, src, dn);
#pragma unroll
            for (int j = spread_to(i, C, M); j < spread_to(i + 1, C, M); ++j)
                copy_one(C0 + j, to, k);
        }
#pragma unroll
        for (int a = 0; a < TN; ++a)
#pragma unroll
            for (int b = 0; b < TM; ++b)
                acc[a][b] = __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4, d.w[a]),
                                                                  __builtin_bit_cast(i32x4, d.x[b]), acc[a][b], 0, 0, 0);
        spread<M, R, C>();
    };
    using C0 = std::integral_constant<int, 0>;
    using CH = std::integral_constant<int, L / 2>;
    using CL = std::integral_constant<int, L>;
    // Step s multiplies stage s. In its middle the wave waits for its copies of
    // stage s + 1 (those of s + 2 and s + 3 stay in flight) and meets the other
    // waves: then stage s + 1 is whole, and every wave has read all of stage
    // s - 1, whose place takes stage s + 4: half of its copies go out in the
    // second half of step s, half in the first half of step s + 1. Reads of
    // stage s may still be on their way at the meeting; its place is not
    // written before the next one. A step's second half has its fragments in
    // registers (or about to be) when the first half of the next step's are read.
    // Steps past the last multiply nothing: a stage past K is not copied, and
    // its place is read (in bounds) but not used.
    const int steps = p.K / kStageK;                    // even
    Fr d0, d1;
#pragma unroll
    for (int s = 0; s < 4; ++s)
        if (s < steps)
            copy(s);
    if (steps > 2)
        wait_barrier<3 * L>();
    else
        wait_barrier<L>();
#pragma unroll
    for (int j = 0; j < TN + TM; ++j)
        read_one(j, s_dyn + f0, d0);
    uint32_t cur = 0, to = 3 * kStageBytes, k = 3 * kStageK;    // stage s; the place and K of the stage being copied
    auto after = [&](uint32_t at) { return at == (kStages - 1) * kStageBytes ? 0u : at + kStageBytes; };
    int s = 0;
    if (steps > 4) {
        half_step(d0, d1, cur + f1, C0(), C0(), 0, 0);  // stage 3 is already on its way
        for (;; ++s) {
            wait_barrier<2 * L>();
            to = after(to);
            k += kStageK;
            const uint32_t next = after(cur);
            half_step(d1, d0, next + f0, C0(), CH(), to, k);
            cur = next;
            if (s + 5 >= steps)
                break;
            half_step(d0, d1, cur + f1, CH(), CL(), to, k);
        }
        // step s + 1 = steps - 4: the rest of the last stage's copies
        half_step(d0, d1, cur + f1, CH(), CL(), to, k);
        ++s;
    } else {
        half_step(d0, d1, cur + f1, C0(), C0(), 0, 0);
    }
    for (;;) {                                          // nothing left to copy; the first half of step s is done
        if (s + 1 < steps)
            wait_barrier<0>();
        const uint32_t next = after(cur);
        half_step(d1, d0, next + f0, C0(), C0(), 0, 0);
        cur = next;
        if (++s >= steps)
            break;
        half_step(d0, d1, cur + f1, C0(), C0(), 0, 0);
    }

    // Epilogue: 32 tokens at a time through the wave's own part of LDS (past
    // the barrier all reads of the stages are done), so that a store writes whole runs of a row
    // (16 TG or 32 TG lanes' worth) instead of 8 bytes per token.
    __syncthreads();
    constexpr int kElem = F32 ? 4 : 2;
    constexpr int kRow = 32 * TG * kElem;               // bytes of a row in the wave's columns
    constexpr int kPitch = kRow + 16;
    constexpr int kLanes = kRow / 16;                   // lanes that store a row
    static_assert(32 * kPitch * 4 <= kStageBytes * kStages, "the epilogue's rows fit the stages");
    unsigned char *buf = s_dyn + wave * (32 * kPitch);
    const int half = lane >> 5, m32 = lane & 31;
    const int nw = n0 + wn * 32 * TG;                   // the wave's first column
    const float *wsp = p.ws + (size_t)e * p.N;
    float wsv[TN][16];
#pragma unroll
    for (int t = 0; t < TN; ++t)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            int n = nw + half * 16 * TG + (t % TG) * 16 + g * 4;
            n = (n < cols ? n : cols - 4) + (SW && t >= TG ? cols : 0);
            const floatx4 v = *reinterpret_cast<const floatx4 *>(wsp + n);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                wsv[t][4 * g + i] = v[i];
        }
#pragma unroll
    for (int b = 0; b < TM; ++b) {
        const int mb = (wm * TM + b) * 32;
        if (mb >= rows)
            break;
        const int m = mb + m32;
        const float as = p.as[act_row(p, r0 + (m < rows ? m : rows - 1))];
#pragma unroll
        for (int t = 0; t < TG; ++t) {
            float v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                v[i] = (float)acc[t][b][i] * as * wsv[t][i];
                if constexpr (SW)
                    v[i] = silu_fast(v[i]) * ((float)acc[t + TG][b][i] * as * wsv[t + TG][i]);
            }
            u32x4 *dst = reinterpret_cast<u32x4 *>(buf + m32 * kPitch + (half * 16 * TG + t * 16) * kElem);
            if constexpr (F32) {
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    dst[g] = __builtin_bit_cast(u32x4, floatx4{v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]});
            } else {
#pragma unroll
                for (int g = 0; g < 2; ++g)
                    dst[g] = u32x4{bf16_pair(v[8 * g], v[8 * g + 1]), bf16_pair(v[8 * g + 2], v[8 * g + 3]),
                                   bf16_pair(v[8 * g + 4], v[8 * g + 5]), bf16_pair(v[8 * g + 6], v[8 * g + 7])};
            }
        }
        // the wave's own writes, in order before its reads
        __builtin_amdgcn_wave_barrier();
        const int at = lane % kLanes, n = nw + at * (16 / kElem);
#pragma unroll
        for (int j = 0; j < 32 * kLanes / 64; ++j) {
            const int row = j * (64 / kLanes) + lane / kLanes;
            const u32x4 v = *reinterpret_cast<const u32x4 *>(buf + row * kPitch + at * 16);
            if (mb + row < rows && n < cols)
                *reinterpret_cast<u32x4 *>(static_cast<unsigned char *>(p.c) +
                                           ((size_t)(r0 + mb + row) * cols + n) * kElem) = v;
        }
        __builtin_amdgcn_wave_barrier();
    }
}

template <int KIND, bool F32, int TN, int TM, int NWN, int NWM>
void allow_lds(int bytes)
{
    (void)hipFuncSetAttribute(reinterpret_cast<const void *>(&w8_tile_kernel<KIND, F32, TN, TM, NWN, NWM>),
                              hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <int KIND, bool F32, int TN, int TM, int NWN, int NWM>
hipError_t launch_tile(const W8GemmLaunch &g, const W8Args &p, hipStream_t st)
{
    constexpr bool SW = KIND == MOE_GEMM_W13_SWIGLU;
    constexpr int BN = 32 * TN * NWN, BM = 32 * TM * NWM, BC = SW ? BN / 2 : BN;
    constexpr int lds = (BN + BM) * kStageK * kStages;
    const int cols = SW ? g.N / 2 : g.N;
    const int tn = (cols + BC - 1) / BC;
    const int tm = g.offsets ? g.max_rows / BM + (g.num_experts < g.max_rows ? g.num_experts : g.max_rows)
                             : (g.max_rows + BM - 1) / BM;
    static std::once_flag once;
    std::call_once(once, allow_lds<KIND, F32, TN, TM, NWN, NWM>, lds);
    hipLaunchKernelGGL((w8_tile_kernel<KIND, F32, TN, TM, NWN, NWM>), dim3((unsigned)(tm * tn)), dim3(256), lds, st, p,
                       tm, tn);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_w8_gemm(const W8GemmLaunch &g, hipStream_t st)
{
    const W8Args p{g.a, g.as, g.a_row_index, g.top_k, g.offsets, g.max_rows, g.num_experts, g.wq, g.ws, g.c, g.K, g.N};
    const int per_expert = g.expected_rows / (g.num_experts > 0 ? g.num_experts : 1);
    if (per_expert > 64) {
        if (g.kind == MOE_GEMM_W13_SWIGLU)
            return launch_tile<MOE_GEMM_W13_SWIGLU, false, 4, 4, 2, 2>(g, p, st);
        if (g.c_f32)
            return launch_tile<MOE_GEMM_W2, true, 4, 4, 2, 2>(g, p, st);
        return launch_tile<MOE_GEMM_W2, false, 4, 4, 2, 2>(g, p, st);
    }
    if (g.kind == MOE_GEMM_W13_SWIGLU)
        return launch_stream<MOE_GEMM_W13_SWIGLU, false>(g, p, st);
    if (g.c_f32)
        return launch_stream<MOE_GEMM_W2, true>(g, p, st);
    return launch_stream<MOE_GEMM_W2, false>(g, p, st);
}

}  // namespace moe
