// gemm_w8a8.hip -- products of int8 rows: dense, and grouped over the experts'
// segments with the SwiGLU epilogue.
//
//   acc[r][n] = sum_k a[r][k] w[n][k]          exact, binary integer
//   c[r][n]   = float(acc) * as[r] * ws[n]     (binary32)
//
// MFMA: v_mfma_i32_16x16x64_i8 (streaming kernel) and 32x32x32 (tile kernel), the
// weight rows as operand A and the tokens as operand B, so that a result lane
// holds four (four times four) consecutive outputs of one token. Both operands
// take the same permutation of K, which leaves the sums as they are.
#include <cmath>
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

struct W8Args {
    const int8_t *a;
    uint32_t a_bytes;
    const float *as;
    const uint16_t *a_bf16;      // instead of a and as (streaming kernel)
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

// Activation row of result row r, in two steps: the index entry (0 where there
// is no index; loaded first, ahead of what can go out without it), then the row,
// kept inside the array whatever the entry holds.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t index_rsrc(const W8Args &p)
{
    return make_rsrc(p.a_row_index, p.a_row_index ? (uint32_t)p.max_rows * 4u : 0u);
}

__device__ __forceinline__ int load_index(__amdgpu_buffer_rsrc_t ri, int r)
{
    return (int)__builtin_amdgcn_raw_buffer_load_b32(ri, (uint32_t)r * 4u, 0, 0);
}

__device__ __forceinline__ int act_row(const W8Args &p, int r, int i)
{
    i = i < 0 ? 0 : (i < p.max_rows ? i : p.max_rows - 1);
    return p.a_row_index ? i / p.top_k : r;
}

// The chunks (at most CS rows of one expert each) as one wave sees them, four
// experts to a lane: expert 64 i + lane has n[i] chunks, the first of them
// chunk first[i]. All offsets are loaded before the first is used; past 256
// experts the rest is scanned in rounds of 256. Offsets are the caller's. An
// expert has at least 0 and at most as many chunks as all rows would give it,
// so that the numbers stay in 32 bits and in order whatever the offsets hold, and
// a chunk counts only where its rows are in the arrays (pick_chunk). CLAMP: each
// offset is moved into the rows first, so that the total counts no other chunks
// (the tile kernel shares the total out; in the streaming kernel, whose
// workgroups each look for one chunk, 64 tokens' gate/up took 69.0 us with it
// and takes 68.2).
constexpr int kScan = 4;

struct Chunks {
    int o0[kScan], o1[kScan], first[kScan], n[kScan];
};

// Experts e0 .. e0 + 255, whose first chunk is `before`; returns the next one's.
template <bool CLAMP>
__device__ __forceinline__ int scan_chunks(const W8Args &p, uint32_t CS, int lane, int e0, int before, Chunks &c)
{
#pragma unroll
    for (int i = 0; i < kScan; ++i) {
        const int e = e0 + 64 * i + lane, ee = e < p.E ? e : p.E - 1;
        c.o0[i] = p.offsets[ee];
        c.o1[i] = p.offsets[ee + 1];
    }
#pragma unroll
    for (int i = 0; i < kScan; ++i) {
        if constexpr (CLAMP) {
            c.o0[i] = min(max(c.o0[i], 0), p.max_rows);
            c.o1[i] = min(max(c.o1[i], 0), p.max_rows);
        }
        const uint32_t rows = __builtin_elementwise_sub_sat((uint32_t)c.o1[i], (uint32_t)c.o0[i]);
        c.n[i] = e0 + 64 * i + lane < p.E ? (int)min((rows + CS - 1) / CS, (uint32_t)p.max_rows / CS + 1) : 0;
        int total;
        c.first[i] = before + wave_exclusive_scan(c.n[i], total);
        before += total;
    }
    return before;
}

// Chunk `chunk`, where it is one of c's: its expert, first row and rows.
__device__ __forceinline__ bool pick_chunk(const W8Args &p, int CS, int e0, int chunk, const Chunks &c, int &e, int &r0,
                                           int &rows)
{
    bool found = false;
#pragma unroll
    for (int i = 0; i < kScan; ++i) {
        const uint64_t at = __ballot(c.first[i] <= chunk && chunk < c.first[i] + c.n[i]);
        if (at) {
            const int l = __builtin_ctzll(at);
            e = e0 + 64 * i + l;
            r0 = (int)((uint32_t)__builtin_amdgcn_readlane(c.o0[i], l) +
                       (uint32_t)(chunk - __builtin_amdgcn_readlane(c.first[i], l)) * (uint32_t)CS);
            const int end = min(__builtin_amdgcn_readlane(c.o1[i], l), p.max_rows);
            found = r0 >= 0 && r0 < end;               // compared: a difference could pass 32 bits
            rows = end - r0;
        }
    }
    rows = rows < CS ? rows : CS;
    return found;
}

__device__ __forceinline__ bool dense_chunk(const W8Args &p, int CS, int chunk, int &e, int &r0, int &rows)
{
    e = 0;
    r0 = chunk * CS;
    rows = p.max_rows - r0;
    rows = rows < CS ? rows : CS;
    return rows > 0;
}

// Chunk `chunk`: its expert, first row and rows; false past the last chunk. One
// wave, every lane gets the result.
template <bool CLAMP>
__device__ __forceinline__ bool find_chunk(const W8Args &p, int CS, int chunk, int lane, int &e, int &r0, int &rows)
{
    if (!p.offsets)
        return dense_chunk(p, CS, chunk, e, r0, rows);
    e = r0 = rows = 0;
    for (int e0 = 0, before = 0; e0 < p.E; e0 += 64 * kScan) {
        Chunks c;
        before = scan_chunks<CLAMP>(p, CS, lane, e0, before, c);
        if (chunk < before)
            return pick_chunk(p, CS, e0, chunk, c, e, r0, rows);
    }
    return false;
}

// Tile (chunk of rows, column tile) of linear index i: the column tiles of
// groups of eight chunks, so that the workgroups running at one time share both
// operands.
__device__ __forceinline__ void tile_of(int i, int tm, int tn, int &m, int &n)
{
    constexpr int G = 8;
    const int g = i / (G * tn), rest = i - g * G * tn;
    const int gm = tm - g * G < G ? tm - g * G : G;
    m = g * G + rest % gm;
    n = rest / gm;
}

// Workgroup b's tile of the tiles that there are (the grid holds as many as
// there can be): XCD x (workgroups x, x + 8, ...) takes the x-th share of them,
// so that those which share operands also share an L2. False where b has none.
__device__ __forceinline__ bool find_tile(const W8Args &p, int CS, int tn, int b, int lane, int &e, int &r0, int &rows,
                                          int &nt)
{
    Chunks c;
    int tm = 0;
    if (!p.offsets)
        tm = (p.max_rows + CS - 1) / CS;
    else
        for (int e0 = 0; e0 < p.E; e0 += 64 * kScan)
            tm = scan_chunks<true>(p, CS, lane, e0, tm, c);
    const int total = tm * tn, per = total / kXcds, extra = total % kXcds;
    const int x = b % kXcds, ix = b / kXcds;
    if (ix >= per + (x < extra ? 1 : 0))
        return false;
    int mt;
    tile_of(x * per + (x < extra ? x : extra) + ix, tm, tn, mt, nt);
    if (!p.offsets)
        return dense_chunk(p, CS, mt, e, r0, rows);
    e = r0 = rows = 0;
    if (p.E <= 64 * kScan)
        return pick_chunk(p, CS, 0, mt, c, e, r0, rows);
    return find_chunk<true>(p, CS, mt, lane, e, r0, rows);
}

// ---------------------------------------------------------------------------
// Few rows per expert: the weights are what such a call has to read, once. Each
// wave streams its own weight rows from memory to registers, RING groups of 128
// bytes of K ahead, and multiplies them with NSUB subtiles of 16 tokens, whose
// rows it fetches the same way (they stay in the caches). WK waves of a
// workgroup share a set of rows, each with its part of K, and add their sums
// (integers, so in any order) through LDS; else no LDS and no barrier. Default
// cache policy: a load takes 64 bytes of each row, half a line, and non-temporal
// ones lose the other half before the next load asks for it (1 x 4096 x 4096
// 6.1 us against 5.3, one token through 128 experts' gate/up 9.0 against 8.1).
// Bound by the weight stream: 128 experts of 2048 -> 2 x 768, 64 tokens, 69 us,
// 5.8 TB/s. Groups left over after whole rounds are fetched together as well.
//
// QV > 0: the rows are bf16 and each workgroup quantizes its chunk's itself (K
// at most 512 QV), a wave every fourth row, into LDS, while the first weights
// are under way; codes and scales are those of the quantizer.
// ---------------------------------------------------------------------------
template <int KIND, bool F32, int NSUB, int TPW, int WK, int RING, int QV>
__global__ __launch_bounds__(256, 2) void w8_stream_kernel(W8Args p, int blocks)
{
    constexpr bool SW = KIND == MOE_GEMM_W13_SWIGLU, QA = QV > 0;
    static_assert(!QA || (NSUB == 1 && !SW && WK > 1), "rows in LDS");
    constexpr int kRowPitch = QV * 512 + 16;            // neighbouring rows 4 banks apart
    __shared__ __align__(16) unsigned char s_rows[QA ? 16 * kRowPitch : 16];
    __shared__ float s_scale[16];
    constexpr int TG = SW ? TPW / 2 : TPW;              // tiles side by side: a lane's outputs are 4 TG consecutive ones
    constexpr int WN = 4 / WK;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int m = lane & 15, q = lane >> 4;
    const int wn = wave / WK, wk = wave % WK;
    const int chunk = blockIdx.x / blocks;
    const int block = blockIdx.x - chunk * blocks;
    int e, r0, rows;
    if (!find_chunk<false>(p, 16 * NSUB, chunk, lane, e, r0, rows))
        return;
    e = uniform(e);
    const int cols = SW ? p.N / 2 : p.N;                // outputs per row
    const int n0 = (block * WN + wn) * 16 * TG;
    if (WK == 1 && n0 >= cols)
        return;
    // weight row of lane row m in tile t: outputs n0 + (m / 4) 4 TG + 4 t + m % 4 (gate), the same + N / 2 (up)
    uint32_t wo[TPW], xo[NSUB];
#pragma unroll
    for (int t = 0; t < TPW; ++t) {
        int n = n0 + (m >> 2) * 4 * TG + (t % TG) * 4 + (m & 3);
        n = n < cols ? n : cols - 1;
        if (SW && t >= TG)
            n += cols;
        wo[t] = (uint32_t)n * p.K + q * 16;
    }
    const __amdgpu_buffer_rsrc_t rw = make_rsrc(p.wq + (size_t)e * p.N * p.K, (uint32_t)p.N * p.K);
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(p.a, p.a_bytes), ri = index_rsrc(p);
    // what the rows and the epilogue need sets out first
    const int nq = n0 + q * 4 * TG;
    int row[NSUB], idx[NSUB];
#pragma unroll
    for (int s = 0; s < NSUB; ++s) {
        row[s] = r0 + (16 * s + m < rows ? 16 * s + m : rows - 1);
        idx[s] = QA ? 0 : load_index(ri, row[s]);
    }
    u32x4 hv[4][QA ? QV : 1];                           // rows wave, wave + 4, ... of the chunk
    if constexpr (QA)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = wave + 4 * i;                 // a descriptor of no bytes where there is no such row
            const __amdgpu_buffer_rsrc_t rh = make_rsrc(p.a_bf16 + (size_t)(r0 + r) * p.K, r < rows ? (uint32_t)p.K * 2 : 0u);
#pragma unroll
            for (int v = 0; v < QV; ++v)
                hv[i][v] = bload16(rh, (uint32_t)(lane + 64 * v) * 16, 0);
        }
    floatx4 ws[TPW];
#pragma unroll
    for (int t = 0; t < TPW; ++t) {
        const int n = nq + 4 * (t % TG);
        ws[t] = *reinterpret_cast<const floatx4 *>(p.ws + (size_t)e * p.N + (n < cols ? n : cols - 4) + (SW && t >= TG ? cols : 0));
    }
    i32x4 acc[NSUB][TPW];
#pragma unroll
    for (int s = 0; s < NSUB; ++s)
#pragma unroll
        for (int t = 0; t < TPW; ++t)
            acc[s][t] = i32x4{0, 0, 0, 0};
    u32x4 w[RING][TPW][2], x[RING][NSUB][2];
    auto load_w = [&](int j, uint32_t k, uint32_t past = 0) {
#pragma unroll
        for (int t = 0; t < TPW; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                w[j][t][h] = bload16(rw, wo[t] + past + 64 * h, k);
    };
    auto load_x = [&](int j, uint32_t k) {
        if constexpr (!QA)
#pragma unroll
        for (int s = 0; s < NSUB; ++s)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                x[j][s][h] = bload16(rx, xo[s] + 64 * h, k);
    };
    auto multiply = [&](int j, uint32_t k) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int s = 0; s < NSUB; ++s) {
                const u32x4 v = QA ? *reinterpret_cast<const u32x4 *>(s_rows + m * kRowPitch + k + 64 * h + q * 16) : x[j][s][h];
#pragma unroll
                for (int t = 0; t < TPW; ++t)
                    acc[s][t] = mfma_i8(w[j][t][h], v, acc[s][t]);
            }
    };
    // n groups from g on are this wave's, in rounds of RING: while a round is multiplied the next one is on its way
    const int G = p.K / 128;
    int g = wk * G / WK, n = (wk + 1) * G / WK - g;
    float as[NSUB];
    auto find_rows = [&]() {
        if constexpr (QA) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = wave + 4 * i;
                if (r >= rows)
                    break;
                auto value = [&](int v, int j) { return bf16_to_f32(j & 1 ? hv[i][v][j >> 1] >> 16 : hv[i][v][j >> 1] & 0xFFFFu); };
                uint32_t top = 0;                      // magnitude bits, as in the quantizer
#pragma unroll
                for (int v = 0; v < QV; ++v)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint32_t b = __float_as_uint(value(v, j)) & 0x7FFFFFFFu;
                        top = b > top ? b : top;
                    }
                const RowCodes codes(__uint_as_float(wave_reduce(top, [](uint32_t a, uint32_t b) { return b > a ? b : a; })));
#pragma unroll
                for (int v = 0; v < QV; ++v) {
                    uint32_t o[2] = {0, 0};
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        o[j >> 2] |= codes.code(value(v, j)) << (8 * (j & 3));
                    *reinterpret_cast<u32x2 *>(s_rows + r * kRowPitch + (lane + 64 * v) * 8) = u32x2{o[0], o[1]};
                }
                if (lane == 0)
                    s_scale[r] = codes.scale;
            }
            __syncthreads();
            as[0] = s_scale[m];                        // of a lane without a row: not used
            return;
        }
#pragma unroll
        for (int s = 0; s < NSUB; ++s) {
            const int ar = act_row(p, row[s], idx[s]);
            xo[s] = (uint32_t)ar * p.K + q * 16;
            as[s] = p.as[ar];
        }
    };
    auto at = [&](int j) { return (uint32_t)(g + j) * 128; };
    // The first round's weights set out before the tokens' rows are known. The waves of a workgroup meet in find_rows,
    // so there is no branch on n, which differs between them, around it: groups past a wave's last one are loaded from
    // behind the array, which fetches nothing (a weight offset is below 2^31).
#pragma unroll
    for (int j = 0; j < RING; ++j)
        load_w(j, at(j), j < n ? 0u : 1u << 31);
    __builtin_amdgcn_sched_barrier(0);
    find_rows();
    if (n >= RING) {
#pragma unroll
        for (int j = 0; j < RING; ++j)
            load_x(j, at(j));
        for (; n >= 2 * RING; n -= RING, g += RING)
#pragma unroll
            for (int j = 0; j < RING; ++j) {
                multiply(j, at(j));
                load_w(j, at(RING + j));
                load_x(j, at(RING + j));
            }
        n -= RING;
#pragma unroll
        for (int j = 0; j < RING; ++j) {
            multiply(j, at(j));
            if (j < n) {
                load_w(j, at(RING + j));
                load_x(j, at(RING + j));
            }
        }
        g += RING;
    } else {
#pragma unroll
        for (int j = 0; j < RING - 1; ++j)
            if (j < n)
                load_x(j, at(j));
    }
#pragma unroll
    for (int j = 0; j < RING - 1; ++j)
        if (j < n)
            multiply(j, at(j));
    if constexpr (WK > 1) {
        __shared__ i32x4 s_part[WN][WK - 1][NSUB * TPW][64];
#pragma unroll
        for (int s = 0; s < NSUB; ++s)
#pragma unroll
            for (int t = 0; t < TPW; ++t)
                if (wk > 0)
                    s_part[wn][wk - 1][s * TPW + t][lane] = acc[s][t];
        __syncthreads();
        if (wk > 0)
            return;
#pragma unroll
        for (int i = 0; i < WK - 1; ++i)
#pragma unroll
            for (int s = 0; s < NSUB; ++s)
#pragma unroll
                for (int t = 0; t < TPW; ++t)
                    acc[s][t] += s_part[wn][i][s * TPW + t][lane];
    }
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
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] = (float)acc[s][t][i] * as[s] * ws[t][i];
                if constexpr (SW)
                    v[i] = silu_fast(v[i]) * ((float)acc[s][t + TG][i] * as[s] * ws[t + TG][i]);
            }
            if constexpr (F32)
                *reinterpret_cast<floatx4 *>(static_cast<float *>(p.c) + crow + n) = floatx4{v[0], v[1], v[2], v[3]};
            else
                *reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(p.c) + crow + n) =
                    u32x2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
        }
    }
}

// At most this many chunks of CS rows: the full ones and one part-filled per expert with rows.
long long chunks_at_most(const W8GemmLaunch &g, int CS)
{
    if (!g.offsets)
        return (g.max_rows + CS - 1) / CS;
    return (long long)g.max_rows / CS + (g.num_experts < g.max_rows ? g.num_experts : g.max_rows);
}

template <int KIND, bool F32, int NSUB, int TPW, int WK, int RING, int QV = 0>
hipError_t launch_stream(const W8GemmLaunch &g, const W8Args &p, hipStream_t st)
{
    constexpr int TG = KIND == MOE_GEMM_W13_SWIGLU ? TPW / 2 : TPW;
    const int cols = KIND == MOE_GEMM_W13_SWIGLU ? g.N / 2 : g.N;
    constexpr int BC = 16 * TG * (4 / WK);
    const int blocks = (cols + BC - 1) / BC;
    hipLaunchKernelGGL((w8_stream_kernel<KIND, F32, NSUB, TPW, WK, RING, QV>),
                       dim3((unsigned)(chunks_at_most(g, 16 * NSUB) * blocks)), dim3(256), 0, st, p, blocks);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Many rows per expert: a workgroup of four waves computes BN weight rows x BM
// tokens, a wave 32 TN x 32 TM of them with v_mfma_i32_32x32x32_i8. Both
// operands pass through LDS, kStageK bytes of K to a stage, NS stages deep.
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
//
// 256 x 256 is the largest tile that four waves' accumulators (256 of a lane's
// 512 registers) hold, and LDS traffic asks for it: per 64 bytes of K a CU moves
// 64 KiB out of LDS and 32 KiB into it, 768 cycles at 128 B per cycle, beside
// 1024 cycles of MFMA. Dense 8192 x 14336 x 4096: 433 us, 2.22 POP/s, the matrix
// units 63% busy at 1.6 GHz (the clock that this load is given; 4.6 POP/s at
// 2.4 GHz for MFMAs alone). The small tiles are bound by the weight stream:
// 128 experts of 2048 -> 2 x 768, 128 tokens, 73 us, 5.6 TB/s.
// ---------------------------------------------------------------------------
constexpr int kStageK = 64;

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
__device__ __forceinline__ void wait_for()
{
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(N));
    __builtin_amdgcn_sched_barrier(0);
}

// The wait of an early step s < NS - 3, while copies that went out weights first
// are still on their way: the tokens' of NS - 3 - s stages, and s whole stages.
template <int NS, int LM, int L, int F = 0>
__device__ __forceinline__ void early_wait(int s)
{
    if constexpr (F < NS - 3) {
        if (s == F)
            wait_for<(NS - 3 - F) * LM + F * L>();
        else
            early_wait<NS, LM, L, F + 1>(s);
    }
}

template <int N>
__device__ __forceinline__ void wait_barrier()
{
    wait_for<N>();
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_s_barrier();
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_sched_barrier(0);
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

template <int KIND, bool F32, int TN, int TM, int NWN, int NWM, int NS>
__global__ __launch_bounds__(256, TN * TM > 8 ? 1 : 2) void w8_tile_kernel(W8Args p, int tn)
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
    int e, r0, rows, nt;
    if (!find_tile(p, BM, tn, blockIdx.x, lane, e, r0, rows, nt))
        return;
    e = uniform(e);
    const int cols = SW ? p.N / 2 : p.N;
    const int n0 = nt * BC;
    const uint32_t K = (uint32_t)p.K;

    // this lane's place in a copy of 16 rows, and the chunk that belongs there
    const int prow = lane >> 2;
    auto chunk_at = [&](int row) { return (uint32_t)(((lane & 3) ^ ((row >> 2) & 3)) * 16); };
    const __amdgpu_buffer_rsrc_t rw = make_rsrc(p.wq + (size_t)e * p.N * K, (uint32_t)p.N * K);
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(p.a, p.a_bytes), ri = index_rsrc(p);
    lds_byte *lds = (lds_byte *)s_dyn;
    uint32_t wo[LN], xo[LM];
    // one of a wave's L copies of a stage: K bytes [k, k + 64) to the stage at byte `at` of LDS
    auto copy_one = [&](int j, uint32_t at, uint32_t k) {
        lds_byte *dst = lds + at;
        if (j < LN)
            copy16(rw, dst + (wave * LN + j) * 1024, wo[j < LN ? j : 0], k);
        else
            copy16(rx, dst + BN * kStageK + (wave * LM + j - LN) * 1024, xo[j < LN ? 0 : j - LN], k);
    };
    // copies [j0, j1) of the first NS - 1 stages (past K: the last one again, which is never read)
    const int steps = p.K / kStageK;                    // even
    auto first_copies = [&](auto j0, auto j1) {
#pragma unroll
        for (int s = 0; s < NS - 1; ++s)
#pragma unroll
            for (int j = decltype(j0)::value; j < decltype(j1)::value; ++j)
                copy_one(j, s * kStageBytes, (uint32_t)(s < steps ? s : steps - 1) * kStageK);
    };
    using C0 = std::integral_constant<int, 0>;
    using CN = std::integral_constant<int, LN>;
    using CH = std::integral_constant<int, L / 2>;
    using CL = std::integral_constant<int, L>;
    // what the tokens' rows and the epilogue need sets out first: index entries
    // of the rows to copy and of the lane's result rows, the columns' scales
    const int half = lane >> 5, m32 = lane & 31;
    int xrow[LM], xidx[LM], crow[TM], cidx[TM];
#pragma unroll
    for (int j = 0; j < LM; ++j) {
        const int row = (wave * LM + j) * 16 + prow;
        xrow[j] = r0 + (row < rows ? row : rows - 1);
        xidx[j] = load_index(ri, xrow[j]);
    }
#pragma unroll
    for (int b = 0; b < TM; ++b) {
        const int m = (wm * TM + b) * 32 + m32;
        crow[b] = r0 + (m < rows ? m : rows - 1);
        cidx[b] = load_index(ri, crow[b]);
    }
    const int nw = n0 + wn * 32 * TG;                   // the wave's first column
    float wsv[TN][16];
    auto load_scales = [&]() {
#pragma unroll
        for (int t = 0; t < TN; ++t)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                int n = nw + half * 16 * TG + (t % TG) * 16 + g * 4;
                n = (n < cols ? n : cols - 4) + (SW && t >= TG ? cols : 0);
                const floatx4 v = *reinterpret_cast<const floatx4 *>(p.ws + (size_t)e * p.N + n);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    wsv[t][4 * g + i] = v[i];
            }
    };
    constexpr bool kScalesFirst = TN * TM <= 8;         // the largest tile has no registers left for them
    if constexpr (kScalesFirst)
        load_scales();
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < LN; ++j) {
        const int row = (wave * LN + j) * 16 + prow;    // row of the stage: wave's columns, tile, row of the tile
        const int w = row / (32 * TN), t = row / 32 % TN, r = row % 32;
        int n = n0 + w * 32 * TG + ((r >> 2) & 1) * 16 * TG + (t % TG) * 16 + (r >> 3) * 4 + (r & 3);
        n = n < cols ? n : cols - 1;
        wo[j] = (uint32_t)(n + (SW && t >= TG ? cols : 0)) * K + chunk_at(row);
    }
    // the weights set out before the tokens' rows are known
    first_copies(C0(), CN());
    __builtin_amdgcn_sched_barrier(0);
    float asv[TM];
#pragma unroll
    for (int b = 0; b < TM; ++b)
        asv[b] = p.as[act_row(p, crow[b], cidx[b])];
#pragma unroll
    for (int j = 0; j < LM; ++j)
        xo[j] = (uint32_t)act_row(p, xrow[j], xidx[j]) * K + chunk_at((wave * LM + j) * 16 + prow);
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
    // Step s multiplies stage s. In its middle the wave waits for its copies of
    // stage s + 1 (those of the NS - 3 after it stay in flight) and meets the other
    // waves: then stage s + 1 is whole, and every wave has read all of stage
    // s - 1, whose place takes stage s + NS - 1: half of its copies go out in the
    // second half of step s, half in the first half of step s + 1. Reads of
    // stage s may still be on their way at the meeting; its place is not
    // written before the next one. A step's second half has its fragments in
    // registers (or about to be) when the first half of the next step's are read.
    // Steps past the last multiply nothing: a stage past K is not copied, and
    // its place is read (in bounds) but not used.
    // (The first stages' copies went out weights first: until their tokens
    // are in, fewer may stay in flight.)
    Fr d0, d1;
    __builtin_amdgcn_sched_barrier(0);
    first_copies(CN(), CL());
    wait_barrier<(NS - 2) * LM>();
#pragma unroll
    for (int j = 0; j < TN + TM; ++j)
        read_one(j, s_dyn + f0, d0);
    uint32_t cur = 0, to = (NS - 2) * kStageBytes, k = (NS - 2) * kStageK;    // stage s; the place and K of the stage being copied
    auto after = [&](uint32_t at) { return at == (NS - 1) * kStageBytes ? 0u : at + kStageBytes; };
    int s = 0;
    if (steps > NS - 1) {
        half_step(d0, d1, cur + f1, C0(), C0(), 0, 0);  // stage NS - 2 is already on its way
        for (;; ++s) {
            early_wait<NS, LM, L>(s);
            wait_barrier<(NS - 3) * L>();
            to = after(to);
            k += kStageK;
            const uint32_t next = after(cur);
            half_step(d1, d0, next + f0, C0(), CH(), to, k);
            cur = next;
            if (s + NS >= steps)
                break;
            half_step(d0, d1, cur + f1, CH(), CL(), to, k);
        }
        // step s + 1 = steps - (NS - 1): the rest of the last stage's copies
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
    if constexpr (!kScalesFirst)
        load_scales();
    __syncthreads();
    constexpr int kElem = F32 ? 4 : 2;
    constexpr int kRow = 32 * TG * kElem;               // bytes of a row in the wave's columns
    constexpr int kPitch = kRow + 16;
    constexpr int kLanes = kRow / 16;                   // lanes that store a row
    static_assert(32 * kPitch * 4 <= kStageBytes * NS, "the epilogue's rows fit the stages");
    unsigned char *buf = s_dyn + wave * (32 * kPitch);
#pragma unroll
    for (int b = 0; b < TM; ++b) {
        const int mb = (wm * TM + b) * 32;
        if (mb >= rows)
            break;
        const float as = asv[b];
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

// A kernel's LDS limit is raised once on each device that launches it.
template <int KIND, bool F32, int TN, int TM, int NWN, int NWM, int NS>
void allow_lds(int bytes)
{
    constexpr int kMaxDevices = 64;
    static std::once_flag once[kMaxDevices];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices)
        return;
    std::call_once(once[dev], [bytes] {
        (void)hipFuncSetAttribute(reinterpret_cast<const void *>(&w8_tile_kernel<KIND, F32, TN, TM, NWN, NWM, NS>),
                                  hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    });
}

template <int KIND, bool F32, int TN, int TM, int NWN, int NWM, int NS>
hipError_t launch_tile(const W8GemmLaunch &g, const W8Args &p, hipStream_t st)
{
    constexpr bool SW = KIND == MOE_GEMM_W13_SWIGLU;
    constexpr int BN = 32 * TN * NWN, BM = 32 * TM * NWM, BC = SW ? BN / 2 : BN;
    constexpr int lds = (BN + BM) * kStageK * NS;       // 256 x 256: all of a CU's; the others: two workgroups to a CU
    const int cols = SW ? g.N / 2 : g.N;
    const int tn = (cols + BC - 1) / BC;
    const long long tm = chunks_at_most(g, BM);
    allow_lds<KIND, F32, TN, TM, NWN, NWM, NS>(lds);
    hipLaunchKernelGGL((w8_tile_kernel<KIND, F32, TN, TM, NWN, NWM, NS>), dim3((unsigned)(tm * tn)), dim3(256), lds, st, p,
                       tn);
    return hipGetLastError();
}

// The expected rows of an expert that has any, and the tiles that a kernel of BN weight rows x BM tokens would have.
struct Load {
    double reached, per;
    int cols, half;                                     // output columns; 2 where a column has two weight rows

    explicit Load(const W8GemmLaunch &g)
    {
        const double R = g.expected_rows < 1 ? 1.0 : (double)g.expected_rows;
        reached = g.offsets ? g.num_experts * (1.0 - pow(1.0 - 1.0 / g.num_experts, R)) : 1.0;
        per = R / reached;
        half = g.kind == MOE_GEMM_W13_SWIGLU ? 2 : 1;
        cols = g.N / half;
    }

    double items(int BN, int BM) const
    {
        const int BC = BN / half;
        return reached * ceil(per / BM) * ((cols + BC - 1) / BC);
    }
};

// Which kernel, from the expected rows R' of an expert that has any and the
// tiles (items) that each kernel would have; us on MI355X, operands rotating
// through more than the 256 MB memory-side cache:
//   R' <= 32 and few items: the streaming kernel, K split over a workgroup's waves, since
//     128 x 64 tiles leave CUs idle: dense 16 x 14336 x 4096 15.3 against 23.0 (M x N x K), 1 x 4096 x
//     4096 5.3 against 13.0, 30 x 4096 x 4096 9.9 against 14.0. A wave has as many tiles as leave
//     most CUs a workgroup: 1 x 4096 x 4096 with one 5.9, two 8.2, four 13.1 (before the default
//     policy). Where even 64 columns to a workgroup do, two waves of two tiles and half of K each
//     go before four tiles and a quarter: 8 x 14336 x 4096 14.9 against 16.5, 16 rows 15.3 against
//     16.1, 16 x 28672 x 4096 31.5 against 30.4
//   experts with R' <= 5 (SwiGLU), 10 (else): the streaming kernel, half of K to a wave, a quarter
//     from 2048 on: 128 experts, 2048 -> 2 x 768, 16 tokens 46.5 against 52.6 with 256 x 64 tiles, 64
//     tokens 69.0 against 72.5, 128 tokens 75.6 against 72.7; 768 -> 2048 26.2 against 29.8, 38.6 against 42.8, 256
//     tokens 56 against 45; 32 experts of 7168 -> 2 x 2048 with a row each 101 against 118. (Halves for
//     the long K: 106; quarters for the short one 32.4.)
//   up to R' = 40 (rows spread over experts; 64 where the count is exact): tiles of 64 rows, of 256
//     weight rows where that gives 1.5 workgroups per CU, else 128 (128 experts, 2048 -> 2 x 768:
//     256 tokens 73.9 against 79.8; 256 x 128 tiles 80.8)
//   above: 128 rows, with 256 weight rows where that gives 1.5 workgroups per CU (32 experts,
//     7168 -> 2 x 2048, 64 rows each: 188 against 204 with 128; tiles of 64 rows 266), else 128 (dense
//     256 x 14336 x 4096 29 against 53), and 64 rows where those leave CUs idle (333 x 2064 x
//     768: 5.9 against 7.1)
//   256 x 256 where it gives nearly every CU a tile (dense 4096 x 4096 x 7168 112 against 132 with
//     256 x 128 and 159 with 128 x 128)
// Dense products of 33 to some hundred rows have no form that splits K, and few workgroups: 64, 128
// and 256 rows of 4096 x 4096 take 22 us each (32, 64 and 128 workgroups), of 2112 x 7168 36 (17,
// 34 and 68), beside 3.3 and 3.0 us for reading the weights; the border at 32 rows is one between
// what there is (30 x 4096 x 4096 10.8)
template <int KIND, bool F32>
hipError_t launch_kind(const W8GemmLaunch &g, const W8Args &p, hipStream_t st)
{
    constexpr bool SW = KIND == MOE_GEMM_W13_SWIGLU;
    const Load load(g);
    const double per = load.per;
    auto items = [&](int BN, int BM) { return load.items(BN, BM); };
    if constexpr (!SW && !F32)
        if (g.a_bf16)
            return g.K <= 1024 ? launch_stream<KIND, F32, 1, 2, 2, 2, 2>(g, p, st)
                               : launch_stream<KIND, F32, 1, 2, 2, 2, 4>(g, p, st);
    if (per <= 32.0 && items(128, 64) < 256.0) {
        // a wave's tiles: as many as still give most CUs a workgroup
        const bool few4 = items(64, 64) < 192.0, few2 = items(32, 64) < 192.0;
        if (per <= 16.0) {
            if (!few4)
                return launch_stream<KIND, F32, 1, 2, 2, 2>(g, p, st);
            if constexpr (!SW)
                if (few2)
                    return launch_stream<KIND, F32, 1, 1, 4, 4>(g, p, st);
            return launch_stream<KIND, F32, 1, 2, 4, 4>(g, p, st);
        }
        return few4 ? launch_stream<KIND, F32, 2, 2, 4, 2>(g, p, st) : launch_stream<KIND, F32, 2, 4, 4, 2>(g, p, st);
    }
    if (g.offsets && per <= (SW ? 5.0 : 10.0))
        return g.K < 2048 ? launch_stream<KIND, F32, 1, 2, 2, 2>(g, p, st) : launch_stream<KIND, F32, 1, 2, 4, 4>(g, p, st);
    if (per <= (g.offsets ? 40.0 : 64.0))
        return items(256, 64) >= 384.0 ? launch_tile<KIND, F32, 2, 2, 4, 1, 4>(g, p, st)
                                       : launch_tile<KIND, F32, 2, 1, 2, 2, 5>(g, p, st);
    if (per >= 256.0 && items(256, 256) >= 240.0)
        return launch_tile<KIND, F32, 4, 4, 2, 2, 5>(g, p, st);
    if (items(256, 128) >= 384.0)
        return launch_tile<KIND, F32, 4, 2, 2, 2, 3>(g, p, st);
    return items(128, 128) >= 128.0 ? launch_tile<KIND, F32, 2, 2, 2, 2, 5>(g, p, st)
                                    : launch_tile<KIND, F32, 2, 1, 2, 2, 5>(g, p, st);
}

}  // namespace

// Where launch_kind streams such a product with half of K to a wave: the layer saves the quantizer's launch, 128 experts
// of 2048/768 with one token 20.5 -> 18.0 us, 16 tokens 80.6 -> 77.5, 128 tokens 124.8 -> 122.2.
bool quantizes_rows(const W8GemmLaunch &g)
{
    const Load load(g);
    return g.kind == MOE_GEMM_W2 && !g.c_f32 && g.offsets && !g.a_row_index && g.K < 2048 && load.per <= 10.0 &&
           load.items(64, 64) >= 192.0;
}

hipError_t launch_w8_gemm(const W8GemmLaunch &g, hipStream_t st)
{
    const W8Args p{g.a, (uint32_t)((size_t)(g.a_row_index ? g.max_rows / g.top_k : g.max_rows) * g.K), g.as, g.a_bf16, g.a_row_index,
                   g.top_k, g.offsets, g.max_rows, g.num_experts, g.wq, g.ws, g.c, g.K, g.N};
    if (g.kind == MOE_GEMM_W13_SWIGLU)
        return launch_kind<MOE_GEMM_W13_SWIGLU, false>(g, p, st);
    if (g.c_f32)
        return launch_kind<MOE_GEMM_W2, true>(g, p, st);
    return launch_kind<MOE_GEMM_W2, false>(g, p, st);
}

}  // namespace moe
