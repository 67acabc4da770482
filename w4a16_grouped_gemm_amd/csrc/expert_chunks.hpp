// expert_chunks.hpp -- which rows of which expert a workgroup of a grouped 8-bit
// product computes, found on the device from the experts' offsets, and how many
// workgroups the host launches for them.
//
// P, a kernel's arguments: a_row_index, top_k, offsets (NULL: one dense expert),
// max_rows (rows of the result) and E. G, a launch: offsets, max_rows,
// num_experts, expected_rows, kind and N.
#pragma once

#include <cmath>

#include "gemm_core.hpp"

namespace moe {

namespace {

// Activation row of result row r, in two steps: the index entry (0 where there
// is no index; loaded first, ahead of what can go out without it), then the row,
// kept inside the array whatever the entry holds.
template <class P>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t index_rsrc(const P &p)
{
    return make_rsrc(p.a_row_index, p.a_row_index ? (uint32_t)p.max_rows * 4u : 0u);
}

__device__ __forceinline__ int load_index(__amdgpu_buffer_rsrc_t ri, int r)
{
    return (int)__builtin_amdgcn_raw_buffer_load_b32(ri, (uint32_t)r * 4u, 0, 0);
}

template <class P>
__device__ __forceinline__ int act_row(const P &p, int r, int i)
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
template <bool CLAMP, class P>
__device__ __forceinline__ int scan_chunks(const P &p, uint32_t CS, int lane, int e0, int before, Chunks &c)
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

// Chunk `chunk`, where it is one of c's: its expert, first row and rows; in only, where asked for, whether the expert has
// no other.
template <class P>
__device__ __forceinline__ bool pick_chunk(const P &p, int CS, int e0, int chunk, const Chunks &c, int &e, int &r0,
                                           int &rows, bool *only = nullptr)
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
            if (only)
                *only = __builtin_amdgcn_readlane(c.n[i], l) == 1;
        }
    }
    rows = rows < CS ? rows : CS;
    return found;
}

template <class P>
__device__ __forceinline__ bool dense_chunk(const P &p, int CS, int chunk, int &e, int &r0, int &rows)
{
    e = 0;
    r0 = chunk * CS;
    rows = p.max_rows - r0;
    rows = rows < CS ? rows : CS;
    return rows > 0;
}

// Chunk `chunk`: its expert, first row and rows; false past the last chunk. One
// wave, every lane gets the result.
template <bool CLAMP, class P>
__device__ __forceinline__ bool find_chunk(const P &p, int CS, int chunk, int lane, int &e, int &r0, int &rows,
                                           bool *only = nullptr)
{
    if (only)
        *only = p.max_rows <= CS;
    if (!p.offsets)
        return dense_chunk(p, CS, chunk, e, r0, rows);
    e = r0 = rows = 0;
    for (int e0 = 0, before = 0; e0 < p.E; e0 += 64 * kScan) {
        Chunks c;
        before = scan_chunks<CLAMP>(p, CS, lane, e0, before, c);
        if (chunk < before)
            return pick_chunk(p, CS, e0, chunk, c, e, r0, rows, only);
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

// The chunks that there are; of the last 256 experts' at most, c holds where they start.
template <class P>
__device__ __forceinline__ int count_chunks(const P &p, int CS, int lane, Chunks &c)
{
    if (!p.offsets)
        return (p.max_rows + CS - 1) / CS;
    int tm = 0;
    for (int e0 = 0; e0 < p.E; e0 += 64 * kScan)
        tm = scan_chunks<true>(p, CS, lane, e0, tm, c);
    return tm;
}

// Segments that do not overlap have no more chunks (chunks_at_most on the device). Overlapping ones can have E times as
// many: a workgroup that takes chunk after chunk of all that are counted stops here.
template <class P>
__device__ __forceinline__ int most_chunks(const P &p, int CS)
{
    return p.offsets ? p.max_rows / CS + min(p.E, p.max_rows) : (p.max_rows + CS - 1) / CS;
}

// Where i of n lands so that XCD x, to which workgroups x, x + 8, ... go, takes the x-th share.
__device__ __forceinline__ int xcd_share(int n, int i)
{
    const int per = n / kXcds, extra = n % kXcds, x = i % kXcds;
    return x * per + (x < extra ? x : extra) + i / kXcds;
}

// Tile b of those that there are (tm chunks, tn column tiles; b counts up to as many as there can be): XCD x (tiles x, x +
// 8, ... as workgroups are) takes the x-th share of them, so that those which share operands also share an L2. False past
// XCD x's last.
__device__ __forceinline__ bool have_tile(int tm, int tn, int b, int &mt, int &nt)
{
    const int total = tm * tn, per = total / kXcds, extra = total % kXcds;
    const int x = b % kXcds, ix = b / kXcds;
    if (ix >= per + (x < extra ? 1 : 0))
        return false;
    tile_of(xcd_share(total, b), tm, tn, mt, nt);
    return true;
}

template <class P>
__device__ __forceinline__ bool rows_of_tile(const P &p, int CS, int mt, int lane, const Chunks &c, int &e, int &r0,
                                             int &rows)
{
    if (!p.offsets)
        return dense_chunk(p, CS, mt, e, r0, rows);
    e = r0 = rows = 0;
    if (p.E <= 64 * kScan)
        return pick_chunk(p, CS, 0, mt, c, e, r0, rows);
    return find_chunk<true>(p, CS, mt, lane, e, r0, rows);
}

// The tile of workgroup b.
template <class P>
__device__ __forceinline__ bool find_tile(const P &p, int CS, int tn, int b, int lane, int &e, int &r0, int &rows,
                                          int &nt)
{
    Chunks c;
    const int tm = count_chunks(p, CS, lane, c);
    int mt;
    return have_tile(tm, tn, b, mt, nt) && rows_of_tile(p, CS, mt, lane, c, e, r0, rows);
}

// At most this many chunks of CS rows: the full ones and one part-filled per expert with rows.
template <class G>
long long chunks_at_most(const G &g, int CS)
{
    if (!g.offsets)
        return (g.max_rows + CS - 1) / CS;
    return (long long)g.max_rows / CS + (g.num_experts < g.max_rows ? g.num_experts : g.max_rows);
}

// The expected rows of an expert that has any, and the tiles that a kernel of BN weight rows x BM tokens would have.
struct Load {
    double reached, per;
    int cols, half;                                     // output columns; 2 where a column has two weight rows

    template <class G>
    explicit Load(const G &g)
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

}  // namespace

}  // namespace moe
