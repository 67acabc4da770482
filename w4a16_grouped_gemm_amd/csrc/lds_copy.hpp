// lds_copy.hpp -- copies from memory straight to LDS, the counted waits and the
// meetings of a workgroup's waves that go with them, and the order of a loop's
// instructions around the matrix unit's.
#pragma once

#include "gemm_core.hpp"

namespace moe {

namespace {

typedef __attribute__((address_space(3))) unsigned char lds_byte;

constexpr uint32_t vmcnt_imm(int n)                   // s_waitcnt vmcnt(n), other counters untouched
{
    return (uint32_t)((n & 15) | ((n >> 4) << 14) | (7 << 4) | (15 << 8));
}

// 16 bytes per lane from memory to LDS: lane l's to dst + 16 l. NT: non-temporal, as bload16_codes.
template <bool NT = false>
__device__ __forceinline__ void copy16(__amdgpu_buffer_rsrc_t r, lds_byte *dst, uint32_t voff, uint32_t soff)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, dst, 16, voff, soff, 0, NT ? 2 : 0);
}

template <int N>
__device__ __forceinline__ void wait_for()
{
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(N));
    __builtin_amdgcn_sched_barrier(0);
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

}  // namespace

}  // namespace moe
