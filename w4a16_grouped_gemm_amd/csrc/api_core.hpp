// api_core.hpp -- what the C entry points of the 8-bit operators share: limits,
// alignment, overlap and the status of a launch.
#pragma once

#include "common.hpp"

namespace moe {

namespace {

constexpr size_t kAlign = 256;
constexpr int32_t kMaxDenseCols = 1 << 18;

size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

moe_status from_hip(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

// [a, a + na) and [b, b + nb) share bytes.
bool overlap(const void *a, size_t na, const void *b, size_t nb)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && x < y + nb && y < x + na;
}

// Rows of one norm or quantizer launch: fewer than 2^32 threads (a wave, 256 or 1024 threads per row).
bool norm_rows_fit(int64_t rows, int32_t K)
{
    return rows < (1LL << (K <= 1024 ? 25 : K <= 16384 ? 23 : 21)) && rows * (int64_t)K * 2 < (1LL << 40);
}

}  // namespace

}  // namespace moe
