// route_scored.hip -- top-k routing on scores: sigmoid or softmax, a bias for
// the selection only, groups of experts, renormalised weights.
//
// With l the logits, b the bias (0 if absent), the binary32 scores are
//   s_e = sigmoid(l_e)  or  s_e = exp(l_e - max l) / sum_f exp(l_f - max l)
// and the selection goes by c_e = s_e + b_e (a binary32 sum), larger first,
// lower index first among equals. With G groups of E / G consecutive experts
// a group's score is its largest c, or the sum of its two largest; the
// topk_groups best groups (lower index first among equals) keep their experts.
// Slot i's weight is s_{e_i} (without the bias), over the sum of the k chosen
// scores if renormalised, times a factor.
//
// A selection has to come out the same however it is computed, so the score
// is the exact function's value rounded to binary32: the exponentials and
// their sum are formed in binary64 to about 2^-44, which changes that rounding
// for about one score in 2^19, and a selection only where that score's
// neighbour is the next binary32 number as well. Everything after it is a
// binary32 comparison or one addition.
//
// Lane q of the TL lanes that hold a token has its experts q PL .. q PL + PL - 1
// (so groups of experts are groups of neighbouring lanes, reduced by DPP); k
// rounds take the largest remaining key (the order-preserving integer image of
// c) and retire it. Bound by the rounds' chain, each a maximum over lanes, a
// ballot and a select that wait for one another: 8192 tokens give two waves per
// SIMD, and vector instructions are active in 52% of the busy cycles. With TL =
// 64 a token costs 632 of them, most in the rounds, whose reductions then serve
// one token; with TL = 16 four tokens share a wave and its rounds, 313 each, but
// the wave takes twice as long. 256 experts in 8 groups, top 8, us with 64 lanes
// and with 16: 2048 tokens 4.6 and 6.1, 4096 6.5 and 6.2, 8192 10.2 and 8.6,
// 32768 31.6 and 22.7. Groups that are not 2^n whole lanes have 64 lanes only, a
// lane to a group: 160 experts in 8 groups, top 6, 3.9 us for one token, 4.3
// for 512, 11.0 for 8192.
#include "route_core.hpp"
#include "w8a8.hpp"

namespace moe {

namespace {

constexpr int kScoredWaves = 4;
constexpr int kManyTokens = 4096;        // with 16 lanes per token a wave for each SIMD

// Key of an expert that may be chosen only after all others (masked): below that of -inf, which a bias can make of c;
// in its group's score it counts as -inf. And of one that may not be chosen.
constexpr uint32_t kLowestKey = 0x007FFFFFu;           // ordered_bits(-inf)
constexpr uint32_t kMaskedKey = kLowestKey - 1;
constexpr uint32_t kNoKey = 0u;

// The maximum of the TL lanes that hold a token, in each of them.
template <int TL>
__device__ __forceinline__ uint32_t token_max(uint32_t v);

template <>
__device__ __forceinline__ uint32_t token_max<16>(uint32_t v) { return row_reduce<true>(v); }

template <>
__device__ __forceinline__ uint32_t token_max<64>(uint32_t v)
{
    v = row_reduce<true>(v);
    uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xA, 0xF, false);   // row_bcast:15
    v = o > v ? o : v;
    o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xC, 0xF, false);            // row_bcast:31
    v = o > v ? o : v;
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// exp(x) in binary64 for |x| <= 110: x = n ln 2 + r with |r| <= ln 2 / 2, the
// polynomial of degree 9 that equals exp(r) at the ten Chebyshev nodes of that
// interval (within 2^-45 of it), times 2^n. n is rounded by adding 1.5 2^52,
// whose sum holds it in its low bits.
__device__ __forceinline__ double exp_near(double x)
{
    const double t = __builtin_fma(x, 0x1.71547652b82fep+0, 0x1.8p+52);
    const double r = __builtin_fma(t - 0x1.8p+52, -0x1.62e42fefa39efp-1, x);
    double y = 0x1.72e107c874de9p-19;
    y = __builtin_fma(y, r, 0x1.a17df0d914d6cp-16);
    y = __builtin_fma(y, r, 0x1.a01994c849582p-13);
    y = __builtin_fma(y, r, 0x1.6c162bb7d965cp-10);
    y = __builtin_fma(y, r, 0x1.11111123bf154p-7);
    y = __builtin_fma(y, r, 0x1.55555588b8403p-5);
    y = __builtin_fma(y, r, 0x1.5555555550d88p-3);
    y = __builtin_fma(y, r, 0x1.ffffffffe74f1p-2);
    y = __builtin_fma(y, r, 0x1.0000000000006p+0);
    y = __builtin_fma(y, r, 0x1.000000000003dp+0);
    return __builtin_ldexp(y, (int)(uint32_t)__builtin_bit_cast(uint64_t, t));
}

// 1 / d for 1 <= d < 2^200: the hardware's estimate (2^-23 or better) and a Newton step, which squares its error.
__device__ __forceinline__ double reciprocal(double d)
{
    const double y = __builtin_amdgcn_rcp(d);
    return __builtin_fma(__builtin_fma(-d, y, 1.0), y, y);
}

// (a, b) and another lane's: the two largest of the four.
__device__ __forceinline__ void merge_top2(uint32_t &a, uint32_t &b, uint32_t oa, uint32_t ob)
{
    const uint32_t lo = a < oa ? a : oa, hi = a < oa ? oa : a;
    b = b > ob ? b : ob;
    b = b > lo ? b : lo;
    a = hi;
}

// B keys in descending order, at[i] being where the i-th was (neighbours change places only where the second is
// larger, so equal ones stay in index order).
template <int B>
__device__ __forceinline__ void sort_keys(uint32_t *key, uint32_t &which)
{
    int at[B];
#pragma unroll
    for (int i = 0; i < B; ++i)
        at[i] = i;
#pragma unroll
    for (int round = 0; round < B; ++round)
#pragma unroll
        for (int i = round & 1; i + 1 < B; i += 2) {
            const uint32_t a = key[i], c = key[i + 1];
            const int ia = at[i], ic = at[i + 1];
            const bool swap = c > a;
            key[i] = swap ? c : a;
            key[i + 1] = swap ? a : c;
            at[i] = swap ? ic : ia;
            at[i + 1] = swap ? ia : ic;
        }
    which = 0;
#pragma unroll
    for (int i = 0; i < B; ++i)
        which |= (uint32_t)at[i] << (8 * i);
}

// TL: lanes that hold a token (64, or 16 and four tokens to a wave).
// GROUPS: 0 none; 1 a group is GL = 2^n whole lanes; 2 any.
template <int TL, int PL, int GROUPS>
__global__ __launch_bounds__(kScoredWaves * 64) void route_scored_kernel(
    int T, int E, int k, moe_router r, const float *__restrict__ logits, const float *__restrict__ bias, bool vec,
    int32_t *__restrict__ ids, float *__restrict__ w)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int q = lane % TL, slot = wave * (64 / TL) + lane / TL;                   // slot: the workgroup's tokens
    const int t = blockIdx.x * (kScoredWaves * 64 / TL) + slot;
    const bool there = t < T;
    const float *row = logits + (size_t)(there ? t : T - 1) * E;
    const int e0 = q * PL;
    float l[PL], b[PL];
    if (vec) {                                         // a lane's experts are all there or none is
        typedef float vecf __attribute__((ext_vector_type(PL < 4 ? PL : 4)));
        constexpr int W = PL < 4 ? PL : 4;
        const int at = e0 < E ? e0 : 0;
#pragma unroll
        for (int i = 0; i < PL; i += W) {
            const vecf v = *reinterpret_cast<const vecf *>(row + at + i);
            vecf c = {};
            if (bias)
                c = *reinterpret_cast<const vecf *>(bias + at + i);
#pragma unroll
            for (int j = 0; j < W; ++j) {
                if constexpr (W == 1) {
                    l[i] = v[0];
                    b[i] = c[0];
                } else {
                    l[i + j] = v[j];
                    b[i + j] = c[j];
                }
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < PL; ++i) {
            const int e = e0 + i < E ? e0 + i : E - 1;
            l[i] = row[e];
            b[i] = bias ? bias[e] : 0.0f;
        }
    }
#pragma unroll
    for (int i = 0; i < PL; ++i)
        l[i] = e0 + i < E ? l[i] : -__builtin_inff();
    float score[PL];
    if (r.score == MOE_SCORE_SIGMOID) {
#pragma unroll
        for (int i = 0; i < PL; ++i)
            // past 110 either way it is 0 or 1 in binary32 (a NaN is masked below)
            score[i] = (float)reciprocal(1.0 + exp_near(-(double)__builtin_amdgcn_fmed3f(l[i], -110.0f, 110.0f)));
    } else {
        float m = -__builtin_inff();
#pragma unroll
        for (int i = 0; i < PL; ++i)
            m = __builtin_fmaxf(m, l[i]);              // the larger, or the one that is no NaN
        const float top = from_ordered_bits(token_max<TL>(ordered_bits(m)));
        double p[PL], sum = 0.0;
#pragma unroll
        for (int i = 0; i < PL; ++i) {
            // below -110 (a NaN too, masked below) the share, under e^-110 < 2^-150, rounds to 0 and adds nothing to a
            // sum that holds e^0
            p[i] = exp_near(__builtin_fmax((double)l[i] - (double)top, -110.0));
            sum += p[i];
        }
#pragma unroll
        for (int d = 1; d < TL; d *= 2)
            sum += __shfl_xor(sum, d);
        // an infinite logit leaves no shares
        const double inv = top < __builtin_inff() ? 1.0 / sum : __builtin_nan("");
#pragma unroll
        for (int i = 0; i < PL; ++i)
            score[i] = (float)(p[i] * inv);
    }
    uint32_t key[PL];
#pragma unroll
    for (int i = 0; i < PL; ++i) {
        const float c = score[i] + b[i];               // never -0: a score is +0 or more
        const bool masked = !(c == c) | !(l[i] > -__builtin_inff());           // NaN too
        const uint32_t u = __float_as_uint(c);
        score[i] = masked ? 0.0f : score[i];
        key[i] = masked ? kMaskedKey : u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
        key[i] = e0 + i < E ? key[i] : kNoKey;
    }
    if constexpr (GROUPS > 0) {
        const int G = r.num_groups, size = E / G;
        uint32_t a = kLowestKey, b2 = kLowestKey;      // the two largest keys of a group
        int my_g, gl;                                  // the lane's group; lanes from one group's holder to the next's
        if constexpr (GROUPS == 1) {
#pragma unroll
            for (int i = 0; i < PL; ++i)
                merge_top2(a, b2, key[i], 0u);
            gl = size / PL;
            my_g = q / gl;
#define MOE_TOP2_STEP(n, ctrl)                                                                             \
            if (gl > n)                                                                                    \
                merge_top2(a, b2, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)a, ctrl, 0xF, 0xF, false), \
                           (uint32_t)__builtin_amdgcn_update_dpp(0, (int)b2, ctrl, 0xF, 0xF, false));
            MOE_TOP2_STEP(1, 0xB1)     // quad_perm [1,0,3,2]
            MOE_TOP2_STEP(2, 0x4E)     // quad_perm [2,3,0,1]
            MOE_TOP2_STEP(4, 0x141)    // row_half_mirror
            MOE_TOP2_STEP(8, 0x140)    // row_mirror
#undef MOE_TOP2_STEP
            if (TL > 16 && gl > 16)
                merge_top2(a, b2, __shfl_xor(a, 16), __shfl_xor(b2, 16));
            if (TL > 16 && gl > 32)
                merge_top2(a, b2, __shfl_xor(a, 32), __shfl_xor(b2, 32));
        } else {
            __shared__ uint32_t s_key[kScoredWaves][PL * 64];
#pragma unroll
            for (int i = 0; i < PL; ++i)
                s_key[wave][e0 + i] = key[i];
            __syncthreads();
            if (lane < G)                              // lane g holds group g
#pragma unroll 4
                for (int i = 0; i < size; ++i)
                    merge_top2(a, b2, s_key[wave][lane * size + i], 0u);
            gl = 1;
            my_g = lane;
        }
        const uint32_t gk = r.group_top == 2 ? ordered_bits(from_ordered_bits(a) + from_ordered_bits(b2)) : a;
        int ahead = 0;                                 // groups that come before this one: earlier ones with as large a
        for (int g = 0; g < G; ++g) {                  // key, later ones with a larger one (no key is 2^32 - 1)
            const uint32_t o = TL == 64 ? (uint32_t)__builtin_amdgcn_readlane((int)gk, g * gl)
                                        : (uint32_t)__shfl((int)gk, g * gl, TL);
            ahead += o >= gk + (g < my_g ? 0u : 1u);
        }
        if constexpr (GROUPS == 1) {
#pragma unroll
            for (int i = 0; i < PL; ++i)
                key[i] = ahead < r.topk_groups ? key[i] : kNoKey;
        } else {
            const uint64_t keep = __ballot(lane < G && ahead < r.topk_groups);
#pragma unroll
            for (int i = 0; i < PL; ++i) {
                const int e = e0 + i;
                if (e >= E || !(keep >> (e / size) & 1))
                    key[i] = kNoKey;
            }
        }
    }
    int my_e = 0;
    float my_s = 0.0f;                                 // lane q < k: slot q's score
    if constexpr (TL == 16) {
        // Blocks of four experts in descending order: the lane's largest is a block's first. The lane that holds a
        // round's expert writes it down; the scores are looked up at the end.
        constexpr int NB = PL / 4;
        __shared__ int s_e[kScoredWaves * 4][16];
        __shared__ float s_score[kScoredWaves * 4][16 * PL];
#pragma unroll
        for (int i = 0; i < PL; ++i)
            s_score[slot][e0 + i] = score[i];
        u32x4 blk[NB];
        uint32_t which[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            sort_keys<4>(key + 4 * b, which[b]);
            blk[b] = u32x4{key[4 * b], key[4 * b + 1], key[4 * b + 2], key[4 * b + 3]};
        }
        const int shift = lane & 16;
        for (int j = 0; j < k; ++j) {
            uint32_t top = blk[0][0];
#pragma unroll
            for (int b = 1; b < NB; ++b)
                top = blk[b][0] > top ? blk[b][0] : top;
            const uint32_t m = token_max<16>(top);
            const uint64_t at = __ballot(top == m);
            const uint32_t field = ((lane & 32 ? (uint32_t)(at >> 32) : (uint32_t)at) >> shift) & 0xFFFFu;
            const bool mine = __builtin_ctz(field) == q;
            bool free = mine;                          // the first block that has it
            int e = 0;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const bool hit = free & (blk[b][0] == m);
                e = hit ? e0 + 4 * b + (int)(which[b] & 255u) : e;
                blk[b] = hit ? u32x4{blk[b][1], blk[b][2], blk[b][3], kNoKey} : blk[b];
                which[b] = hit ? which[b] >> 8 : which[b];
                free = free & !hit;
            }
            if (mine)
                s_e[slot][j] = e;
        }
        __builtin_amdgcn_wave_barrier();               // the wave's own writes, in order before its reads
        if (q < k) {
            my_e = s_e[slot][q];
            my_s = s_score[slot][my_e];
        }
    } else if constexpr (PL <= 4) {
        // the lane's keys in descending order, which expert each one was in the bytes of `which`
        uint32_t which;
        sort_keys<PL>(key, which);
        for (int j = 0; j < k; ++j) {
            const uint32_t m = token_max<64>(key[0]);
            const int owner = __builtin_ctzll(__ballot(key[0] == m));
            const int e = __builtin_amdgcn_readlane(e0 + (int)(which & 255u), owner);
            my_e = lane == j ? e : my_e;
            const bool mine = lane == owner;
#pragma unroll
            for (int i = 0; i < PL; ++i)
                key[i] = mine ? (i + 1 < PL ? key[i + 1 < PL ? i + 1 : i] : kNoKey) : key[i];
            which = mine ? which >> 8 : which;
        }
    } else {
        for (int j = 0; j < k; ++j) {
            uint32_t bv = 0;
#pragma unroll
            for (int i = 0; i < PL; ++i)
                bv = key[i] > bv ? key[i] : bv;
            int at = 0;                                // the lane's first expert that has it
#pragma unroll
            for (int i = PL - 1; i >= 0; --i)
                at = key[i] == bv ? i : at;
            const uint32_t m = token_max<64>(bv);
            const int owner = __builtin_ctzll(__ballot(bv == m));
            const int e = __builtin_amdgcn_readlane(e0 + at, owner);
            my_e = lane == j ? e : my_e;
            if (lane == owner)
#pragma unroll
                for (int i = 0; i < PL; ++i)
                    key[i] = i == at ? kNoKey : key[i];
        }
    }
    if constexpr (TL == 64) {                          // from the lane that has it
#pragma unroll
        for (int i = 0; i < PL; ++i) {
            const float v = __int_as_float(__builtin_amdgcn_ds_bpermute(my_e / PL * 4, __float_as_int(score[i])));
            my_s = my_e % PL == i ? v : my_s;
        }
        my_s = lane < k ? my_s : 0.0f;
    }
    float z = my_s;                                    // lanes q >= k hold 0
#define MOE_DPP_ADD(ctrl) z += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(z), ctrl, 0xF, 0xF, false));
    MOE_DPP_ADD(0xB1)      // quad_perm [1,0,3,2]
    MOE_DPP_ADD(0x4E)      // quad_perm [2,3,0,1]
    MOE_DPP_ADD(0x141)     // row_half_mirror
    MOE_DPP_ADD(0x140)     // row_mirror
#undef MOE_DPP_ADD
    if (there && q < k) {
        const float wt = r.renormalize ? (z > 0.0f ? my_s / z : 0.0f) : my_s;
        ids[(size_t)t * k + q] = my_e;
        w[(size_t)t * k + q] = wt * r.scale;
    }
}

// Groups of `size` experts are 2^n whole lanes of PL experts.
bool whole_lanes(int size, int PL)
{
    const int gl = size / PL;
    return size % PL == 0 && (gl & (gl - 1)) == 0;
}

template <int TL, int PL>
void launch_scored(int T, int E, int k, const moe_router &r, const float *logits, const float *bias, int32_t *ids,
                   float *w, hipStream_t st)
{
    constexpr size_t W = PL < 4 ? PL : 4;              // values of a vector load
    const bool vec = E % PL == 0 && reinterpret_cast<uintptr_t>(logits) % (4 * W) == 0 &&
                     reinterpret_cast<uintptr_t>(bias) % (4 * W) == 0;
    constexpr int TPB = kScoredWaves * 64 / TL;
    const dim3 grid((T + TPB - 1) / TPB), block(kScoredWaves * 64);
    if (r.num_groups == 1)
        hipLaunchKernelGGL((route_scored_kernel<TL, PL, 0>), grid, block, 0, st, T, E, k, r, logits, bias, vec, ids, w);
    else if (whole_lanes(E / r.num_groups, PL))
        hipLaunchKernelGGL((route_scored_kernel<TL, PL, 1>), grid, block, 0, st, T, E, k, r, logits, bias, vec, ids, w);
    else if constexpr (TL == 64)
        hipLaunchKernelGGL((route_scored_kernel<TL, PL, 2>), grid, block, 0, st, T, E, k, r, logits, bias, vec, ids, w);
}

}  // namespace

hipError_t launch_route_scored(const moe_shape &sh, const moe_router &r, const float *logits, const float *bias,
                               int32_t *ids, float *w, hipStream_t st)
{
    const int T = sh.num_tokens, E = sh.num_experts, k = sh.top_k;
    // 16 lanes per token from the number on whose waves fill the GPU (figures at the top; with 128 experts 4.5 and 4.5
    // at 4096 tokens, 6.6 and 5.3 at 8192; with 64 3.8 and 3.5, 5.3 and 3.9)
    const int pl16 = E <= 64 ? 4 : E <= 128 ? 8 : 16;
    if (T >= kManyTokens && E <= 256 && (r.num_groups == 1 || whole_lanes(E / r.num_groups, pl16))) {
        if (pl16 == 4)
            launch_scored<16, 4>(T, E, k, r, logits, bias, ids, w, st);
        else if (pl16 == 8)
            launch_scored<16, 8>(T, E, k, r, logits, bias, ids, w, st);
        else
            launch_scored<16, 16>(T, E, k, r, logits, bias, ids, w, st);
    } else if (E <= 64)
        launch_scored<64, 1>(T, E, k, r, logits, bias, ids, w, st);
    else if (E <= 128)
        launch_scored<64, 2>(T, E, k, r, logits, bias, ids, w, st);
    else if (E <= 256)
        launch_scored<64, 4>(T, E, k, r, logits, bias, ids, w, st);
    else if (E <= 512)
        launch_scored<64, 8>(T, E, k, r, logits, bias, ids, w, st);
    else
        launch_scored<64, kMaxExperts / 64>(T, E, k, r, logits, bias, ids, w, st);
    return hipGetLastError();
}

}  // namespace moe
