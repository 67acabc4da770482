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
// their sum are formed in binary64 to about 2^-42, which changes that rounding
// for about one score in 2^17, and a selection only where that score's
// neighbour is the next binary32 number as well. Everything after it is a
// binary32 comparison or one addition.
//
// One wave holds a token, lane q its experts q PL .. q PL + PL - 1 (so groups
// of experts are groups of neighbouring lanes, reduced by DPP); k rounds take
// the largest remaining key (the order-preserving integer image of c) and
// retire it. Bound by instructions (about 600 per token, the vector units 85%
// busy): 8192 tokens of 256 experts in 8 groups, top 8: 10.4 us.
#include "route_core.hpp"
#include "w8a8.hpp"

namespace moe {

namespace {

constexpr int kScoredWaves = 4;

// Key of an expert that may be chosen only after all others (masked) and of one that may not be chosen.
constexpr uint32_t kMaskedKey = 0x007FFFFFu;           // ordered_bits(-inf): below every finite value's
constexpr uint32_t kNoKey = 0u;

// The wave's maximum, in every lane.
__device__ __forceinline__ uint32_t wave_max(uint32_t v)
{
    v = row_reduce<true>(v);
    uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xA, 0xF, false);   // row_bcast:15
    v = o > v ? o : v;
    o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xC, 0xF, false);            // row_bcast:31
    v = o > v ? o : v;
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// exp(x) in binary64 for |x| <= 110: x = n ln 2 + r with |r| <= ln 2 / 2, the
// Taylor sum of exp(r) to r^10 / 10! (what is left out is below 0.35^11 / 11!
// = 2e-13 of it), times 2^n.
__device__ __forceinline__ double exp_near(double x)
{
    const double n = __builtin_rint(x * 0x1.71547652b82fep+0);
    double r = __builtin_fma(n, -0x1.62e42fefa39efp-1, x);       // ln 2 in two parts
    r = __builtin_fma(n, -0x1.abc9e3b39803fp-56, r);
    double y = 1.0 / 3628800.0;
    y = __builtin_fma(y, r, 1.0 / 362880.0);
    y = __builtin_fma(y, r, 1.0 / 40320.0);
    y = __builtin_fma(y, r, 1.0 / 5040.0);
    y = __builtin_fma(y, r, 1.0 / 720.0);
    y = __builtin_fma(y, r, 1.0 / 120.0);
    y = __builtin_fma(y, r, 1.0 / 24.0);
    y = __builtin_fma(y, r, 1.0 / 6.0);
    y = __builtin_fma(y, r, 0.5);
    y = __builtin_fma(y, r, 1.0);
    y = __builtin_fma(y, r, 1.0);
    return __builtin_ldexp(y, (int)n);
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

// GROUPS: 0 none; 1 a group is GL = 2^n whole lanes; 2 any.
template <int PL, int GROUPS>
__global__ __launch_bounds__(kScoredWaves * 64) void route_scored_kernel(
    int T, int E, int k, moe_router r, const float *__restrict__ logits, const float *__restrict__ bias, bool vec,
    int32_t *__restrict__ ids, float *__restrict__ w)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int t = blockIdx.x * kScoredWaves + wave;
    const bool there = t < T;
    const float *row = logits + (size_t)(there ? t : T - 1) * E;
    const int e0 = lane * PL;
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
    float score[PL];
    if (r.score == MOE_SCORE_SIGMOID) {
#pragma unroll
        for (int i = 0; i < PL; ++i)
            // past 110 either way it is 0 or 1 in binary32 (a NaN is masked below)
            score[i] = (float)reciprocal(1.0 + exp_near(-(double)__builtin_amdgcn_fmed3f(l[i], -110.0f, 110.0f)));
    } else {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < PL; ++i) {
            const uint32_t o = e0 + i < E && l[i] == l[i] ? ordered_bits(l[i]) : 0u;
            m = o > m ? o : m;
        }
        const float top = from_ordered_bits(wave_max(m));
        double p[PL], sum = 0.0;
#pragma unroll
        for (int i = 0; i < PL; ++i) {
            // below -110 (e^-110 < 2^-150) the share rounds to 0; inf - inf (nothing is left, or an infinite logit) is NaN
            const float d0 = l[i] - top;
            p[i] = exp_near(__builtin_fmax((double)l[i] - (double)top, -110.0));
            p[i] = d0 < -110.0f ? 0.0 : (d0 == d0 ? p[i] : (double)d0);
            sum += e0 + i < E && p[i] == p[i] ? p[i] : 0.0;
        }
#pragma unroll
        for (int d = 1; d < 64; d *= 2)
            sum += __shfl_xor(sum, d);
        const double inv = 1.0 / sum;
#pragma unroll
        for (int i = 0; i < PL; ++i)
            score[i] = (float)(p[i] * inv);
    }
    uint32_t key[PL];
#pragma unroll
    for (int i = 0; i < PL; ++i) {
        const float c = score[i] + b[i];
        const bool masked = !(c == c) || !(l[i] > -__builtin_inff());          // NaN too
        score[i] = masked ? 0.0f : score[i];
        const uint32_t o = masked ? kMaskedKey : ordered_bits(c);
        key[i] = e0 + i < E ? o : kNoKey;
    }
    if constexpr (GROUPS > 0) {
        const int G = r.num_groups, size = E / G;
        uint32_t a = 0, b2 = 0;                        // the two largest keys of a group
        int my_g, gl;                                  // the lane's group; lanes from one group's holder to the next's
        if constexpr (GROUPS == 1) {
#pragma unroll
            for (int i = 0; i < PL; ++i)
                merge_top2(a, b2, key[i], 0u);
            gl = size / PL;
            my_g = lane / gl;
#define MOE_TOP2_STEP(n, ctrl)                                                                             \
            if (gl > n)                                                                                    \
                merge_top2(a, b2, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)a, ctrl, 0xF, 0xF, false), \
                           (uint32_t)__builtin_amdgcn_update_dpp(0, (int)b2, ctrl, 0xF, 0xF, false));
            MOE_TOP2_STEP(1, 0xB1)     // quad_perm [1,0,3,2]
            MOE_TOP2_STEP(2, 0x4E)     // quad_perm [2,3,0,1]
            MOE_TOP2_STEP(4, 0x141)    // row_half_mirror
            MOE_TOP2_STEP(8, 0x140)    // row_mirror
#undef MOE_TOP2_STEP
            if (gl > 16)
                merge_top2(a, b2, __shfl_xor(a, 16), __shfl_xor(b2, 16));
            if (gl > 32)
                merge_top2(a, b2, __shfl_xor(a, 32), __shfl_xor(b2, 32));
        } else {
            __shared__ uint32_t s_key[kScoredWaves][PL * 64];
#pragma unroll
            for (int i = 0; i < PL; ++i)
                s_key[wave][e0 + i] = key[i];
            __syncthreads();
            if (lane < G)                              // lane g holds group g
                for (int i = 0; i < size; ++i)
                    merge_top2(a, b2, s_key[wave][lane * size + i], 0u);
            gl = 1;
            my_g = lane;
        }
        const uint32_t gk = r.group_top == 2 ? ordered_bits(from_ordered_bits(a) + from_ordered_bits(b2)) : a;
        int ahead = 0;                                 // groups that come before this one: earlier ones with as large a
        for (int g = 0; g < G; ++g) {                  // key, later ones with a larger one (no key is 2^32 - 1)
            const uint32_t o = (uint32_t)__builtin_amdgcn_readlane((int)gk, g * gl);
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
    if constexpr (PL <= 4) {
        // A lane's keys in descending order (neighbours change places only where the second is larger, so equal ones
        // stay in index order), which expert each one was in the bytes of `which`: its largest is then always the first.
        int at[PL];
#pragma unroll
        for (int i = 0; i < PL; ++i)
            at[i] = i;
#pragma unroll
        for (int round = 0; round < PL; ++round)
#pragma unroll
            for (int i = round & 1; i + 1 < PL; i += 2) {
                const uint32_t a = key[i], c = key[i + 1];
                const int ia = at[i], ic = at[i + 1];
                const bool swap = c > a;
                key[i] = swap ? c : a;
                key[i + 1] = swap ? a : c;
                at[i] = swap ? ic : ia;
                at[i + 1] = swap ? ia : ic;
            }
        uint32_t which = 0;
#pragma unroll
        for (int i = 0; i < PL; ++i)
            which |= (uint32_t)at[i] << (8 * i);
        for (int j = 0; j < k; ++j) {
            const uint32_t m = wave_max(key[0]);
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
            const uint32_t m = wave_max(bv);
            const int owner = __builtin_ctzll(__ballot(bv == m));
            const int e = __builtin_amdgcn_readlane(e0 + at, owner);
            my_e = lane == j ? e : my_e;
            if (lane == owner)
#pragma unroll
                for (int i = 0; i < PL; ++i)
                    key[i] = i == at ? kNoKey : key[i];
        }
    }
    float my_s = 0.0f;                                 // lane j < k: slot j's score, from the lane that has it
#pragma unroll
    for (int i = 0; i < PL; ++i) {
        const float v = __int_as_float(__builtin_amdgcn_ds_bpermute(my_e / PL * 4, __float_as_int(score[i])));
        my_s = my_e % PL == i ? v : my_s;
    }
    my_s = lane < k ? my_s : 0.0f;
    float z = my_s;                                    // lanes >= k hold 0
#define MOE_DPP_ADD(ctrl) z += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(z), ctrl, 0xF, 0xF, false));
    MOE_DPP_ADD(0xB1)      // quad_perm [1,0,3,2]
    MOE_DPP_ADD(0x4E)      // quad_perm [2,3,0,1]
    MOE_DPP_ADD(0x141)     // row_half_mirror
    MOE_DPP_ADD(0x140)     // row_mirror
#undef MOE_DPP_ADD
    if (there && lane < k) {
        const float wt = r.renormalize ? (z > 0.0f ? my_s / z : 0.0f) : my_s;
        ids[(size_t)t * k + lane] = my_e;
        w[(size_t)t * k + lane] = wt * r.scale;
    }
}

template <int PL>
void launch_scored(int T, int E, int k, const moe_router &r, const float *logits, const float *bias, int32_t *ids,
                   float *w, hipStream_t st)
{
    constexpr size_t W = PL < 4 ? PL : 4;              // values of a vector load
    const bool vec = E % PL == 0 && reinterpret_cast<uintptr_t>(logits) % (4 * W) == 0 &&
                     reinterpret_cast<uintptr_t>(bias) % (4 * W) == 0;
    const int size = E / r.num_groups, gl = size / PL;
    const dim3 grid((T + kScoredWaves - 1) / kScoredWaves), block(kScoredWaves * 64);
    if (r.num_groups == 1)
        hipLaunchKernelGGL((route_scored_kernel<PL, 0>), grid, block, 0, st, T, E, k, r, logits, bias, vec, ids, w);
    else if (size % PL == 0 && (gl & (gl - 1)) == 0)
        hipLaunchKernelGGL((route_scored_kernel<PL, 1>), grid, block, 0, st, T, E, k, r, logits, bias, vec, ids, w);
    else
        hipLaunchKernelGGL((route_scored_kernel<PL, 2>), grid, block, 0, st, T, E, k, r, logits, bias, vec, ids, w);
}

}  // namespace

hipError_t launch_route_scored(const moe_shape &sh, const moe_router &r, const float *logits, const float *bias,
                               int32_t *ids, float *w, hipStream_t st)
{
    const int T = sh.num_tokens, E = sh.num_experts, k = sh.top_k;
    if (E <= 64)
        launch_scored<1>(T, E, k, r, logits, bias, ids, w, st);
    else if (E <= 128)
        launch_scored<2>(T, E, k, r, logits, bias, ids, w, st);
    else if (E <= 256)
        launch_scored<4>(T, E, k, r, logits, bias, ids, w, st);
    else if (E <= 512)
        launch_scored<8>(T, E, k, r, logits, bias, ids, w, st);
    else
        launch_scored<kMaxExperts / 64>(T, E, k, r, logits, bias, ids, w, st);
    return hipGetLastError();
}

}  // namespace moe
