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
// their sum are formed in binary64, whose error (about 2^-52) changes that
// rounding for about one score in 2^27. Everything after it is a binary32
// comparison or one addition.
//
// One wave holds a token, lane q its experts q, q + 64, ...; k rounds take the
// largest remaining key (the order-preserving integer image of c) by DPP and
// retire it.
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

template <int PL>
__global__ __launch_bounds__(kScoredWaves * 64) void route_scored_kernel(
    int T, int E, int k, moe_router r, const float *__restrict__ logits, const float *__restrict__ bias,
    int32_t *__restrict__ ids, float *__restrict__ w)
{
    __shared__ uint32_t s_key[kScoredWaves][PL * 64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int t = blockIdx.x * kScoredWaves + wave;
    const bool there = t < T;
    const float *row = logits + (size_t)(there ? t : T - 1) * E;
    float l[PL], b[PL];
#pragma unroll
    for (int i = 0; i < PL; ++i) {
        const int e = lane + 64 * i;
        l[i] = row[e < E ? e : E - 1];
        b[i] = bias ? bias[e < E ? e : E - 1] : 0.0f;
    }
    float score[PL];
    if (r.score == MOE_SCORE_SIGMOID) {
#pragma unroll
        for (int i = 0; i < PL; ++i)
            score[i] = (float)(1.0 / (1.0 + exp(-(double)l[i])));
    } else {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < PL; ++i) {
            const uint32_t o = lane + 64 * i < E && l[i] == l[i] ? ordered_bits(l[i]) : 0u;
            m = o > m ? o : m;
        }
        const double top = (double)from_ordered_bits(wave_max(m));
        double p[PL], sum = 0.0;
#pragma unroll
        for (int i = 0; i < PL; ++i) {
            p[i] = exp((double)l[i] - top);
            sum += lane + 64 * i < E && p[i] == p[i] ? p[i] : 0.0;
        }
#pragma unroll
        for (int d = 1; d < 64; d *= 2)
            sum += __shfl_xor(sum, d);
#pragma unroll
        for (int i = 0; i < PL; ++i)
            score[i] = (float)(p[i] / sum);
    }
    uint32_t key[PL];
#pragma unroll
    for (int i = 0; i < PL; ++i) {
        const float c = score[i] + b[i];
        const bool masked = !(c == c) || l[i] == -__builtin_inff();
        score[i] = masked ? 0.0f : score[i];
        const uint32_t o = masked ? kMaskedKey : ordered_bits(c);
        key[i] = lane + 64 * i < E ? o : kNoKey;
    }
    if (r.num_groups > 1) {
        // lane g scores group g, then counts the groups ahead of it
        const int G = r.num_groups, size = E / G;
#pragma unroll
        for (int i = 0; i < PL; ++i)
            s_key[wave][lane + 64 * i] = key[i];
        __syncthreads();
        uint32_t a = 0, b2 = 0;                        // the two largest keys of the group
        if (lane < G)
            for (int i = 0; i < size; ++i) {
                const uint32_t v = s_key[wave][lane * size + i];
                b2 = v > a ? a : (v > b2 ? v : b2);
                a = v > a ? v : a;
            }
        uint32_t gk = a;
        if (r.group_top == 2)
            gk = ordered_bits(from_ordered_bits(a) + from_ordered_bits(b2));
        int ahead = 0;
        for (int g = 0; g < G; ++g) {
            const uint32_t o = (uint32_t)__builtin_amdgcn_readlane((int)gk, g);
            ahead += o > gk || (o == gk && g < lane);
        }
        const uint64_t keep = __ballot(lane < G && ahead < r.topk_groups);
#pragma unroll
        for (int i = 0; i < PL; ++i) {
            const int e = lane + 64 * i;
            if (e >= E || !(keep >> (e / size) & 1))
                key[i] = kNoKey;
        }
    }
    int my_e = 0;
    float my_s = 0.0f;
    for (int j = 0; j < k; ++j) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < PL; ++i)
            m = key[i] > m ? key[i] : m;
        m = wave_max(m);
        int e = 0;
#pragma unroll
        for (int i = PL - 1; i >= 0; --i) {
            const uint64_t at = __ballot(key[i] == m);
            if (at)
                e = 64 * i + __builtin_ctzll(at);
        }
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < PL; ++i)
            if (lane + 64 * i == e) {
                s = score[i];
                key[i] = kNoKey;
            }
        s = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(s), e & 63));
        if (lane == j) {
            my_e = e;
            my_s = s;
        }
    }
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

}  // namespace

hipError_t launch_route_scored(const moe_shape &sh, const moe_router &r, const float *logits, const float *bias,
                               int32_t *ids, float *w, hipStream_t st)
{
    const int T = sh.num_tokens, E = sh.num_experts, k = sh.top_k;
    const dim3 grid((T + kScoredWaves - 1) / kScoredWaves), block(kScoredWaves * 64);
    if (E <= 64)
        hipLaunchKernelGGL((route_scored_kernel<1>), grid, block, 0, st, T, E, k, r, logits, bias, ids, w);
    else if (E <= 128)
        hipLaunchKernelGGL((route_scored_kernel<2>), grid, block, 0, st, T, E, k, r, logits, bias, ids, w);
    else if (E <= 256)
        hipLaunchKernelGGL((route_scored_kernel<4>), grid, block, 0, st, T, E, k, r, logits, bias, ids, w);
    else if (E <= 512)
        hipLaunchKernelGGL((route_scored_kernel<8>), grid, block, 0, st, T, E, k, r, logits, bias, ids, w);
    else
        hipLaunchKernelGGL((route_scored_kernel<kMaxExperts / 64>), grid, block, 0, st, T, E, k, r, logits, bias, ids, w);
    return hipGetLastError();
}

}  // namespace moe
