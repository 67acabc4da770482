// api_w8a8.hip -- C entry points of the W8A8 operators: the scored router, the
// RMS norm, the int8 quantizer, the dense and grouped products and the layer.
// Conventions as in api.hip: validation before any launch, nothing allocated,
// no synchronisation, no device reads on the host.
#include "common.hpp"
#include "w8a8.hpp"

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

// The layer's limits with one scale per row (group_size 0) and plain codes.
moe_status check_shape_w8(const moe_shape *sh, moe_shape *s)
{
    if (!sh)
        return MOE_ERR_NULL;
    if (sh->group_size != 0 || sh->weight_layout != MOE_WEIGHTS_PLAIN)
        return MOE_ERR_UNSUPPORTED;
    *s = *sh;
    s->group_size = kGroup;
    return moe_w4a16_check_shape(s);
}

struct Workspace {
    int32_t *counts, *offsets, *perm, *inv_perm, *part;
    uint16_t *h, *y;
    int8_t *hq;
    float *hs;
    size_t bytes;
};

Workspace carve(const moe_shape &sh, void *base)
{
    const size_t S = (size_t)sh.num_tokens * sh.top_k, E = (size_t)sh.num_local_experts;
    char *p = static_cast<char *>(base);
    size_t off = 0;
    auto take = [&](size_t bytes) {
        char *r = p ? p + off : nullptr;
        off += align_up(bytes);
        return r;
    };
    Workspace ws{};
    ws.counts = reinterpret_cast<int32_t *>(take(E * 4));
    ws.offsets = reinterpret_cast<int32_t *>(take((E + 1) * 4));
    ws.perm = reinterpret_cast<int32_t *>(take(S * 4));
    ws.inv_perm = reinterpret_cast<int32_t *>(take(S * 4));
    ws.part = reinterpret_cast<int32_t *>(take(permute_workspace_bytes(sh)));
    ws.h = reinterpret_cast<uint16_t *>(take(S * sh.inter * 2));
    ws.y = reinterpret_cast<uint16_t *>(take(S * sh.hidden * 2));
    ws.hq = reinterpret_cast<int8_t *>(take(S * sh.inter));
    ws.hs = reinterpret_cast<float *>(take(S * 4));
    ws.bytes = off;
    return ws;
}

W8GemmLaunch grouped_args(const moe_shape &sh, moe_gemm_kind kind)
{
    W8GemmLaunch g{};
    g.kind = kind;
    g.top_k = sh.top_k;
    g.num_experts = sh.num_local_experts;
    g.max_rows = sh.num_tokens * sh.top_k;
    g.expected_rows = (int)((long long)g.max_rows * sh.num_local_experts / sh.num_experts);
    g.K = kind == MOE_GEMM_W2 ? sh.inter : sh.hidden;
    g.N = kind == MOE_GEMM_W2 ? sh.hidden : 2 * sh.inter;
    return g;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_route_scored(const moe_shape *shape, const moe_router *router, const float *logits, const float *bias,
                            int32_t *topk_ids, float *topk_w, void *stream)
{
    moe_status st = moe_w4a16_check_shape(shape);
    if (st != MOE_OK)
        return st;
    if (!router)
        return MOE_ERR_NULL;
    const moe_router &r = *router;
    if (r.score != MOE_SCORE_SOFTMAX && r.score != MOE_SCORE_SIGMOID)
        return MOE_ERR_UNSUPPORTED;
    if (r.num_groups < 1 || shape->num_experts % r.num_groups || r.topk_groups < 1 || r.topk_groups > r.num_groups)
        return MOE_ERR_SHAPE;
    if (r.num_groups > kMaxRouteGroups || (r.group_top != 1 && r.group_top != 2))
        return MOE_ERR_UNSUPPORTED;
    const int size = shape->num_experts / r.num_groups;
    if (r.group_top > size || shape->top_k > r.topk_groups * size)
        return MOE_ERR_SHAPE;
    if (shape->num_tokens == 0)
        return MOE_OK;
    if (!logits || !topk_ids || !topk_w)
        return MOE_ERR_NULL;
    if (!aligned(logits, 4) || !aligned(bias, 4) || !aligned(topk_ids, 4) || !aligned(topk_w, 4))
        return MOE_ERR_ALIGN;
    return from_hip(launch_route_scored(*shape, r, logits, bias, topk_ids, topk_w, static_cast<hipStream_t>(stream)));
}

moe_status moe_rms_norm(int64_t rows, int32_t K, const uint16_t *x, const uint16_t *residual, const uint16_t *weight,
                        float eps, uint16_t *sum, uint16_t *y, int8_t *q, float *q_scale, void *stream)
{
    if (rows < 0 || K < 8 || K % 8 != 0 || K > kMaxNormDim || !(eps >= 0.0f))
        return MOE_ERR_SHAPE;
    if (!norm_rows_fit(rows, K))
        return MOE_ERR_UNSUPPORTED;
    if (rows == 0)
        return MOE_OK;
    if (!x || !weight || (!y && !q) || (residual == nullptr) != (sum == nullptr) || (q == nullptr) != (q_scale == nullptr))
        return MOE_ERR_NULL;
    if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(sum, 16) || !aligned(y, 16) ||
        !aligned(q, 16) || !aligned(q_scale, 4))
        return MOE_ERR_ALIGN;
    // an output may stand in place of x or of the residual (the whole array), and nowhere else over another array
    const size_t nb = (size_t)rows * K * 2, nq = (size_t)rows * K, ns = (size_t)rows * 4, nw = (size_t)K * 2;
    const struct { const void *p; size_t n; bool in_place; } out[] = {
        {sum, nb, true}, {y, nb, true}, {q, nq, false}, {q_scale, ns, false}};
    for (int i = 0; i < 4; ++i) {
        if (overlap(out[i].p, out[i].n, weight, nw))
            return MOE_ERR_UNSUPPORTED;
        for (const void *in : {static_cast<const void *>(x), static_cast<const void *>(residual)})
            if (overlap(out[i].p, out[i].n, in, nb) && !(out[i].in_place && out[i].p == in))
                return MOE_ERR_UNSUPPORTED;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i].p, out[i].n, out[j].p, out[j].n))
                return MOE_ERR_UNSUPPORTED;
    }
    return from_hip(launch_norm(NormLaunch{rows, K, x, residual, weight, eps, sum, y, q, q_scale, nullptr},
                                static_cast<hipStream_t>(stream)));
}

moe_status moe_int8_quantize(int64_t rows, int32_t K, const uint16_t *x, int8_t *q, float *q_scale, void *stream)
{
    if (rows < 0 || K < 8 || K % 8 != 0 || K > kMaxNormDim)
        return MOE_ERR_SHAPE;
    if (!norm_rows_fit(rows, K))
        return MOE_ERR_UNSUPPORTED;
    if (rows == 0)
        return MOE_OK;
    if (!x || !q || !q_scale)
        return MOE_ERR_NULL;
    if (!aligned(x, 16) || !aligned(q, 16) || !aligned(q_scale, 4))
        return MOE_ERR_ALIGN;
    const size_t nb = (size_t)rows * K * 2, nq = (size_t)rows * K, ns = (size_t)rows * 4;
    if (overlap(x, nb, q, nq) || overlap(x, nb, q_scale, ns) || overlap(q, nq, q_scale, ns))
        return MOE_ERR_UNSUPPORTED;
    return from_hip(launch_norm(NormLaunch{rows, K, x, nullptr, nullptr, 0.0f, nullptr, nullptr, q, q_scale, nullptr},
                                static_cast<hipStream_t>(stream)));
}

moe_status moe_w8a8_dense_gemm(int32_t M, int32_t N, int32_t K, const int8_t *a, const float *a_scale, const int8_t *wq,
                               const float *w_scale, void *c, moe_dtype c_dtype, void *stream)
{
    if (M < 0 || N < 16 || N % 16 != 0 || K < 128 || K % 128 != 0 || N > kMaxDenseCols || K > kMaxNormDim)
        return MOE_ERR_SHAPE;
    if ((size_t)N * K >= (size_t(1) << 31) || (size_t)M * K >= (size_t(1) << 31) ||
        (size_t)M * N >= (size_t(1) << 36))
        return MOE_ERR_UNSUPPORTED;
    if (c_dtype != MOE_BF16 && c_dtype != MOE_F32)
        return MOE_ERR_UNSUPPORTED;
    if (M == 0)
        return MOE_OK;
    if (!a || !a_scale || !wq || !w_scale || !c)
        return MOE_ERR_NULL;
    if (!aligned(a, 16) || !aligned(wq, 16) || !aligned(c, 16) || !aligned(a_scale, 4) || !aligned(w_scale, 16))
        return MOE_ERR_ALIGN;
    W8GemmLaunch g{};
    g.kind = MOE_GEMM_W2;
    g.top_k = 1;
    g.num_experts = 1;
    g.max_rows = g.expected_rows = M;
    g.K = K;
    g.N = N;
    g.a = a;
    g.as = a_scale;
    g.wq = wq;
    g.ws = w_scale;
    g.c = c;
    g.c_f32 = c_dtype == MOE_F32;
    return from_hip(launch_w8_gemm(g, static_cast<hipStream_t>(stream)));
}

moe_status moe_grouped_gemm_w8a8(const moe_shape *shape, moe_gemm_kind kind, const int8_t *a, const float *a_scale,
                                 const int32_t *a_row_index, const int32_t *offsets, const int8_t *wq,
                                 const float *w_scale, void *c, moe_dtype c_dtype, void *stream)
{
    moe_shape sh;
    moe_status st = check_shape_w8(shape, &sh);
    if (st != MOE_OK)
        return st;
    if (kind != MOE_GEMM_W13_SWIGLU && kind != MOE_GEMM_W2 && kind != MOE_GEMM_W13_RAW)
        return MOE_ERR_UNSUPPORTED;
    if ((c_dtype != MOE_BF16 && c_dtype != MOE_F32) || (kind == MOE_GEMM_W13_SWIGLU && c_dtype != MOE_BF16))
        return MOE_ERR_UNSUPPORTED;
    if (sh.num_tokens == 0)
        return MOE_OK;
    if (!a || !a_scale || !offsets || !wq || !w_scale || !c)
        return MOE_ERR_NULL;
    if (!aligned(a, 16) || !aligned(wq, 16) || !aligned(c, 16) || !aligned(a_scale, 4) || !aligned(w_scale, 16) ||
        !aligned(offsets, 4) || !aligned(a_row_index, 4))
        return MOE_ERR_ALIGN;
    W8GemmLaunch g = grouped_args(sh, kind);
    g.a = a;
    g.as = a_scale;
    g.a_row_index = a_row_index;
    g.offsets = offsets;
    g.wq = wq;
    g.ws = w_scale;
    g.c = c;
    g.c_f32 = c_dtype == MOE_F32;
    return from_hip(launch_w8_gemm(g, static_cast<hipStream_t>(stream)));
}

size_t moe_w8a8_workspace_size(const moe_shape *shape)
{
    moe_shape sh;
    if (check_shape_w8(shape, &sh) != MOE_OK)
        return 0;
    return carve(sh, nullptr).bytes;
}

moe_status moe_w8a8_forward(const moe_shape *shape, const int8_t *x, const float *x_scale, const int32_t *topk_ids,
                            const float *topk_w, const int8_t *w13_q, const float *w13_s, const int8_t *w2_q,
                            const float *w2_s, uint16_t *out, void *workspace, size_t workspace_bytes, void *stream)
{
    moe_shape sh;
    moe_status st = check_shape_w8(shape, &sh);
    if (st != MOE_OK)
        return st;
    if (sh.num_tokens == 0)
        return MOE_OK;
    if (!x || !x_scale || !topk_ids || !topk_w || !w13_q || !w13_s || !w2_q || !w2_s || !out || !workspace)
        return MOE_ERR_NULL;
    if (!aligned(x, 16) || !aligned(x_scale, 4) || !aligned(topk_ids, 4) || !aligned(topk_w, 4) || !aligned(w13_q, 16) ||
        !aligned(w13_s, 16) || !aligned(w2_q, 16) || !aligned(w2_s, 16) || !aligned(out, 16) || !aligned(workspace, kAlign))
        return MOE_ERR_ALIGN;
    const Workspace ws = carve(sh, workspace);
    if (workspace_bytes < ws.bytes)
        return MOE_ERR_WORKSPACE;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const int S = sh.num_tokens * sh.top_k;
    hipError_t e = launch_permute(sh, topk_ids, ws.counts, ws.offsets, ws.perm, ws.inv_perm, s, 0, ws.part);
    if (e == hipSuccess) {
        W8GemmLaunch g = grouped_args(sh, MOE_GEMM_W13_SWIGLU);
        g.a = x;
        g.as = x_scale;
        g.a_row_index = ws.perm;
        g.offsets = ws.offsets;
        g.wq = w13_q;
        g.ws = w13_s;
        g.c = ws.h;
        e = launch_w8_gemm(g, s);
    }
    W8GemmLaunch g = grouped_args(sh, MOE_GEMM_W2);
    g.offsets = ws.offsets;
    g.wq = w2_q;
    g.ws = w2_s;
    g.c = ws.y;
    if (quantizes_rows(g)) {
        g.a_bf16 = ws.h;
    } else {
        g.a = ws.hq;
        g.as = ws.hs;
        // h requantized: the routed rows only, counted on the device
        if (e == hipSuccess)
            e = launch_norm(NormLaunch{S, sh.inter, ws.h, nullptr, nullptr, 0.0f, nullptr, nullptr, ws.hq, ws.hs,
                                       ws.offsets + sh.num_local_experts}, s);
    }
    if (e == hipSuccess)
        e = launch_w8_gemm(g, s);
    if (e == hipSuccess)
        e = launch_finalize(sh, ws.y, false, topk_w, ws.inv_perm, out, false, s);
    return from_hip(e);
}

}  // extern "C"
