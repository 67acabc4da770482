"""The W8A8 products and layer against their definition in 64 bits.

Error bounds (u = 2^-24): the integer sum is exact; its conversion and two products with scales are three half steps,
so an fp32 result is within 3 u (4 u with second-order terms) relative, a bf16 one 2^-8 more. SwiGLU: gate and up are
off by 3 u each; the sigmoid's argument by 2 u relative, so exp(-g) by 2 |g| u and a few u for exp2, the sum, the
reciprocal and the products: with |g| < 90 (beyond it the result is below any bf16 step of the others) less than
(3 + 3 |g| + 2 |g| + 16) u < 2^-15.
"""
import numpy as np
import pytest
import torch

from helpers import assert_layer_close, say, to_np_u16

pytestmark = pytest.mark.gpu

F32_REL, BF16_REL, SWIGLU_REL = 4 * 2.0 ** -24, 2.0 ** -8 + 2.0 ** -20, 2.0 ** -8 + 2.0 ** -14


def codes(g, *shape):
    return torch.randint(-128, 128, shape, generator=g, device="cuda", dtype=torch.int8)


def scales(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda") * 0.015 + 0.005


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def near(got, want, rel):
    return bool(((got.double() - want).abs() <= want.abs() * rel + 1e-30).all())


def dense(a, s, w, ws):
    """Exact in 64 bits (every sum is below 2^53)."""
    return (a.double() @ w.double().t()) * s.double()[:, None] * ws.double()


def swiglu(c):
    n = c.shape[-1] // 2
    return c[..., :n] / (1 + torch.exp(-c[..., :n])) * c[..., n:]


DENSE = [(1, 16, 128), (1, 2064, 768), (3, 4096, 256), (15, 48, 1280), (16, 128, 2048), (17, 272, 128), (31, 4096, 4096),
         (33, 400, 896), (64, 256, 512), (65, 1040, 640), (100, 128, 7168), (129, 2064, 768), (256, 256, 128),
         (257, 512, 384), (333, 2064, 768), (512, 768, 2048), (700, 1552, 1024), (1500, 2048, 256), (2049, 272, 1152), (4100, 4112, 256),
         (3000, 4112, 384), (1, 4096, 14336), (30, 14336, 1152), (60, 16400, 256), (12, 14336, 640)]


@pytest.mark.parametrize("M,N,K", DENSE)
def test_dense(M, N, K):
    from w4a16_grouped_gemm_amd import ops
    say(f"dense_gemm_w8a8 M={M} N={N} K={K}")
    g = gen(M * 31 + N + K)
    a, s, w, ws = codes(g, M, K), scales(g, M), codes(g, N, K), scales(g, N)
    want = dense(a, s, w, ws)
    guard = torch.full((M + 2, N), 7.0, device="cuda")            # rows behind the last stay as they were
    out = ops.dense_gemm_w8a8(a, s, w, ws, out=guard[:M])
    assert near(out, want, F32_REL) and bool((guard[M:] == 7).all())
    assert near(ops.dense_gemm_w8a8(a, s, w, ws), want, BF16_REL)


def test_dense_extreme_codes():
    """All codes -128 at the longest K: sums of 2^30, exact."""
    from w4a16_grouped_gemm_amd import ops
    for M in (3, 300):
        a = torch.full((M, 65536), -128, dtype=torch.int8, device="cuda")
        w = torch.full((272, 65536), -128, dtype=torch.int8, device="cuda")
        w[5] = 127
        out = ops.dense_gemm_w8a8(a, torch.ones(M, device="cuda"), w, torch.ones(272, device="cuda"), out_dtype=torch.float32)
        assert bool((out[:, :5] == 2.0 ** 30).all()) and bool((out[:, 5] == -128.0 * 127 * 65536).all())
        assert bool((out[:, 6:] == 2.0 ** 30).all())


def test_dense_nan_scale_stays_in_its_row():
    from w4a16_grouped_gemm_amd import ops
    g = gen(1)
    for M in (5, 300):
        a, s, w, ws = codes(g, M, 256), scales(g, M), codes(g, 272, 256), scales(g, 272)
        s[2] = float("nan")
        out = ops.dense_gemm_w8a8(a, s, w, ws)
        assert bool(out[2].isnan().all())
        keep = torch.arange(M, device="cuda") != 2
        assert near(out[keep], dense(a, s, w, ws)[keep], BF16_REL)


def routing(T, E, k, g, mode):
    if mode == "uniform":
        return torch.rand(T, E, generator=g, device="cuda").argsort(-1)[:, :k].to(torch.int32).contiguous()
    if mode == "one":                                             # every token to the same experts
        return torch.arange(E - k, E, device="cuda", dtype=torch.int32).repeat(T, 1)
    p = torch.arange(1, E + 1, device="cuda", dtype=torch.float32).pow(-1.1).log()
    u = torch.rand(T, E, generator=g, device="cuda").clamp_(1e-6, 1 - 1e-6)
    return (p - torch.log(-torch.log(u))).argsort(-1, descending=True)[:, :k].to(torch.int32).contiguous()


GROUPED = [  # T, E, local from, local, k, H, I, routing
    (1, 8, 0, 8, 2, 256, 512, "uniform"), (1, 128, 0, 128, 8, 2048, 768, "uniform"), (5, 8, 2, 3, 3, 128, 128, "uniform"),
    (16, 128, 0, 128, 8, 2048, 768, "uniform"), (33, 60, 15, 30, 4, 384, 256, "zipf"), (40, 4, 0, 4, 1, 640, 384, "one"),
    (64, 16, 0, 16, 2, 256, 128, "zipf"), (130, 8, 0, 8, 2, 512, 256, "one"), (300, 16, 0, 16, 4, 1024, 384, "zipf"),
    (513, 32, 8, 16, 8, 256, 640, "uniform"), (700, 3, 0, 3, 3, 384, 1024, "uniform"), (2048, 64, 0, 64, 2, 256, 128, "zipf"),
    (50, 16, 12, 4, 2, 256, 256, "one"), (50, 16, 0, 4, 2, 256, 256, "one"), (1024, 64, 0, 64, 8, 256, 768, "uniform"),
    (600, 64, 0, 64, 8, 1792, 256, "zipf"), (4096, 4, 0, 4, 2, 2048, 1024, "uniform"), (200, 300, 0, 300, 3, 256, 256, "zipf"),
    (3, 1024, 0, 1024, 16, 256, 128, "uniform")]


@pytest.mark.parametrize("T,E,begin,L,k,H,I,mode", GROUPED)
def test_grouped(T, E, begin, L, k, H, I, mode):
    from w4a16_grouped_gemm_amd import ops
    say(f"grouped_gemm_w8a8 T={T} E={E} local {begin}+{L} k={k} H={H} I={I} {mode}")
    g = gen(T + E * 3 + H)
    ids = routing(T, E, k, g, mode)
    _, offsets, perm, _, _ = ops.permute(ids, L, num_experts=E, expert_begin=begin)
    off = offsets.tolist()
    R = off[-1]
    x, xs, w13, s13 = codes(g, T, H), scales(g, T), codes(g, L, 2 * I, H), scales(g, L, 2 * I)
    h, hs, w2, s2 = codes(g, T * k, I), scales(g, T * k), codes(g, L, H, I), scales(g, L, H)
    token = perm.long() // k
    raw = torch.zeros(T * k, 2 * I, dtype=torch.float64, device="cuda")
    down = torch.zeros(T * k, H, dtype=torch.float64, device="cuda")
    for e in range(L):
        r = slice(off[e], off[e + 1])
        raw[r] = dense(x[token[r]], xs[token[r]], w13[e], s13[e])
        down[r] = dense(h[r], hs[r], w2[e], s2[e])
    kw = dict(num_tokens=T, top_k=k, num_experts=E)

    def run(kind, a, s, w, ws, cols, dtype, index):
        out = torch.full((T * k, cols), 7.0, dtype=dtype, device="cuda")
        ops.grouped_gemm_w8a8(kind, a, s, offsets, w, ws, a_row_index=index, out=out, **kw)
        assert bool((out[R:] == 7).all())                         # rows behind the last sequence
        return out[:R]

    B, F = torch.bfloat16, torch.float32
    assert near(run(ops.W13_RAW, x, xs, w13, s13, 2 * I, F, perm), raw[:R], F32_REL)
    assert near(run(ops.W13_RAW, x, xs, w13, s13, 2 * I, B, perm), raw[:R], BF16_REL)
    assert near(run(ops.W13_SWIGLU, x, xs, w13, s13, I, B, perm), swiglu(raw[:R]), SWIGLU_REL)
    assert near(run(ops.W2, h, hs, w2, s2, H, F, None), down[:R], F32_REL)
    assert near(run(ops.W2, h, hs, w2, s2, H, B, None), down[:R], BF16_REL)
    # rows in permuted order give the gathered rows' results
    xp, xsp = x[token.clamp(min=0)].contiguous(), xs[token.clamp(min=0)].contiguous()
    assert torch.equal(run(ops.W13_SWIGLU, xp, xsp, w13, s13, I, B, None),
                       run(ops.W13_SWIGLU, x, xs, w13, s13, I, B, perm))


@pytest.mark.parametrize("H,I", [(128, 384), (640, 128), (640, 256), (640, 384), (768, 512), (896, 640), (1024, 768), (1920, 896),
                                 (2048, 1024), (2176, 1920), (2304, 2048), (2432, 2176), (2560, 2304), (4096, 2432)])
def test_grouped_few_rows(H, I):
    """A few rows of each of 64 experts: every length of what is left of K after whole rounds of the weight stream."""
    test_grouped(64, 64, 0, 64, 2, H, I, "uniform")
    test_grouped(70, 64, 0, 64, 3, H, I, "zipf")


@pytest.mark.parametrize("M", [1, 9, 16])
@pytest.mark.parametrize("N", [14336, 12304])
@pytest.mark.parametrize("K", [128, 256, 384, 512, 640, 1152, 2432])
def test_dense_few_rows(M, N, K):
    test_dense(M, N, K)


def layer_inputs(T, E, begin, L, k, H, I, mode, seed):
    g = gen(seed)
    ids = routing(T, E, k, g, mode)
    w = torch.rand(T, k, generator=g, device="cuda") + 0.1
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    w13, s13 = codes(g, L, 2 * I, H), scales(g, L, 2 * I) / H ** 0.5
    w2, s2 = codes(g, L, H, I), scales(g, L, H) / I ** 0.5
    return x, ids, w, w13, s13, w2, s2


def quantized(v):
    top = v.abs().amax(-1, keepdim=True).clamp(min=1e-300)
    return (127 * v / top).round() * (top / 127)


def layer_reference(xq, xs, ids, w, w13, s13, w2, s2, begin):
    T, k = ids.shape
    v = xq.double() * xs.double()[:, None]
    out = torch.zeros(T, w2.shape[1], dtype=torch.float64, device="cuda")
    for e in range(w13.shape[0]):
        for j in range(k):
            t = (ids[:, j] == begin + e).nonzero().flatten()
            if t.numel():
                h = swiglu(v[t] @ (w13[e].double() * s13[e].double()[:, None]).t()).bfloat16().double()
                y = quantized(h) @ (w2[e].double() * s2[e].double()[:, None]).t()
                out[t] += w[t, j].double()[:, None] * y.bfloat16().double()
    return out


LAYERS = GROUPED[:11] + [(1, 128, 96, 32, 8, 256, 256, "one"), (385, 32, 0, 32, 4, 256, 256, "uniform")]


@pytest.mark.parametrize("T,E,begin,L,k,H,I,mode", LAYERS)
def test_layer(T, E, begin, L, k, H, I, mode):
    """Equal to the entry points it is made of, and near the definition."""
    from w4a16_grouped_gemm_amd import ops
    say(f"moe_w8a8_forward T={T} E={E} local {begin}+{L} k={k} H={H} I={I} {mode}")
    x, ids, w, w13, s13, w2, s2 = layer_inputs(T, E, begin, L, k, H, I, mode, T + H)
    xq, xs = ops.int8_quantize(x)
    out = ops.moe_w8a8_forward(xq, xs, ids, w, w13, s13, w2, s2, num_experts=E, expert_begin=begin)
    _, offsets, perm, inv, _ = ops.permute(ids, L, num_experts=E, expert_begin=begin)
    R = int(offsets[-1])
    kw = dict(num_tokens=T, top_k=k, num_experts=E)
    h = ops.grouped_gemm_w8a8(ops.W13_SWIGLU, xq, xs, offsets, w13, s13, a_row_index=perm, **kw)
    h[R:] = 0
    hq, hs = ops.int8_quantize(h)
    y = ops.grouped_gemm_w8a8(ops.W2, hq, hs, offsets, w2, s2, **kw)
    y[R:] = 0
    assert torch.equal(out, ops.finalize(y, w, inv))
    want = layer_reference(xq, xs, ids, w, w13, s13, w2, s2, begin).bfloat16()
    assert_layer_close(to_np_u16(out), to_np_u16(want), "layer")


FUSED = [  # few rows of each expert, I below 2048: the down product quantizes its rows
    (1, 128, 0, 128, 8, 2048, 768, "uniform"), (16, 64, 0, 64, 6, 2048, 1408, "uniform"), (40, 64, 0, 64, 4, 2048, 1152, "one"),
    (3, 64, 0, 64, 8, 4096, 1920, "zipf"), (100, 128, 0, 128, 4, 2048, 128, "zipf"), (33, 128, 32, 64, 8, 1024, 1024, "uniform"),
    (64, 64, 0, 64, 2, 2048, 384, "one"), (90, 256, 16, 32, 16, 2048, 1152, "zipf"), (150, 64, 0, 64, 4, 1024, 640, "uniform"),
    (17, 1024, 512, 300, 8, 2048, 256, "uniform")]


@pytest.mark.parametrize("T,E,begin,L,k,H,I,mode", FUSED)
def test_layer_of_few_rows(T, E, begin, L, k, H, I, mode):
    test_layer(T, E, begin, L, k, H, I, mode)


@pytest.mark.parametrize("T,I", [(5, 768), (20, 1152), (300, 768)])
def test_layer_rows_of_nan_and_zero(T, I):
    """A token's NaN or zero scale reaches its own output only."""
    from w4a16_grouped_gemm_amd import ops
    x, ids, w, w13, s13, w2, s2 = layer_inputs(T, 64, 0, 64, 4, 2048, I, "uniform", I + T)
    xq, xs = ops.int8_quantize(x)
    want = ops.moe_w8a8_forward(xq, xs, ids, w, w13, s13, w2, s2)
    xs[1] = float("nan")
    xs[3] = 0.0
    out = ops.moe_w8a8_forward(xq, xs, ids, w, w13, s13, w2, s2)
    assert bool(out[1].isnan().all()) and bool((out[3] == 0).all())
    keep = torch.tensor([t not in (1, 3) for t in range(T)], device="cuda")
    assert torch.equal(out[keep], want[keep])


def test_layer_with_an_expert_named_twice():
    from w4a16_grouped_gemm_amd import ops
    # the permutation of one workgroup (one and several token ranges) and of many
    for T, E in ((3, 8), (40, 8), (300, 1024), (500, 8)):
        x, ids, w, w13, s13, w2, s2 = layer_inputs(T, E, 0, E, 4, 256, 128, "uniform", 2)
        ids[:, 3] = ids[:, 0]
        ids[0, :] = 5
        ids[1, 1] = -1                                            # no such expert: the slot adds nothing
        ids[1, 2] = E
        xq, xs = ops.int8_quantize(x)
        out = ops.moe_w8a8_forward(xq, xs, ids, w, w13, s13, w2, s2)
        want = layer_reference(xq, xs, ids, w, w13, s13, w2, s2, 0).bfloat16()
        assert_layer_close(to_np_u16(out), to_np_u16(want), f"twice T={T}")


def block(x, res, gain, logits, bias, weights, k, begin=0, E=None):
    """What stands between two residual additions: norm, router, experts."""
    from w4a16_grouped_gemm_amd import ops
    q, s, h = ops.add_rms_norm_int8(x, res, gain)
    ids, w = ops.route_scored(logits, k, bias=bias, num_groups=4, topk_groups=2, group_top=2, scale=2.0)
    return ops.moe_w8a8_forward(q, s, ids, w, *weights, num_experts=E, expert_begin=begin), h, ids, w


def block_inputs(T, E, H, I, seed):
    g = gen(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")   # noqa: E731
    weights = (codes(g, E, 2 * I, H), scales(g, E, 2 * I) / H ** 0.5, codes(g, E, H, I), scales(g, E, H) / I ** 0.5)
    return r(T, H).bfloat16(), r(T, H).bfloat16(), (1 + 0.1 * r(H)).bfloat16(), r(T, E), r(E) * 0.1, weights


@pytest.mark.parametrize("T", [1, 4, 37, 600])
def test_operators_together(T):
    """Norm, router and layer in a row, against their definitions in a row."""
    x, res, gain, logits, bias, weights = block_inputs(T, 16, 256, 384, T)
    out, h, ids, w = block(x, res, gain, logits, bias, weights, 4)
    assert torch.equal(h, (x.float() + res.float()).bfloat16())
    d = h.double()
    v = d / (d.square().mean(-1, keepdim=True) + 1e-6).sqrt() * gain.double()
    want = layer_reference(quantized(v), torch.ones(T, device="cuda"), ids, w, *weights, 0).bfloat16()
    assert_layer_close(to_np_u16(out), to_np_u16(want), f"together T={T}")


def test_captured_and_replayed():
    """One graph of the whole run, replayed on changing inputs with eager work between: equal to the eager results."""
    T = 24
    x, res, gain, logits, bias, weights = block_inputs(T, 16, 256, 384, 9)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(2):
            block(x, res, gain, logits, bias, weights, 4)
    torch.cuda.synchronize()
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = block(x, res, gain, logits, bias, weights, 4)
    with torch.cuda.graph(other):
        got2 = block(x, res, gain, logits, bias, weights, 4)
    for i in range(4):
        n = block_inputs(T, 16, 256, 384, 100 + i)
        x.copy_(n[0])
        res.copy_(n[1])
        logits.copy_(n[3])
        want = block(x, res, gain, logits, bias, weights, 4)
        torch.cuda.synchronize()
        graph.replay()
        block(n[1], n[0], gain, n[3], bias, weights, 4)
        other.replay()
        torch.cuda.synchronize()
        for a, b, c in zip(got, want, got2):
            assert torch.equal(a, b) and torch.equal(c, b), i


def test_two_streams():
    """Two runs at once, each on its own stream: nothing is shared."""
    ins = [block_inputs(64, 16, 256, 384, s) for s in (1, 2)]
    want = [block(*n, 4) for n in ins]
    streams = [torch.cuda.Stream() for _ in ins]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(block(*ins[i], 4))
    torch.cuda.synchronize()
    for i in range(2):
        for r in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(r, want[i]))


def test_stream_argument():
    from w4a16_grouped_gemm_amd import ops
    g = gen(3)
    x = torch.randn(64, 512, generator=g, device="cuda").bfloat16()
    w, ws = codes(g, 256, 512), scales(g, 256)
    q0, s0 = ops.int8_quantize(x)
    want = ops.dense_gemm_w8a8(q0, s0, w, ws)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    for stream in (st, st.cuda_stream):
        q, s = ops.int8_quantize(x, stream=stream)
        out = ops.dense_gemm_w8a8(q, s, w, ws, stream=stream)
        st.synchronize()
        assert torch.equal(out, want)


def test_refusals():
    from w4a16_grouped_gemm_amd import ops
    g = gen(4)
    a, s, w, ws = codes(g, 4, 256), scales(g, 4), codes(g, 32, 256), scales(g, 32)
    bad = [(a.t(), s, w, ws), (a, s[:3], w, ws), (a, s.double(), w, ws), (a, s, w[:, :128], ws), (a, s, w, ws[:16]),
           (a, s.cpu(), w, ws), (a[:, :192].contiguous(), s, w[:, :192].contiguous(), ws), (a, s, w[:24], ws[:24])]
    for args in bad:
        with pytest.raises(ValueError):
            ops.dense_gemm_w8a8(*args)
    with pytest.raises(ValueError):
        ops.dense_gemm_w8a8(a, s, w, ws, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        ops.dense_gemm_w8a8(a, s, w, ws, out=torch.empty(4, 16, device="cuda"))
    x, ids, tw, w13, s13, w2, s2 = layer_inputs(4, 8, 0, 8, 2, 256, 256, "uniform", 2)
    xq, xs = ops.int8_quantize(x)
    for args in [(xq, xs, ids.long(), tw, w13, s13, w2, s2), (xq, xs, ids, tw[:, :1], w13, s13, w2, s2),
                 (xq, xs, ids, tw, w13, s13, w2[:, :128], s2), (xq, xs, ids, tw, w13, s13[:, :256], w2, s2)]:
        with pytest.raises(ValueError):
            ops.moe_w8a8_forward(*args)
    with pytest.raises(ValueError):
        ops.moe_w8a8_forward(xq, xs, ids, tw, w13, s13, w2, s2, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        ops.moe_w8a8_forward(xq, xs, ids, tw, w13, s13, w2, s2, num_experts=4)
    out = torch.empty(4, 256, dtype=torch.bfloat16, device="cuda")
    assert ops.moe_w8a8_forward(xq[:0], xs[:0], ids[:0], tw[:0], w13, s13, w2, s2, out=out[:0]).shape == (0, 256)


@pytest.mark.parametrize("T,E,k", [(1, 1024, 16), (3, 8, 4), (40, 8, 4), (64, 128, 16), (128, 1000, 8), (300, 1024, 3), (380, 8, 4),
                                   (500, 8, 4), (3000, 64, 16)])
def test_permute_with_an_expert_named_twice(T, E, k):
    """Both slots of such a token have the expert's one row for it, and every row below R holds a slot."""
    from w4a16_grouped_gemm_amd import ops
    say(f"permute T={T} E={E} k={k} with repeated ids")
    g = gen(T)
    ids = torch.randint(-1, E + 1, (T, k), generator=g, device="cuda", dtype=torch.int32)
    ids[0] = 1
    counts, offsets, perm, inv, _ = (t.cpu().numpy() if t is not None else None for t in ops.permute(ids, E))
    named = ids.cpu().numpy()
    want, rows = np.zeros(E, int), {}
    for e in range(E):
        for t in np.flatnonzero((named == e).any(1)):
            rows[e, t] = want[e]
            want[e] += 1
    off = np.concatenate([[0], want.cumsum()])
    assert np.array_equal(counts, want) and np.array_equal(offsets, off)
    for t in range(T):
        for j in range(k):
            e = named[t, j]
            r = off[e] + rows[e, t] if 0 <= e < E else -1
            assert inv[t, j] == r
            assert r < 0 or (perm[r] // k == t and named[t, perm[r] % k] == e)
    assert (perm[off[-1]:] == -1).all()


def test_outputs_are_ordinary_tensors():
    """Own storage, dense, on the inputs' device; inference tensors in inference mode; also without the short allocation."""
    from w4a16_grouped_gemm_amd import ops
    g = gen(9)
    x = torch.randn(3, 2, 256, generator=g, device="cuda").bfloat16()
    a, s, w, ws = codes(g, 4, 256), scales(g, 4), codes(g, 32, 256), scales(g, 32)
    l, gain = torch.randn(5, 16, generator=g, device="cuda"), torch.ones(256, device="cuda").bfloat16()

    def outputs():
        return [*ops.int8_quantize(x), *ops.add_rms_norm_int8(x, x, gain, with_bf16=True), *ops.route_scored(l, 2),
                ops.dense_gemm_w8a8(a, s, w, ws), ops.rms_norm(x.view(6, 256), gain)]

    want = outputs()
    assert [tuple(t.shape) for t in want] == [(3, 2, 256), (3, 2), (3, 2, 256), (3, 2), (3, 2, 256), (3, 2, 256), (5, 2),
                                              (5, 2), (4, 32), (6, 256)]
    assert len({t.data_ptr() for t in want}) == len(want)
    for t in want:
        assert t.is_contiguous() and t.device == x.device and not t.requires_grad and not t.is_inference()
    with torch.inference_mode():
        inside = outputs()
    short = ops._empty
    try:
        ops._empty = lambda size, stride, dtype: torch.empty_strided(size, stride, dtype=dtype, device="cuda")
        plain = outputs()
    finally:
        ops._empty = short
    for t, i, p in zip(want, inside, plain):
        assert i.is_inference() and torch.equal(t, i) and torch.equal(t, p)


LOW, HIGH = -2 ** 31, 2 ** 31 - 1


@pytest.mark.parametrize("E", [6, 300])
@pytest.mark.parametrize("T", [40, 700])
@pytest.mark.parametrize("hostile", [(LOW, -3, LOW + 7), (LOW, 0, LOW), (-1, LOW, -40), (HIGH, HIGH, HIGH), (LOW, HIGH, HIGH)])
def test_offsets_that_leave_the_rows(E, T, hostile):
    """Offsets are the caller's: whatever they hold, only rows of the arrays are read and written. Here two experts have
    their rows, what follows them goes below 0, past the rows or through the ends of 32 bits."""
    from w4a16_grouped_gemm_amd import ops
    say(f"offsets E={E} T={T} {hostile}")
    g, H, I = gen(E + T), 256, 128
    a, s, w, ws = codes(g, T, I), scales(g, T), codes(g, E, H, I), scales(g, E, H)
    n = T // 3
    offsets = torch.tensor([0, n, 2 * n] + [hostile[i % 3] for i in range(E - 2)], dtype=torch.int32, device="cuda")
    memory = torch.full((T + 128, H), 7.0, device="cuda")
    ops.grouped_gemm_w8a8(ops.W2, a, s, offsets, w, ws, num_tokens=T, top_k=1, num_experts=E, out=memory[64:64 + T])
    out = memory[64:64 + T]
    assert bool((memory[:64] == 7).all()) and bool((memory[64 + T:] == 7).all())
    if hostile != (LOW, HIGH, HIGH):                              # else an expert's segment becomes all rows
        for e in (0, 1):
            r = slice(e * n, (e + 1) * n)
            assert near(out[r], dense(a[r], s[r], w[e], ws[e]), F32_REL)
        if hostile[0] == HIGH:                                    # the third expert's: up to the last row
            assert near(out[2 * n:], dense(a[2 * n:], s[2 * n:], w[2], ws[2]), F32_REL)
        else:
            assert bool((out[2 * n:] == 7).all())


@pytest.mark.parametrize("T", [12, 500])
def test_index_entries_that_leave_the_rows(T):
    """So are index entries: rows with entries of the array come out right beside others."""
    from w4a16_grouped_gemm_amd import ops
    g, E, k, H, I = gen(T), 4, 2, 256, 128
    x, xs, w, ws = codes(g, T, H), scales(g, T), codes(g, E, 2 * I, H), scales(g, E, 2 * I)
    perm = torch.randperm(T * k, generator=g, device="cuda").to(torch.int32)
    bad = torch.arange(T * k, device="cuda") % 5 == 3
    perm[bad] = torch.tensor([LOW, -1, HIGH, T * k], dtype=torch.int32, device="cuda").repeat(T)[:int(bad.sum())]
    n = T * k // 4
    offsets = torch.tensor([0, n, 2 * n, 3 * n, T * k], dtype=torch.int32, device="cuda")
    out = ops.grouped_gemm_w8a8(ops.W13_RAW, x, xs, offsets, w, ws, num_tokens=T, top_k=k, a_row_index=perm,
                                out_dtype=torch.float32)
    token = perm.long().clamp(0, T * k - 1) // k
    for e in range(E):
        r = slice(int(offsets[e]), int(offsets[e + 1]))
        assert near(out[r], dense(x[token[r]], xs[token[r]], w[e], ws[e]), F32_REL)


@pytest.mark.parametrize("T,E,k", [(1, 16, 16), (5, 4, 3), (40, 7, 7), (64, 128, 16), (93, 11, 11), (100, 1000, 10), (128, 8, 8),
                                   (300, 1024, 3), (380, 8, 4), (500, 8, 4), (3000, 64, 16)])
def test_permute_keeps_the_last_slot_of_a_row(T, E, k):
    """The row of a token that names an expert more than once holds the last of those slots, in every variant and at
    every call."""
    from w4a16_grouped_gemm_amd import ops
    say(f"permute T={T} E={E} k={k}, the slot of a shared row")
    ids = torch.randint(-1, E + 1, (T, k), generator=gen(T + k), device="cuda", dtype=torch.int32)
    first = ops.permute(ids, E)
    for _ in range(5):
        again = ops.permute(ids, E)
        assert all(torch.equal(a, b) for a, b in zip(first[:4], again[:4]))
    offsets, perm, inv = (t.cpu().numpy() for t in first[1:4])
    want = np.full(T * k, -1)
    for slot in range(T * k):                                     # in order, so the last one stays
        if inv[slot // k, slot % k] >= 0:
            want[inv[slot // k, slot % k]] = slot
    assert np.array_equal(perm, want) and (want[:offsets[-1]] >= 0).all()


VARIANTS = [  # shapes for the kernel variants that no shape above reaches
    (256, 128, 0, 128, 8, 1024, 768, "uniform"),                  # 256 x 64 tiles, in all three kinds
    (24, 4, 0, 4, 4, 256, 256, "uniform"),                        # the streaming SwiGLU product of two token subtiles,
    (24, 4, 0, 4, 4, 256, 2048, "uniform")]                       # of two tiles a wave and of four


@pytest.mark.parametrize("T,E,begin,L,k,H,I,mode", VARIANTS)
def test_grouped_in_the_other_variants(T, E, begin, L, k, H, I, mode):
    test_grouped(T, E, begin, L, k, H, I, mode)


def test_workspace_of_the_caller_may_hold_anything():
    """One workspace for calls of several sizes, full of ones' bits or of what the last call left: the same results."""
    from w4a16_grouped_gemm_amd import ops
    space = None
    for T, E, L, begin, k, H, I in [(700, 16, 16, 0, 4, 512, 384), (3, 16, 8, 4, 4, 512, 384), (64, 64, 64, 0, 8, 2048, 768),
                                    (1, 64, 64, 0, 8, 2048, 768), (300, 16, 4, 12, 2, 256, 256)]:
        x, ids, w, w13, s13, w2, s2 = layer_inputs(T, E, begin, L, k, H, I, "uniform", T + H)
        xq, xs = ops.int8_quantize(x)
        kw = dict(num_experts=E, expert_begin=begin)
        want = ops.moe_w8a8_forward(xq, xs, ids, w, w13, s13, w2, s2, **kw)
        if space is None:
            space = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
        for fill in (255, None):
            if fill is not None:
                space.fill_(fill)
            assert torch.equal(ops.moe_w8a8_forward(xq, xs, ids, w, w13, s13, w2, s2, workspace=space, **kw), want)


def test_two_threads():
    """Two threads, each with its stream and its own sizes, through the same binding."""
    import threading
    ins = [block_inputs(T, 16, 256, 384, T) for T in (5, 300)]
    want = [block(*n, 4) for n in ins]
    torch.cuda.synchronize()
    got, errors = [[], []], []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    got[i].append(block(*ins[i], 4))
                torch.cuda.current_stream().synchronize()
        except Exception as e:                                    # shown by the assertion below
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for i in range(2):
        assert len(got[i]) == 20
        for r in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(r, want[i]))
