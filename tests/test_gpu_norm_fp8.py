"""FP8 rows and weight blocks against their definition in 64 bits.

Without powers of two a code is the nearest one to the exact quotient (ties to the even one) wherever the values are
bf16 or products of two of them, behind the norm too, so codes are compared for equality. Scales: the quantizers'
max / 448 is rounded once, to within 2^-23 relative even where the last bit is off. The norm's carries rstd, which is
off by less than 2^-18 relative (u = 2^-24: a mean of K squares of at most 64 FMAs per thread, 6 steps in a wave and 16
over waves is off by less than 90 u, rstd by half of that and 3 u, the products by 4 u). With powers of two behind the
norm, a value next to a power of two may get either, and a value next to the middle of two codes either code: the code
is within half a step of the quotient of v (1 +- 2^-18).
"""
import pytest
import torch

from helpers import say

pytestmark = pytest.mark.gpu

V = 2.0 ** -18
NOTHING = 2.0 ** -100


def step(v):
    """The distance of neighbouring codes around v."""
    return torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)


def e4m3(v):
    return ((v / step(v)).round() * step(v)).clamp(-448, 448)


def least_power(v):
    """The least power of two that is not less than v > 0, exact."""
    m, e = torch.frexp(v)
    return torch.ldexp(torch.ones_like(v), e - (m == 0.5).int())


def blocks(v, rows=1):
    R, K = v.shape
    full = torch.zeros(-(-R // rows) * rows, K, dtype=torch.float64)
    full[:R] = v
    return full.view(-1, rows, K // 128, 128)


def quantized(v, pow2, rows=1):
    """Codes as values [R, K] and scales of 64-bit values with few bits, in blocks of rows x 128."""
    b = blocks(v, rows)
    top = b.abs().amax((1, 3))
    fine, dead = top.isfinite(), top < NOTHING
    safe = torch.where(fine & ~dead, top, torch.ones_like(top))
    scale = least_power(safe / 448) if pow2 else safe / 448       # / 448 in 64 bits keeps which side of a power it is on
    over = scale if pow2 else safe
    q = e4m3(b.nan_to_num(0, 0, 0) * (1 if pow2 else 448) / over[:, None, :, None])
    q = torch.where((fine & ~dead)[:, None, :, None], q, torch.zeros_like(q))
    scale = torch.where(dead, torch.zeros_like(scale), scale)
    return q.view(-1, v.shape[1])[:v.shape[0]], torch.where(fine, scale, torch.full_like(scale, float("nan")))


def check(q, s, v, pow2, rows=1):
    want, scale = quantized(v, pow2, rows)
    got = s.double().cpu()
    assert torch.equal(got.isnan(), scale.isnan())
    ok = ~scale.isnan()
    assert bool(((got - scale).abs()[ok] <= scale[ok] * (0 if pow2 else 2.0 ** -23)).all())
    assert torch.equal(q.float().double().cpu().view(want.shape), want)


def rows_of(rows, K, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, K, generator=g) * spread
    return x, g


SIZES = [(1, 128), (3, 256), (5, 512), (9, 640), (1, 1024), (7, 1152), (3, 2048), (1500, 2048), (2, 4096), (5, 7168),
         (3, 16384), (2, 16512), (1, 65536), (300, 384)]


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("rows,K", SIZES)
def test_quantize(rows, K, pow2):
    from w4a16_grouped_gemm_amd import ops
    say(f"fp8_quantize {rows}x{K} pow2={pow2}")
    x, g = rows_of(rows, K, rows * 7 + K)
    x = (x * torch.exp2(torch.randint(-40, 40, (rows, K // 128), generator=g).float()).repeat_interleave(128, 1)).bfloat16()
    q, s = ops.fp8_quantize(x.cuda(), pow2=pow2)
    assert q.dtype == torch.float8_e4m3fn and q.shape == x.shape and s.shape == (rows, K // 128)
    check(q, s, x.double(), pow2)


@pytest.mark.parametrize("pow2", [False, True])
def test_quantize_unusual_blocks(pow2):
    """Zeros, minus zeros, blocks below what counts, subnormals, the largest values, NaN, infinities, ties, one value."""
    from w4a16_grouped_gemm_amd import ops
    big = torch.finfo(torch.bfloat16).max
    b = torch.zeros(16, 128)
    b[1] = -0.0
    b[2] = 2.0 ** -101
    b[3] = 2.0 ** -100
    b[4, 7] = 2.0 ** -133
    b[5] = big
    b[6] = torch.linspace(-1, 1, 128) * big
    b[7], b[7, 9] = 1.0, float("nan")
    b[8], b[8, 127] = 1.0, -float("inf")
    b[9] = torch.arange(128).float()                              # ties of every kind beside 448
    b[9, 0] = 448.0
    b[10] = torch.arange(128).float() / 8
    b[10, 1] = -28.0
    b[11, 64] = -3.0
    b[12] = 448.0
    b[13] = 449.0
    b[14] = 2.0 ** -99 * 1.75
    b[15, :2] = torch.tensor([1.0, 2.0 ** -9])
    x = b.view(4, 512).bfloat16()
    q, s = ops.fp8_quantize(x.cuda(), pow2=pow2)
    check(q, s, x.double(), pow2)


def test_every_bf16_value_beside_every_exponent_of_a_largest():
    """All 256 x 2 codes' neighbourhoods: each positive bf16 significand under each largest significand."""
    from w4a16_grouped_gemm_amd import ops
    top = (1 + torch.arange(128).float() / 128)                   # 128 significands of the largest
    v = (1 + torch.arange(128).float() / 128)
    for down in range(0, 12):
        rows = (v[None, None, :] * 2.0 ** -down).expand(128, 1, 128).clone()
        rows = torch.minimum(rows, top[:, None, None])
        rows[:, 0, 0] = top
        x = rows.view(128, 128).bfloat16()
        q, s = ops.fp8_quantize(x.cuda())
        check(q, s, x.double(), False)


def reference(x, r, w, eps):
    h = x if r is None else (x.float() + r.float()).bfloat16()
    d = h.double()
    return h, d * w.double(), (d.square().mean(-1, keepdim=True) + eps).pow(-0.5)


def check_norm(q, s, u, rstd, pow2):
    q, s = q.float().double().cpu(), s.double().cpu()
    if not pow2:
        want, _ = quantized(u * torch.exp2(torch.floor(torch.log2(rstd))), False)    # of v's magnitude: which blocks count
        top = blocks(u).abs().amax((1, 3)) * rstd
        assert torch.equal(q, want)
        assert bool(((s - top / 448).abs() <= top / 448 * V).all())
        return
    v = blocks(u * rstd)
    top = v.abs().amax((1, 3))
    low, high = least_power(top * (1 - V) / 448), least_power(top * (1 + V) / 448)
    assert bool(((s == low) | (s == high)).all())
    t = v / s[:, None, :, None]
    off = (blocks(q) - t).abs()
    assert bool((off <= step(t * (1 - V)).maximum(step(t * (1 + V))) / 2 + t.abs() * V).all())


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("res", [False, True])
@pytest.mark.parametrize("rows,K", SIZES)
def test_norm(rows, K, res, pow2):
    from w4a16_grouped_gemm_amd import ops
    say(f"norm to FP8 {rows}x{K} residual={res} pow2={pow2}")
    x, g = rows_of(rows, K, rows + K)
    x, r = x.bfloat16(), (torch.randn(rows, K, generator=g) * 2).bfloat16()
    w = (1 + 0.2 * torch.randn(K, generator=g)).bfloat16()
    h, u, rstd = reference(x, r if res else None, w, 1e-5)
    xd, rd, wd = x.cuda(), r.cuda(), w.cuda()
    kw = dict(eps=1e-5, pow2=pow2)
    if res:
        q, s, hs = ops.add_rms_norm_fp8(xd, rd, wd, **kw)
        q2, s2, hs2, y = ops.add_rms_norm_fp8(xd, rd, wd, with_bf16=True, **kw)
        assert torch.equal(hs.cpu(), h) and torch.equal(hs2.cpu(), h)
        assert torch.equal(y, ops.add_rms_norm(xd, rd, wd, eps=1e-5)[0])
        for target in (rd.clone(), xd.clone()):                   # in place of the residual, of x
            args = (xd, target) if target.data_ptr() != xd.data_ptr() and torch.equal(target, rd) else (target, rd)
            q3, s3, hs3 = ops.add_rms_norm_fp8(*args, wd, sum_out=target, **kw)
            assert hs3 is target and torch.equal(target.cpu(), h)
            assert torch.equal(q3.view(torch.uint8), q.view(torch.uint8)) and torch.equal(s3, s)
    else:
        q, s = ops.rms_norm_fp8(xd, wd, **kw)
        q2, s2, y = ops.rms_norm_fp8(xd, wd, with_bf16=True, **kw)
        assert torch.equal(y, ops.rms_norm(xd, wd, eps=1e-5))
    assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s, s2)
    check_norm(q, s, u, rstd, pow2)


@pytest.mark.parametrize("K", [128, 2048, 7168, 16512])
@pytest.mark.parametrize("scale", [2.0 ** 100, 2.0 ** 66, 2.0 ** -70, 2.0 ** -110])
def test_norm_of_rows_out_of_range(K, scale):
    """Finite rows whose squares leave binary32: among ordinary rows, with and without the bf16 rows, in place too."""
    from w4a16_grouped_gemm_amd import ops
    say(f"norm to FP8 of rows times {scale}, K={K}")
    x, g = rows_of(6, K, K)
    x[1::2] *= scale
    x = x.bfloat16()
    w = (1 + 0.2 * torch.randn(K, generator=g)).bfloat16()
    eps = 2.0 ** -126 if scale < 1 else 1e-6                      # an eps that leaves the small rows their norm
    _, u, rstd = reference(x, None, w, eps)
    for pow2 in (False, True):
        q, s = ops.rms_norm_fp8(x.cuda(), w.cuda(), eps=eps, pow2=pow2)
        check_norm(q, s, u, rstd, pow2)
        q2, s2, y = ops.rms_norm_fp8(x.cuda(), w.cuda(), eps=eps, pow2=pow2, with_bf16=True)
        assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s, s2)
        assert torch.equal(y, ops.rms_norm(x.cuda(), w.cuda(), eps=eps))
        r = torch.zeros_like(x).cuda()
        q3, s3, h = ops.add_rms_norm_fp8(x.cuda(), r, w.cuda(), eps=eps, pow2=pow2, sum_out=r)
        assert h is r and torch.equal(q.view(torch.uint8), q3.view(torch.uint8)) and torch.equal(s, s3)


def test_norm_rows_of_zeros_nan_and_infinities():
    from w4a16_grouped_gemm_amd import ops
    for K in (256, 7168):
        x, _ = rows_of(6, K, 1)
        x[1], x[2, 5], x[3, 200], x[4] = 0, float("nan"), float("inf"), -0.0
        x = x.bfloat16()
        w = torch.ones(K).bfloat16()
        want = ops.rms_norm_fp8(x[:1].cuda(), w.cuda())
        q, s = ops.rms_norm_fp8(x.cuda(), w.cuda())
        assert torch.equal(q[:1].view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(s[:1], want[1])
        for row in (1, 4):
            assert bool((q[row].float() == 0).all()) and bool((s[row] == 0).all())
        for row in (2, 3):
            assert bool((q[row].float() == 0).all()) and bool(s[row].isnan().all())
        q, s = ops.rms_norm_fp8(x.cuda(), w.cuda(), eps=0.0)
        assert bool(s[1].isnan().all()) and bool((q[1].float() == 0).all())


def test_norm_of_gains_that_leave_the_range():
    """A product that binary32 does not hold is an infinity, and its block's alone."""
    from w4a16_grouped_gemm_amd import ops
    x, _ = rows_of(2, 384, 3)
    w = torch.ones(384)
    w[130] = torch.finfo(torch.bfloat16).max
    x[:, 130] = 100.0
    q, s = ops.rms_norm_fp8(x.bfloat16().cuda(), w.bfloat16().cuda())
    assert bool(s[:, 1].isnan().all()) and bool((q[:, 128:256].float() == 0).all()) and bool(s[:, [0, 2]].isfinite().all())


WEIGHTS = [(1, 16, 128), (1, 128, 128), (1, 127, 256), (2, 129, 384), (3, 2112, 256), (1, 1, 7168), (5, 256, 512),
           (1, 576, 1024), (40, 128, 128)]


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("E,N,K", WEIGHTS)
def test_weights(E, N, K, pow2):
    from w4a16_grouped_gemm_amd import ops
    say(f"fp8_quantize_weights {E}x{N}x{K} pow2={pow2}")
    g = torch.Generator().manual_seed(E * N + K)
    w = torch.randn(E, N, K, generator=g)
    w[:, : (N + 1) // 2, :128] *= 2.0 ** -20
    w[0, 0, :] = 0
    if N > 128:
        w[-1, 128:, -128:] = 0
    w = w.bfloat16()
    q, s = ops.fp8_quantize_weights(w.cuda(), pow2=pow2)
    assert q.shape == w.shape and s.shape == (E, -(-N // 128), K // 128)
    for e in range(E):
        check(q[e], s[e], w[e].double(), pow2, 128)
    q1, s1 = ops.fp8_quantize_weights(w[0].cuda(), pow2=pow2)
    assert torch.equal(q1.view(torch.uint8), q[0].view(torch.uint8)) and torch.equal(s1, s[0])


def test_weights_with_nan_and_infinity():
    from w4a16_grouped_gemm_amd import ops
    w = torch.ones(300, 384)
    w[5, 5], w[299, 383] = float("nan"), float("inf")
    w = w.bfloat16()
    q, s = ops.fp8_quantize_weights(w.cuda())
    check(q, s, w.double(), False, 128)
    assert int(s.isnan().sum()) == 2


def test_nothing_to_do():
    from w4a16_grouped_gemm_amd import ops
    x, w = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda"), torch.ones(256, dtype=torch.bfloat16, device="cuda")
    assert [tuple(t.shape) for t in ops.fp8_quantize(x)] == [(0, 256), (0, 2)]
    assert [tuple(t.shape) for t in ops.add_rms_norm_fp8(x, x, w)] == [(0, 256), (0, 2), (0, 256)]
    assert [tuple(t.shape) for t in ops.fp8_quantize_weights(x)] == [(0, 256), (0, 2)]
    assert [tuple(t.shape) for t in ops.fp8_quantize_weights(x.view(0, 5, 256))] == [(0, 5, 256), (0, 1, 2)]


@pytest.mark.parametrize("K", [256, 2048, 7168, 20480])
def test_norm_of_infinite_eps(K):
    """Every eps >= 0 is taken. An infinite one makes rows of finite values zeros, codes and scales, as in the int8 norm;
    a row with a NaN or an infinity still has NaN scales."""
    from w4a16_grouped_gemm_amd import ops
    x, _ = rows_of(4, K, K)
    x[2, 5], x[3, 7] = float("inf"), float("nan")
    x, w = x.bfloat16().cuda(), torch.ones(K, device="cuda").bfloat16()
    for pow2 in (False, True):
        q, s, y = ops.rms_norm_fp8(x, w, eps=float("inf"), pow2=pow2, with_bf16=True)
        assert bool((q[:2].float() == 0).all()) and bool((s[:2] == 0).all()) and bool((y[:2] == 0).all())
        assert bool(s[2:].isnan().all())
