"""RMS norm and the int8 quantizer against their definition in 64 bits.

Error bounds (u = 2^-24, half a binary32 step): a mean of K squares is summed by at most 64 FMAs per thread, 6 steps
in a wave and 16 over waves, so it is off by less than 90 u; rstd by half of that and 3 u, the two products by 2 u: in
all less than 64 u = 2^-18 relative. bf16 adds half a step, 2^-8. A code is within 1/2 + 127 * 2^-17 of the exact
quotient (the value's and the maximum's 2^-18 each, the division's far less).
"""
import pytest
import torch

from helpers import say

pytestmark = pytest.mark.gpu

V = 2.0 ** -18


def inputs(rows, K, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(rows, K, generator=g) * spread).bfloat16()
    r = (torch.randn(rows, K, generator=g) * 2 * spread).bfloat16()
    w = (1 + 0.2 * torch.randn(K, generator=g)).bfloat16()
    return x, r, w


def reference(x, r, w, eps):
    h = x if r is None else (x.float() + r.float()).bfloat16()
    d = h.double()
    return h, d / (d.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()


def near(got, want, rel):
    return ((got.double().cpu() - want).abs() <= want.abs() * rel + 2.0 ** -130).all()


def check_codes(q, s, v):
    top = v.abs().amax(-1, keepdim=True)
    assert ((s.double().cpu()[:, None] - top / 127).abs() <= top / 127 * 2 * V).all()
    assert ((q.double().cpu() - 127 * v / top).abs() <= 0.5 + 127 * 2 * V).all()


SIZES = [(1, 8), (3, 128), (5, 504), (9, 512), (1, 520), (7, 2048), (3, 2056), (2, 4096), (5, 7168), (3, 16384),
         (2, 16392), (1, 65536), (300, 256)]


@pytest.mark.parametrize("rows,K", SIZES)
@pytest.mark.parametrize("res", [False, True])
def test_norm(rows, K, res):
    from w4a16_grouped_gemm_amd import ops
    say(f"norm {rows}x{K} residual={res}")
    x, r, w = inputs(rows, K, rows * 7 + K)
    r = r if res else None
    h, v = reference(x, r, w, 1e-5)
    xd, wd = x.cuda(), w.cuda()
    if res:
        rd = r.cuda()
        y, s = ops.add_rms_norm(xd, rd, wd, eps=1e-5)
        q, sc, s2, y2 = ops.add_rms_norm_int8(xd, rd, wd, eps=1e-5, with_bf16=True)
        q3, sc3, s3 = ops.add_rms_norm_int8(xd, rd, wd, eps=1e-5)
        for t in (s, s2, s3):
            assert torch.equal(t.cpu(), h)
        assert torch.equal(rd.cpu(), r)
    else:
        y = ops.rms_norm(xd, wd, eps=1e-5)
        q, sc, y2 = ops.rms_norm_int8(xd, wd, eps=1e-5, with_bf16=True)
        q3, sc3 = ops.rms_norm_int8(xd, wd, eps=1e-5)
    assert torch.equal(y, y2) and torch.equal(q, q3) and torch.equal(sc, sc3)
    assert near(y, v, 2.0 ** -8 + 2 * V)
    check_codes(q, sc, v)


def test_in_place_and_leading_dimensions():
    from w4a16_grouped_gemm_amd import ops
    x, r, w = inputs(24, 2048, 5)
    want = ops.add_rms_norm_int8(x.cuda(), r.cuda(), w.cuda(), with_bf16=True)
    rd = r.cuda().view(2, 3, 4, 2048)
    q, s, h, y = ops.add_rms_norm_int8(x.cuda().view(2, 3, 4, 2048), rd, w.cuda(), sum_out=rd, with_bf16=True)
    assert h.data_ptr() == rd.data_ptr() and q.shape == rd.shape and s.shape == (2, 3, 4)
    for a, b in zip((q, s, h, y), want):
        assert torch.equal(a.flatten(), b.flatten())
    xd = x.cuda()
    y2, h2 = ops.add_rms_norm(xd, r.cuda(), w.cuda(), sum_out=xd)
    assert torch.equal(y2, want[3]) and torch.equal(h2, want[2]) and h2.data_ptr() == xd.data_ptr()
    with pytest.raises(ops.MoeError):
        both = torch.zeros(48, 2048, dtype=torch.bfloat16, device="cuda")
        ops.add_rms_norm(both[:24], both[24:], w.cuda(), sum_out=both[12:36])


def test_special_rows():
    from w4a16_grouped_gemm_amd import ops
    x, _, w = inputs(8, 768, 11)
    x[0] = 0
    x[1] = 2.0 ** -120                       # below what a scale is made for
    x[2, 5] = float("inf")
    x[3, 700] = float("nan")
    x[4] = 0
    x[4, 767] = -3.0                         # one value alone
    x[5] *= 2.0 ** 100                       # squares past binary32's range: the mean is infinite
    q, s = ops.int8_quantize(x.cuda())
    q, s = q.cpu(), s.cpu()
    assert (q[0] == 0).all() and (q[1] == 0).all() and s[0] == 0 and s[1] == 0
    assert (q[2] == 0).all() and (q[3] == 0).all() and s[2].isnan() and s[3].isnan()
    assert q[4, 767] == -127 and (q[4, :767] == 0).all() and s[4] == torch.tensor(3.0) / 127
    x[6] = (x[6].double() / x[6].abs().max() * 1.9 * 2.0 ** 127).bfloat16()      # the end of the range
    q, s = ops.int8_quantize(x.cuda())
    q, s = q.cpu(), s.cpu()
    for i in (5, 6, 7):
        d = x[i].double()
        assert torch.equal(q[i].double(), (127 * d / d.abs().max()).round())
    qn, sn, y = ops.rms_norm_int8(x.cuda(), w.cuda(), with_bf16=True)
    y, qn, sn = y.cpu(), qn.cpu(), sn.cpu()
    assert (y[0] == 0).all() and (qn[0] == 0).all() and sn[0] == 0
    assert sn[2].isnan() and sn[3].isnan() and y[3].isnan().all()
    _, v = reference(x[7:], None, w, 1e-6)
    check_codes(qn[7:], sn[7:], v)


@pytest.mark.parametrize("rows,K", [(1, 8), (4, 128), (33, 768), (1000, 512), (5, 2048), (6, 14336), (3, 40960)])
def test_quantizer_is_exact(rows, K):
    """Codes equal round-half-even of the exact quotient: a bf16 value over a bf16 maximum is at least 2^-16 of its
    size away from a tie that it does not hit, far more than the quotient's error, and an exact tie is representable."""
    from w4a16_grouped_gemm_amd import ops
    say(f"quantize {rows}x{K}")
    x, _, _ = inputs(rows, K, K + rows)
    x[0, ::3] = (torch.arange(0, K, 3) % 128).bfloat16() / 2          # many exact ties
    x[0, 0] = 127.0
    q, s = ops.int8_quantize(x.cuda())
    d = x.double()
    top = d.abs().amax(-1, keepdim=True)
    assert torch.equal(q.cpu().double(), (127 * d / top).round())
    assert torch.equal(s.cpu(), top[:, 0].float() / 127)


def test_every_bf16_pair_of_mantissas():
    """Each of the 128 mantissas as a row's maximum, over all mantissas and nine exponents of the values."""
    from w4a16_grouped_gemm_amd import ops
    m = (128 + torch.arange(128)).float()
    vals = torch.cat([m * 2.0 ** -e for e in range(9)] + [-m * 2.0 ** -e for e in range(9)])
    x = vals.repeat(128, 1)
    x = torch.where(x.abs() > m[:, None], torch.zeros_like(x), x)
    x = torch.cat([m[:, None], x, torch.zeros(128, 7)], 1).bfloat16().contiguous()
    q, s = ops.int8_quantize(x.cuda())
    d = x.double()
    assert torch.equal(q.cpu().double(), (127 * d / m.double()[:, None]).round())


def test_no_rows():
    from w4a16_grouped_gemm_amd import ops
    e = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    assert ops.rms_norm(e, w).shape == (0, 256)
    q, s, h = ops.add_rms_norm_int8(e, e.clone(), w)
    assert q.shape == (0, 256) and s.shape == (0,) and h.shape == (0, 256)
    assert ops.int8_quantize(e)[1].shape == (0,)


def test_refuses_a_tensor_without_dimensions():
    from w4a16_grouped_gemm_amd import ops
    x = torch.zeros((), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(8, dtype=torch.bfloat16, device="cuda")
    for call in (lambda: ops.rms_norm(x, w), lambda: ops.add_rms_norm_int8(x, x, w), lambda: ops.int8_quantize(x)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("K", [8, 512, 1032, 2048, 7168, 16384, 40960])
@pytest.mark.parametrize("rows", [3, 1100])
@pytest.mark.parametrize("res", [False, True])
def test_rows_whose_squares_leave_binary32(rows, K, res):
    """Finite rows have a norm of order one however large or small they are: among ordinary rows some whose squares
    are infinite (the largest bf16 values among them), none at all (bf16 subnormals among them) or subnormal. rstd of
    rows above 2^126 is subnormal itself, off by up to 2^-22 = 4 u more, which the bound of 64 u has room for."""
    from w4a16_grouped_gemm_amd import ops
    if rows * K > 1 << 24:
        rows = 300
    say(f"norm of extreme rows {rows}x{K} residual={res}")
    x, r, w = inputs(rows, K, rows + K)
    power = torch.tensor([0.0, 62, 64, 66, 100, 122, -50, -54, -60, -64, -70, -100, -120, -128])
    scale = 2.0 ** power[torch.arange(rows) % 14].double()
    x = (x.double().clamp(-15, 15) * scale[:, None]).bfloat16()
    r = (r.double().clamp(-15, 15) * scale[:, None]).bfloat16() if res else None
    x[0] = 0
    x[0, K // 2] = 3.0 * 2.0 ** 125                   # one value alone, a large and a small one
    x[2] = 0
    x[2, K - 1] = -2.0 ** -133
    if res:
        r[0] = 0
        r[2] = 0
    for eps in (0.0, 1e-6, 2.0 ** -130):
        h, v = reference(x, r, w, eps)
        assert h.isfinite().all() and v.isfinite().all()
        if res:
            q, sc, s2, y = ops.add_rms_norm_int8(x.cuda(), r.cuda(), w.cuda(), eps=eps, with_bf16=True)
            y2, _ = ops.add_rms_norm(x.cuda(), r.cuda(), w.cuda(), eps=eps)
            assert torch.equal(s2.cpu(), h)
        else:
            q, sc, y = ops.rms_norm_int8(x.cuda(), w.cuda(), eps=eps, with_bf16=True)
            y2 = ops.rms_norm(x.cuda(), w.cuda(), eps=eps)
        assert torch.equal(y, y2)
        assert near(y, v, 2.0 ** -8 + 2 * V)
        some = v.abs().amax(-1) >= 2.0 ** -100        # a row below that counts as zero
        check_codes(q[some.cuda()], sc[some.cuda()], v[some])
        assert (q[~some.cuda()] == 0).all() and (sc[~some.cuda()] == 0).all()


@pytest.mark.parametrize("rows,K", [(1025, 2048), (1024, 1032)])
@pytest.mark.parametrize("res", [False, True])
def test_norm_of_many_rows(rows, K, res):
    """A wave to a row of more than 1024 values, which many rows get."""
    test_norm(rows, K, res)


@pytest.mark.parametrize("rows,K", [(3, 7168), (2, 4104)])
def test_quantizer_of_more_row_lengths(rows, K):
    test_quantizer_is_exact(rows, K)


@pytest.mark.parametrize("rows,K", [(9, 512), (5, 2048), (1030, 2048), (4, 7168), (3, 40960)])
@pytest.mark.parametrize("extreme", [False, True])
def test_outputs_in_place_of_inputs(rows, K, extreme):
    """The C entry's in-place forms: y over x, the sum over the residual and y over x, the sum over x and y over the
    residual; rows out of binary32's range for squares are read again, so they must not be overwritten first."""
    import ctypes

    from w4a16_grouped_gemm_amd import ops
    say(f"norm in place {rows}x{K} extreme={extreme}")
    lib = ops.load_library()
    x, r, w = inputs(rows, K, rows + 3 * K)
    if extreme:
        scale = 2.0 ** torch.tensor([0.0, 66, 120, -70, -125])[torch.arange(rows) % 5].double()[:, None]
        x, r = (x.double().clamp(-15, 15) * scale).bfloat16(), (r.double().clamp(-15, 15) * scale).bfloat16()
    wd = w.cuda()

    def call(xd, rd, sd, yd):
        q = torch.empty(rows, K, dtype=torch.int8, device="cuda")
        s = torch.empty(rows, device="cuda")
        p = [None if t is None else t.data_ptr() for t in (xd, rd, wd)]
        assert lib.moe_rms_norm(rows, K, *p, 1e-20, None if sd is None else sd.data_ptr(), yd.data_ptr(), q.data_ptr(),
                                s.data_ptr(), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) == 0
        return [t.clone() for t in (yd, q, s)] + ([] if sd is None else [sd.clone()])

    def fresh():
        return x.cuda(), r.cuda()

    xd, rd = fresh()
    alone = call(xd, None, None, torch.empty_like(xd))
    both = call(xd, rd, torch.empty_like(xd), torch.empty_like(xd))
    for form in range(3):
        xd, rd = fresh()
        want = both if form else alone
        got = call(xd, None, None, xd) if form == 0 else call(xd, rd, rd, xd) if form == 1 else call(xd, rd, xd, rd)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), form
