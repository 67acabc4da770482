"""Sums of the FP8 products of few rows: binary32's, whatever the type of the result.

Each run of eight consecutive k holds a pair of products 4096 and -4096 beside six that are multiples of 1/16 below 1. Every
partial sum of a group is a multiple of 1/16 below 2^17, exact in binary32 in any order, and the scales are powers of two.
An adder that keeps 13 bits below the largest product of a run of eight loses the small ones.
"""
import pytest
import torch

from helpers import say
from test_gpu_fp8 import B16, F32, FP8, gen, powers, raw, values, weight_values

pytestmark = pytest.mark.gpu


def cancelling(g, rows, K, sign):
    """Rows of small multiples of 1/4, with 64 at one place of each run of eight and 64 or -64 at the next."""
    a = torch.randint(-3, 4, (rows, K // 8, 8), generator=g, device="cuda").float() / 4
    a[:, :, 2] = 64
    a[:, :, 3] = 64 * sign
    return a.view(rows, K).to(FP8)


@pytest.mark.parametrize("M", [1, 2, 9, 16, 17, 24, 32])
@pytest.mark.parametrize("N,K", [(4096, 1024), (1040, 640), (14336, 128), (2112, 4096)])
def test_dense(M, N, K):
    from w4a16_grouped_gemm_amd import ops
    if M > 16 and N == 14336:
        N = 7168
    say(f"dense_gemm_fp8 sums M={M} N={N} K={K}")
    g = gen(M + N + K)
    a, s = cancelling(g, M, K, 1), powers(g, M, K // 128)
    w, ws = cancelling(g, N, K, -1), powers(g, -(-N // 128), K // 128)
    want = values(a, s) @ weight_values(w, ws).t()
    assert torch.equal(ops.dense_gemm_fp8(a, s, w, ws, out_dtype=F32).double(), want)
    assert torch.equal(ops.dense_gemm_fp8(a, s, w, ws), want.to(F32).to(B16))


@pytest.mark.parametrize("T,E,k,H,I", [(1, 8, 2, 256, 128), (1, 128, 8, 2048, 768), (7, 16, 4, 640, 256), (64, 128, 8, 2048, 768),
                                       (30, 64, 2, 512, 1280)])
def test_grouped(T, E, k, H, I):
    """Gate, up and down rows; SwiGLU's sigmoid and products within 2^-13 and the rounding 2^-8 of the exact value."""
    from w4a16_grouped_gemm_amd import ops
    say(f"grouped_gemm_fp8 sums T={T} E={E} k={k} H={H} I={I}")
    g = gen(T + E + H)
    ids = torch.rand(T, E, generator=g, device="cuda").argsort(-1)[:, :k].to(torch.int32).contiguous()
    _, offsets, perm, _, _ = ops.permute(ids, E)
    off, token = offsets.tolist(), perm.long() // k
    x, xs = cancelling(g, T, H, 1), powers(g, T, H // 128) / 64
    w, ws = cancelling(g, E, 2 * I * H, -1).view(E, 2 * I, H), powers(g, E, 2 * I // 128, H // 128) / 8
    kw = dict(num_tokens=T, top_k=k, a_row_index=perm)
    raws = ops.grouped_gemm_fp8(ops.W13_RAW, x, xs, offsets, w, ws, **kw)
    out = ops.grouped_gemm_fp8(ops.W13_SWIGLU, x, xs, offsets, w, ws, **kw).double()
    for e in range(E):
        r = slice(off[e], off[e + 1])
        if off[e] < off[e + 1]:
            c = values(raw(x)[token[r]].view(FP8), xs[token[r]]) @ weight_values(w[e], ws[e]).t()
            assert torch.equal(raws[r], c.to(F32).to(B16))
            h = c[:, :I] / (1 + torch.exp(-c[:, :I])) * c[:, I:]
            assert bool(((out[r] - h).abs() <= h.abs() * (2.0 ** -8 + 2.0 ** -13) + 1e-30).all())
