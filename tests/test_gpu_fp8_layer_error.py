"""How far the FP8 layer as a whole is from its definition in 64 bits, in the mean square.

Single values of the layer have no small bound: a gate/up value that the error of its sum takes over the middle of two bf16 or
two e4m3 values becomes another code, a step of up to 1/8 of it. In the mean square it has (all relative to the result's own):
  * the result's rounding to bf16: uniform within half a step, at most 2^-8 / sqrt(3) = 2.26e-3;
  * codes that change: an error d of a value h changes its code with probability |d| / step, by one step <= |h| / 8, so the
    mean square is at most E|h d| / 8 / E h^2 <= (1/8) rms(d) / rms(h). Gate and up are each off by e (rms, relative), the
    slope of silu is at most 1.1: rms(d) / rms(h) <= (1.1 + 1) e. e = 1.5e-5 for sums of the FP8 instruction, so
    3.9e-6 = (2.0e-3)^2; binary32 sums (e < 2e-7) and the sigmoid (2^-14 at most, 2^-18 in the mean) 4 times less than that;
  * y's roundings that change, steps of 2^-7 at most: (2^-7 e)^(1/2) = 3.4e-4, with the combine's sums far below.
The sum of squares: (3.1e-3)^2 with many rows, (2.5e-3)^2 where all sums are binary32's. A test from the library's own gate/up
rows on cannot see the second.
The share of gate/up rows' values whose bf16 differs from the exact value's: an error of e of the typical value r and a step of
2^-8 |v| at least, v of a density at most 1 / (2 r): below e * 2^8 * ln(1 / e) = 4.3e-2 in sums of the FP8 instruction, 8e-4 in
binary32 ones.
"""
import pytest
import torch

from helpers import say
from test_gpu_fp8 import B16, layer_inputs, raw, requantized, values, weight_values, FP8

pytestmark = pytest.mark.gpu


def definition(xq, xs, ids, w, w13, s13, w2, s2, begin, pow2):
    T, k = ids.shape
    y = torch.zeros(T * k, w2.shape[1], dtype=torch.float64, device="cuda")
    for e in range(w13.shape[0]):
        t, j = (ids == begin + e).nonzero().unbind(1)
        if t.numel():
            gate, up = (values(raw(xq)[t].view(FP8), xs[t]) @ weight_values(w13[e], s13[e]).t()).chunk(2, -1)
            h = (gate / (1 + torch.exp(-gate)) * up).float().to(B16).double()
            y[t * k + j] = (requantized(h, pow2) @ weight_values(w2[e], s2[e]).t()).float().to(B16).double()
    return (y.view(T, k, -1) * w.double()[:, :, None]).sum(1)


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("T,E,begin,L,k,H,I,few", [(1, 128, 0, 128, 8, 2048, 768, True), (16, 128, 0, 128, 8, 2048, 768, True),
                                                   (60, 64, 16, 32, 4, 1152, 384, True), (700, 32, 8, 16, 4, 2048, 768, False),
                                                   (1100, 16, 0, 16, 4, 4096, 1024, False)])
def test_layer(T, E, begin, L, k, H, I, few, pow2):
    from w4a16_grouped_gemm_amd import ops
    x, ids, w, w13, s13, w2, s2 = layer_inputs(T, E, begin, L, k, H, I, "uniform", T + I)
    xq, xs = ops.fp8_quantize(x)
    out = ops.moe_fp8_forward(xq, xs, ids, w, w13, s13, w2, s2, num_experts=E, expert_begin=begin, pow2=pow2)
    want = definition(xq, xs, ids, w, w13, s13, w2, s2, begin, pow2)
    error = float(((out.double() - want).square().mean() / want.square().mean()).sqrt())
    say(f"  FP8 layer T={T} H={H} I={I} pow2={pow2}: rms error {error:.2e}")
    assert error <= (2.5e-3 if few else 3.1e-3)


@pytest.mark.parametrize("T,E,k,H,I,few", [(16, 128, 8, 2048, 768, True), (64, 64, 8, 4096, 256, True), (900, 16, 4, 2048, 768, False)])
def test_gate_up_rows(T, E, k, H, I, few):
    from w4a16_grouped_gemm_amd import ops
    x, ids, _, w13, s13, _, _ = layer_inputs(T, E, 0, E, k, H, I, "uniform", T + H)
    xq, xs = ops.fp8_quantize(x)
    _, offsets, perm, _, _ = ops.permute(ids, E)
    rows = ops.grouped_gemm_fp8(ops.W13_RAW, xq, xs, offsets, w13, s13, num_tokens=T, top_k=k, a_row_index=perm)
    other, off = 0, offsets.tolist()
    for e in range(E):
        t = perm[off[e]:off[e + 1]].long() // k
        exact = values(raw(xq)[t].view(FP8), xs[t]) @ weight_values(w13[e], s13[e]).t()
        other += int((rows[off[e]:off[e + 1]] != exact.float().to(B16)).sum())
    share = other / rows.numel()
    say(f"  FP8 gate/up rows T={T} E={E} H={H}: {share:.2e} of the bf16 values differ")
    assert share <= (8e-4 if few else 4.3e-2)
