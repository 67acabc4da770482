"""Offsets that go up and down, so that many experts name the same rows.

Such segments have up to E / 2 times as many chunks as there are rows for, while a launch has workgroups for
rows / CS + E chunks of CS rows. The tile kernel's workgroups take tile after tile: they stop at that number too, else a
call takes hundreds of times its time, and with fewer than four groups of K, where a workgroup has one tile, a second one
would be read from a record in LDS that nobody has written yet.
"""
import pytest
import torch

from helpers import say
from test_gpu_fp8 import B16, F32, gen, powers, small, values, weight_values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K", [128, 256, 384, 512, 640, 1024])
@pytest.mark.parametrize("E", [64, 128, 300])
def test_overlapping_segments(E, K):
    """Every other expert has all rows. Results are those of the experts whose chunks are within the launch's number, chunks in
    the experts' order: at most ceil((R / CS + E) / (R / CS)) of them for chunks of CS >= 64 and <= 128 rows."""
    from w4a16_grouped_gemm_amd import ops
    say(f"FP8 overlapping offsets E={E} K={K}")
    g, R, N = gen(E + K), 2048, 384
    a, s, w, ws = small(g, R, K), powers(g, R, K // 128), small(g, E, N, K), powers(g, E, 3, K // 128)
    offsets = torch.tensor([0, R] * E, dtype=torch.int32, device="cuda")[:E + 1].contiguous()
    allowed = range(0, 2 * (1 + -(-E * 128 // R)), 2)
    assert len(allowed) < E // 4
    for dtype in (B16, F32):
        memory = torch.full((R + 128, N), 7.0, device="cuda", dtype=dtype)
        out = memory[64:64 + R]
        ops.grouped_gemm_fp8(ops.W2, a, s, offsets, w, ws, num_tokens=R, top_k=1, num_experts=E, out=out)
        assert bool((memory[:64] == 7).all()) and bool((memory[64 + R:] == 7).all())
        known = torch.zeros(R, N, dtype=torch.bool, device="cuda")
        for e in allowed:
            known |= out == (values(a, s) @ weight_values(w[e], ws[e]).t()).to(F32).to(dtype)
        assert bool(known.all())
