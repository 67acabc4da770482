"""The FP8 entry points refuse bad calls on the host, before any launch (CPU only)."""
import ctypes

import pytest
import torch

from w4a16_grouped_gemm_amd import ops

P = ctypes.c_void_p
A = P(1 << 20)                       # never dereferenced: every call below ends in the validation
NULL, SHAPE, UNSUPPORTED, ALIGN, WORKSPACE = 1, 2, 3, 4, 5


def at(n):
    return P((1 << 20) + n)


@pytest.fixture(scope="module")
def lib():
    return ops.load_library()


def shape(T=4, H=256, I=512, E=8, L=8, k=2, begin=0, group=128, layout=0):
    return ctypes.byref(ops.make_shape(T, H, I, E, L, k, begin, group, layout))


def test_norm(lib):
    f = lib.moe_rms_norm_fp8
    x, r, w, s, y, q, qs = [P((i + 1) << 40) for i in range(7)]
    assert f(0, 256, None, None, None, 1e-6, 0, None, None, None, None, None) == 0
    for rows, K, eps in [(-1, 256, 1e-6), (4, 0, 1e-6), (4, 192, 1e-6), (4, 264, 1e-6), (4, 65664, 1e-6), (4, 256, -1.0),
                         (4, 256, float("nan"))]:
        assert f(rows, K, x, None, w, eps, 0, None, None, q, qs, None) == SHAPE, (rows, K, eps)
    assert f(1 << 25, 128, x, None, w, 1e-6, 0, None, None, q, qs, None) == UNSUPPORTED
    for args in [(None, None, w, None, None, q, qs), (x, None, None, None, None, q, qs), (x, None, w, None, y, None, qs),
                 (x, None, w, None, y, q, None), (x, r, w, None, None, q, qs), (x, None, w, s, None, q, qs)]:
        assert f(4, 256, *args[:3], 1e-6, 0, *args[3:], None) == NULL, args
    assert f(4, 256, P((1 << 40) + 8), None, w, 1e-6, 0, None, None, q, qs, None) == ALIGN
    assert f(4, 256, x, None, w, 1e-6, 0, None, None, P((6 << 40) + 8), qs, None) == ALIGN
    assert f(4, 256, x, None, w, 1e-6, 0, None, None, q, P((7 << 40) + 2), None) == ALIGN
    assert f(4, 256, x, r, w, 1e-6, 0, P((1 << 40) + 512), None, q, qs, None) == UNSUPPORTED   # a shifted overlap
    assert f(4, 256, x, r, w, 1e-6, 0, s, s, q, qs, None) == UNSUPPORTED                       # two outputs in one place
    assert f(4, 256, x, None, w, 1e-6, 0, None, None, x, qs, None) == UNSUPPORTED              # codes over x
    assert f(4, 256, x, None, w, 1e-6, 0, None, None, q, P((6 << 40) + 1020), None) == UNSUPPORTED   # scales over codes
    assert f(4, 256, x, None, w, 1e-6, 0, None, w, q, qs, None) == UNSUPPORTED                 # over the gains


def test_quantize(lib):
    f = lib.moe_fp8_quantize
    x, q, s = P(1 << 40), P(2 << 40), P(3 << 40)
    assert f(0, 256, None, 0, None, None, None) == 0
    for rows, K in [(-1, 256), (4, 64), (4, 200), (4, 65664)]:
        assert f(rows, K, x, 0, q, s, None) == SHAPE
    assert f(1 << 25, 128, x, 0, q, s, None) == UNSUPPORTED
    assert f(4, 256, None, 0, q, s, None) == NULL
    assert f(4, 256, x, 0, None, s, None) == NULL
    assert f(4, 256, x, 0, q, None, None) == NULL
    assert f(4, 256, x, 0, P((2 << 40) + 4), s, None) == ALIGN
    assert f(4, 256, x, 0, q, P((3 << 40) + 2), None) == ALIGN
    assert f(4, 256, x, 0, x, s, None) == UNSUPPORTED
    assert f(4, 256, x, 0, q, q, None) == UNSUPPORTED
    assert f(4, 256, x, 0, q, P((1 << 40) + 2044), None) == UNSUPPORTED


def test_weights(lib):
    f = lib.moe_fp8_quantize_weights
    w, q, s = P(1 << 40), P(2 << 40), P(3 << 40)
    assert f(0, 16, 256, None, 0, None, None, None) == 0 and f(3, 0, 256, None, 0, None, None, None) == 0
    for E, N, K in [(-1, 16, 256), (1, -1, 256), (1, 16, 192), (1, 16, 0), (1, 262145, 128), (1, 16, 65664)]:
        assert f(E, N, K, w, 0, q, s, None) == SHAPE, (E, N, K)
    assert f(1 << 24, 16, 128, w, 0, q, s, None) == UNSUPPORTED
    assert f(20000, 4096, 4096, w, 0, q, s, None) == UNSUPPORTED
    assert f(1, 16, 256, None, 0, q, s, None) == NULL
    assert f(1, 16, 256, w, 0, q, None, None) == NULL
    assert f(1, 16, 256, P((1 << 40) + 8), 0, q, s, None) == ALIGN
    assert f(1, 16, 256, w, 0, w, s, None) == UNSUPPORTED


def test_dense(lib):
    f = lib.moe_fp8_dense_gemm
    assert f(0, 256, 256, None, None, None, None, None, 0, None) == 0
    for M, N, K in [(-1, 256, 256), (4, 8, 256), (4, 200, 256), (4, 256, 64), (4, 256, 192), (4, 262160, 128),
                    (4, 256, 65664)]:
        assert f(M, N, K, A, A, A, A, A, 0, None) == SHAPE, (M, N, K)
    assert f(4, 65536, 65536, A, A, A, A, A, 0, None) == UNSUPPORTED
    assert f(1 << 24, 256, 128, A, A, A, A, A, 0, None) == UNSUPPORTED
    assert f(1 << 23, 8192, 128, A, A, A, A, A, 0, None) == UNSUPPORTED
    assert f(4, 256, 256, A, A, A, A, A, 7, None) == UNSUPPORTED
    assert f(4, 256, 256, A, None, A, A, A, 0, None) == NULL
    assert f(4, 256, 256, at(8), A, A, A, A, 0, None) == ALIGN
    assert f(4, 256, 256, A, A, A, at(2), A, 0, None) == ALIGN


def test_grouped(lib):
    f = lib.moe_grouped_gemm_fp8
    assert f(shape(T=0), 0, None, None, None, None, None, None, None, 0, None) == 0
    assert f(None, 0, A, A, A, A, A, A, A, 0, None) == NULL
    assert f(shape(group=0), 0, A, A, A, A, A, A, A, 0, None) == UNSUPPORTED
    assert f(shape(group=32), 0, A, A, A, A, A, A, A, 0, None) == UNSUPPORTED
    assert f(shape(layout=1), 0, A, A, A, A, A, A, A, 0, None) == UNSUPPORTED
    assert f(shape(H=200), 0, A, A, A, A, A, A, A, 0, None) == SHAPE
    assert f(shape(k=9), 0, A, A, A, A, A, A, A, 0, None) == SHAPE
    assert f(shape(), 3, A, A, A, A, A, A, A, 0, None) == UNSUPPORTED
    assert f(shape(), 0, A, A, A, A, A, A, A, 1, None) == UNSUPPORTED      # SwiGLU gives bf16
    assert f(shape(), 1, A, A, None, A, A, A, None, 1, None) == NULL
    assert f(shape(), 1, A, A, at(2), A, A, A, A, 1, None) == ALIGN


def test_layer(lib):
    f, size = lib.moe_fp8_forward, lib.moe_fp8_workspace_size
    assert size(shape(group=0)) == 0 and size(shape(H=100)) == 0 and size(None) == 0
    need = size(shape())
    assert need > 4 * 2 * (512 + 256 * 2)
    big = 1 << 40
    assert f(shape(T=0), None, None, None, None, None, None, None, None, 0, None, None, 0, None) == 0
    assert f(shape(), A, A, A, A, A, A, A, A, 0, A, A, need - 1, None) == WORKSPACE
    assert f(shape(), A, A, A, A, A, A, A, A, 0, A, None, big, None) == NULL
    assert f(shape(), A, A, None, A, A, A, A, A, 0, A, A, big, None) == NULL
    assert f(shape(), A, A, A, A, A, at(2), A, A, 0, A, A, big, None) == ALIGN
    assert f(shape(), A, A, A, A, A, A, A, A, 0, A, at(16), big, None) == ALIGN
    assert f(shape(group=32), A, A, A, A, A, A, A, A, 0, A, A, big, None) == UNSUPPORTED


def test_binding_refuses_host_tensors_and_types():
    x, w = torch.zeros(4, 256, dtype=torch.bfloat16), torch.ones(256, dtype=torch.bfloat16)
    q, s = x.to(torch.float8_e4m3fn), torch.ones(4, 2)
    off, ids = torch.zeros(2, dtype=torch.int32), torch.zeros(4, 1, dtype=torch.int32)
    for call in (lambda: ops.fp8_quantize(x), lambda: ops.fp8_quantize(x.float()), lambda: ops.fp8_quantize_weights(x),
                 lambda: ops.rms_norm_fp8(x, w), lambda: ops.add_rms_norm_fp8(x, x, w),
                 lambda: ops.add_rms_norm_fp8(x, None, w), lambda: ops.dense_gemm_fp8(q, s, q, s),
                 lambda: ops.grouped_gemm_fp8(ops.W2, q, s, off, q[None], s[None], num_tokens=4, top_k=1),
                 lambda: ops.moe_fp8_forward(q, s, ids, ids.float(), q[None], s[None], q[None], s[None])):
        with pytest.raises(ValueError):
            call()
