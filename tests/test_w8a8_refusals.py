"""The W8A8 entry points, the norm and the scored router refuse bad calls on the host, before any launch (CPU only)."""
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


def shape(T=4, H=256, I=512, E=8, L=8, k=2, begin=0, group=0, layout=0):
    return ctypes.byref(ops.make_shape(T, H, I, E, L, k, begin, group, layout))


def test_norm(lib):
    f = lib.moe_rms_norm
    far = [P((i + 1) << 40) for i in range(7)]
    x, r, w, s, y, q, qs = far
    assert f(0, 256, None, None, None, 1e-6, None, None, None, None, None) == 0
    assert f(-1, 256, x, None, w, 1e-6, None, y, None, None, None) == SHAPE
    assert f(4, 4, x, None, w, 1e-6, None, y, None, None, None) == SHAPE
    assert f(4, 260, x, None, w, 1e-6, None, y, None, None, None) == SHAPE
    assert f(4, 65544, x, None, w, 1e-6, None, y, None, None, None) == SHAPE
    assert f(4, 256, x, None, w, -1.0, None, y, None, None, None) == SHAPE
    assert f(4, 256, x, None, w, float("nan"), None, y, None, None, None) == SHAPE
    assert f(1 << 31, 8, x, None, w, 1e-6, None, y, None, None, None) == UNSUPPORTED
    assert f(4, 256, None, None, w, 1e-6, None, y, None, None, None) == NULL
    assert f(4, 256, x, None, w, 1e-6, None, None, None, None, None) == NULL          # no output
    assert f(4, 256, x, r, w, 1e-6, None, y, None, None, None) == NULL                # residual without its sum
    assert f(4, 256, x, None, w, 1e-6, s, y, None, None, None) == NULL
    assert f(4, 256, x, None, w, 1e-6, None, None, q, None, None) == NULL             # codes without scales
    assert f(4, 256, P((1 << 40) + 8), None, w, 1e-6, None, y, None, None, None) == ALIGN
    assert f(4, 256, x, r, w, 1e-6, P((1 << 40) + 512), y, None, None, None) == UNSUPPORTED   # a shifted overlap
    assert f(4, 256, x, r, w, 1e-6, s, s, None, None, None) == UNSUPPORTED            # two outputs in one place
    assert f(4, 256, x, None, w, 1e-6, None, None, x, qs, None) == UNSUPPORTED        # codes over x
    assert f(4, 256, x, None, w, 1e-6, None, w, None, None, None) == UNSUPPORTED      # over the weights


def test_quantize(lib):
    f = lib.moe_int8_quantize
    x, q, s = P(1 << 40), P(2 << 40), P(3 << 40)
    assert f(0, 256, None, None, None, None) == 0
    assert f(4, 12, x, q, s, None) == SHAPE
    assert f(-1, 256, x, q, s, None) == SHAPE
    assert f(4, 65544, x, q, s, None) == SHAPE
    assert f(4, 256, x, None, s, None) == NULL
    assert f(4, 256, x, P((2 << 40) + 4), s, None) == ALIGN
    assert f(4, 256, x, x, s, None) == UNSUPPORTED
    assert f(4, 256, x, q, q, None) == UNSUPPORTED


def test_dense(lib):
    f = lib.moe_w8a8_dense_gemm
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
    assert f(4, 256, 256, A, A, A, at(4), A, 0, None) == ALIGN


def test_grouped(lib):
    f = lib.moe_grouped_gemm_w8a8
    assert f(shape(T=0), 0, None, None, None, None, None, None, None, 0, None) == 0
    assert f(None, 0, A, A, A, A, A, A, A, 0, None) == NULL
    assert f(shape(group=128), 0, A, A, A, A, A, A, A, 0, None) == UNSUPPORTED
    assert f(shape(layout=1), 0, A, A, A, A, A, A, A, 0, None) == UNSUPPORTED
    assert f(shape(H=200), 0, A, A, A, A, A, A, A, 0, None) == SHAPE
    assert f(shape(k=9), 0, A, A, A, A, A, A, A, 0, None) == SHAPE
    assert f(shape(), 3, A, A, A, A, A, A, A, 0, None) == UNSUPPORTED
    assert f(shape(), 0, A, A, A, A, A, A, A, 1, None) == UNSUPPORTED      # SwiGLU gives bf16
    assert f(shape(), 1, A, A, None, A, A, A, None, 1, None) == NULL
    assert f(shape(), 1, A, A, at(2), A, A, A, A, 1, None) == ALIGN


def test_layer(lib):
    f, size = lib.moe_w8a8_forward, lib.moe_w8a8_workspace_size
    assert size(shape(group=128)) == 0 and size(shape(H=100)) == 0 and size(None) == 0
    need = size(shape())
    assert need > 4 * 2 * (512 * 3 + 256 * 2)
    big = 1 << 40
    assert f(shape(T=0), None, None, None, None, None, None, None, None, None, None, 0, None) == 0
    assert f(shape(), A, A, A, A, A, A, A, A, A, A, need - 1, None) == WORKSPACE
    assert f(shape(), A, A, A, A, A, A, A, A, A, None, big, None) == NULL
    assert f(shape(), A, A, None, A, A, A, A, A, A, A, big, None) == NULL
    assert f(shape(), A, A, A, A, A, at(8), A, A, A, A, big, None) == ALIGN
    assert f(shape(), A, A, A, A, A, A, A, A, A, at(16), big, None) == ALIGN
    assert f(shape(group=32), A, A, A, A, A, A, A, A, A, A, big, None) == UNSUPPORTED


def test_router(lib):
    f = lib.moe_route_scored

    def call(sh, score=1, G=1, kept=1, top=1, renorm=1, scale=1.0, logits=A, ids=A):
        r = ops.Router(score, G, kept, top, renorm, scale)
        return f(sh, ctypes.byref(r), logits, None, ids, A, None)

    sh = shape(H=128, I=128, group=128)
    assert call(shape(T=0, H=128, I=128, group=128), logits=None) == 0
    assert f(sh, None, A, None, A, A, None) == NULL
    assert call(sh, score=2) == UNSUPPORTED
    assert call(sh, G=0) == SHAPE and call(sh, G=3) == SHAPE
    assert call(sh, G=4, kept=0) == SHAPE and call(sh, G=4, kept=5) == SHAPE
    assert call(sh, G=4, kept=2, top=3) == UNSUPPORTED
    assert call(sh, G=8, kept=2, top=2) == SHAPE                           # groups of one expert
    assert call(shape(H=128, I=128, k=3, group=128), G=4, kept=1) == SHAPE   # fewer experts than slots
    wide = shape(H=128, I=128, E=256, L=256, group=128)
    assert call(wide, G=128, kept=4) == UNSUPPORTED
    assert call(sh, logits=None) == NULL
    assert call(sh, ids=at(2)) == ALIGN


def test_binding_refuses_host_tensors_and_types():
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    w = torch.ones(256, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ops.rms_norm(x, w)
    with pytest.raises(ValueError):
        ops.rms_norm(x.float(), w)
    with pytest.raises(ValueError):
        ops.add_rms_norm(x, None, w)
    with pytest.raises(ValueError):
        ops.int8_quantize(x)
    with pytest.raises(ValueError):
        ops.route_scored(torch.zeros(4, 8), 2)
    with pytest.raises(ValueError):
        ops.dense_gemm_w8a8(x.to(torch.int8), torch.ones(4), torch.zeros(16, 256, dtype=torch.int8), torch.ones(16))
