"""What the Python side of the FP8 operators checks and passes on, without a GPU: host tensors stand for device ones,
and a recorder for the library."""
import pytest
import torch

from test_w8a8_binding import Stream, library   # noqa: F401  (a fixture)
from w4a16_grouped_gemm_amd import ops

FP8, B16 = torch.float8_e4m3fn, torch.bfloat16


def q(*shape):
    return torch.zeros(shape, dtype=FP8)


def grouped(kind, E=2, N=256, K=128, T=3, k=2, **kw):
    args = dict(a=q(T * k, K), s=torch.ones(T * k, K // 128), off=torch.zeros(E + 1, dtype=torch.int32), w=q(E, N, K),
                ws=torch.ones(E, N // 128, K // 128))
    args.update(kw)
    more = args.pop("more", {})
    return ops.grouped_gemm_fp8(kind, *args.values(), num_tokens=T, top_k=k, **more)


def test_grouped_refuses_other_shapes(library):   # noqa: F811
    for kind in (ops.W13_SWIGLU, ops.W13_RAW):
        with pytest.raises(ValueError):
            grouped(kind, N=257)
    for kw in [dict(a=q(5, 128)), dict(s=torch.ones(5, 1)), dict(s=torch.ones(6)), dict(off=torch.zeros(2, dtype=torch.int32)),
               dict(w=q(256, 128)), dict(ws=torch.ones(2, 256)), dict(ws=torch.ones(2, 1, 1)),
               dict(off=torch.zeros(3, dtype=torch.int64)), dict(a=torch.zeros(6, 128, dtype=torch.int8)),
               dict(more=dict(a_row_index=torch.zeros(5, dtype=torch.int32))),
               dict(more=dict(out=torch.zeros(6, 256, dtype=B16))), dict(more=dict(out_dtype=torch.float16))]:
        with pytest.raises(ValueError):
            grouped(ops.W13_SWIGLU, **kw)
    assert not library.calls
    assert grouped(ops.W13_SWIGLU).shape == (6, 128) and grouped(ops.W13_RAW).shape == (6, 256)
    assert grouped(ops.W2, N=128, K=256).shape == (6, 128)
    assert [name for name, _ in library.calls] == ["moe_grouped_gemm_fp8"] * 3


def test_dense_refuses_other_shapes(library):   # noqa: F811
    a, s, w, ws = q(3, 256), torch.ones(3, 2), q(144, 256), torch.ones(2, 2)
    for args in [(a, s[:2], w, ws), (a, s[:, :1], w, ws), (a, s, w, ws[:1]), (a, s, w[:, :128], ws), (a[0], s, w, ws),
                 (a, s.double(), w, ws), (a.to(torch.float32), s, w, ws), (a, torch.ones(2, 3).t(), w, ws)]:
        with pytest.raises(ValueError):
            ops.dense_gemm_fp8(*args)
    assert not library.calls
    assert ops.dense_gemm_fp8(a, s, w, ws, out_dtype=torch.float32).shape == (3, 144)
    (name, args), = library.calls
    assert name == "moe_fp8_dense_gemm" and args[:3] == (3, 144, 256) and args[8] == ops.MOE_F32


def test_rows_of_whole_blocks_only(library):   # noqa: F811
    for K in (0, 64, 200):
        x, w = torch.zeros(2, K, dtype=B16), torch.ones(K, dtype=B16)
        for call in (lambda: ops.fp8_quantize(x), lambda: ops.rms_norm_fp8(x, w), lambda: ops.add_rms_norm_fp8(x, x, w),
                     lambda: ops.fp8_quantize_weights(x)):
            with pytest.raises(ValueError):
                call()
    for bad in (torch.zeros((), dtype=B16), torch.zeros(2, 256), torch.zeros(256, 2, dtype=B16).t()):
        with pytest.raises(ValueError):
            ops.fp8_quantize(bad)
    with pytest.raises(ValueError):
        ops.fp8_quantize_weights(torch.zeros(128, dtype=B16))
    assert not library.calls


def test_a_shape_goes_by_values(library):   # noqa: F811
    T, E = torch.tensor(3), torch.tensor(2)
    a, s, off, w, ws = q(6, 128), torch.ones(6, 1), torch.zeros(3, dtype=torch.int32), q(2, 256, 128), torch.ones(2, 2, 1)
    ops.grouped_gemm_fp8(ops.W13_SWIGLU, a, s, off, w, ws, num_tokens=T, top_k=2, num_experts=E)
    T.fill_(6)
    E.fill_(8)
    ops.grouped_gemm_fp8(ops.W13_SWIGLU, a, s, off, w, ws, num_tokens=T, top_k=1, num_experts=E)
    begin, E = torch.tensor(0), torch.tensor(4)
    ids, space = torch.zeros(6, 2, dtype=torch.int32), torch.empty(256, dtype=torch.uint8)
    layer = (a, s, ids, ids.float(), w, ws, q(2, 128, 128), torch.ones(2, 1, 1))
    ops.moe_fp8_forward(*layer, num_experts=E, expert_begin=begin, workspace=space)
    begin.fill_(2)
    ops.moe_fp8_forward(*layer, num_experts=E, expert_begin=begin, workspace=space, pow2=True)
    got = [args[0]._obj for name, args in library.calls]
    assert [(s.num_tokens, s.num_experts, s.expert_begin, s.group_size) for s in got] == [
        (3, 2, 0, 128), (6, 8, 0, 128), (6, 4, 0, 128), (6, 4, 2, 128)]
    assert [args[9] for name, args in library.calls[2:]] == [False, True]


def test_a_stream_of_another_device_is_refused(monkeypatch):
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(ops, "_on_gpu", lambda t, name: 0)
    other = Stream(1)
    x, w = torch.zeros(2, 128, dtype=B16), torch.ones(128, dtype=B16)
    a, s, ids, off = q(2, 128), torch.ones(2, 1), torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    w3, ws3 = q(1, 256, 128), torch.ones(1, 2, 1)
    for call in (lambda: ops.rms_norm_fp8(x, w, stream=other), lambda: ops.add_rms_norm_fp8(x, x, w, stream=other),
                 lambda: ops.fp8_quantize(x, stream=other), lambda: ops.fp8_quantize_weights(x, stream=other),
                 lambda: ops.dense_gemm_fp8(a, s, w3[0], ws3[0], stream=other),
                 lambda: ops.grouped_gemm_fp8(ops.W13_SWIGLU, a, s, off, w3, ws3, num_tokens=2, top_k=1, stream=other),
                 lambda: ops.moe_fp8_forward(a, s, ids, ids.float(), w3, ws3, w3, ws3, stream=other)):
        with pytest.raises(ValueError, match="stream"):
            call()
