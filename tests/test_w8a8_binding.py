"""What the Python side of the W8A8 operators and the scored router checks and passes on, without a GPU: host tensors
stand for device ones, and a recorder for the library."""
import pytest
import torch

from w4a16_grouped_gemm_amd import ops


class Recorder:
    """Stands for the library: the calls it gets, with success as the answer."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def library(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(ops, "_lib", r)
    monkeypatch.setattr(ops, "_on_gpu", lambda t, name: t.get_device())
    monkeypatch.setattr(ops, "_elsewhere", lambda index, stream: None)
    monkeypatch.setattr(ops, "_empty", lambda size, stride, dtype: torch.empty_strided(size, stride, dtype=dtype))
    monkeypatch.setattr(ops, "_current_stream", lambda index: 0)
    return r


def grouped(kind, E=2, N=256, K=128, T=3, k=2):
    a_rows = T * k
    return ops.grouped_gemm_w8a8(kind, torch.zeros(a_rows, K, dtype=torch.int8), torch.ones(a_rows),
                                 torch.zeros(E + 1, dtype=torch.int32), torch.zeros(E, N, K, dtype=torch.int8),
                                 torch.ones(E, N), num_tokens=T, top_k=k)


def test_grouped_refuses_a_row_without_its_half(library):
    """A gate row belongs to an up row: weights with an odd number of rows are not two halves."""
    for kind in (ops.W13_SWIGLU, ops.W13_RAW):
        with pytest.raises(ValueError):
            grouped(kind, N=257)
    assert not library.calls
    assert grouped(ops.W13_SWIGLU).shape == (6, 128) and grouped(ops.W13_RAW).shape == (6, 256)
    assert grouped(ops.W2, N=128, K=256).shape == (6, 128)
    assert [name for name, _ in library.calls] == ["moe_grouped_gemm_w8a8"] * 3


def test_grouped_refuses_other_shapes(library):
    a, s, off = torch.zeros(6, 128, dtype=torch.int8), torch.ones(6), torch.zeros(3, dtype=torch.int32)
    w, ws = torch.zeros(2, 256, 128, dtype=torch.int8), torch.ones(2, 256)
    kw = dict(num_tokens=3, top_k=2)
    for args, more in [((a[:5], s, off, w, ws), {}), ((a, s[:5], off, w, ws), {}), ((a, s, off[:2], w, ws), {}),
                       ((a, s, off, w[0], ws), {}), ((a, s, off, w, ws[:, :128]), {}), ((a, s, off.long(), w, ws), {}),
                       ((a, s, off, w, ws), dict(a_row_index=torch.zeros(5, dtype=torch.int32))),
                       ((a, s, off, w, ws), dict(out=torch.zeros(6, 256, dtype=torch.bfloat16))),
                       ((a, s, off, w, ws), dict(out_dtype=torch.float16))]:
        with pytest.raises(ValueError):
            ops.grouped_gemm_w8a8(ops.W13_SWIGLU, *args, **{**kw, **more})
    assert not library.calls
