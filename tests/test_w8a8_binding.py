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


def routers(library):
    return [args[1]._obj for name, args in library.calls if name == "moe_route_scored"]


def test_a_router_goes_by_values_not_by_the_objects_that_held_them(library):
    """A number given as a tensor of no dimensions is read at each call, and -0.0 is another factor than 0.0."""
    logits = torch.zeros(3, 16)
    scale, groups, k = torch.tensor(2.0), torch.tensor(4), torch.tensor(2)
    ops.route_scored(logits, k, scale=scale, num_groups=groups, topk_groups=2)
    scale.fill_(3.0)
    groups.fill_(2)
    k.fill_(3)
    ids, w = ops.route_scored(logits, k, scale=scale, num_groups=groups, topk_groups=2)
    assert ids.shape == w.shape == (3, 3)
    first, second = routers(library)
    assert (first.scale, first.num_groups, second.scale, second.num_groups) == (2.0, 4, 3.0, 2)
    shapes = [args[0]._obj for _, args in library.calls]
    assert [s.top_k for s in shapes] == [2, 3]
    for factor in (0.0, -0.0, 0.0):
        ops.route_scored(logits, 2, scale=factor)
    assert [str(r.scale) for r in routers(library)[2:]] == ["0.0", "-0.0", "0.0"]


def test_a_shape_goes_by_values_too(library):
    a, s, off = torch.zeros(6, 128, dtype=torch.int8), torch.ones(6), torch.zeros(3, dtype=torch.int32)
    w, ws = torch.zeros(2, 256, 128, dtype=torch.int8), torch.ones(2, 256)
    T, E = torch.tensor(3), torch.tensor(2)
    ops.grouped_gemm_w8a8(ops.W13_SWIGLU, a, s, off, w, ws, num_tokens=T, top_k=2, num_experts=E)
    T.fill_(6)
    E.fill_(8)
    ops.grouped_gemm_w8a8(ops.W13_SWIGLU, a, s, off, w, ws, num_tokens=T, top_k=1, num_experts=E)
    begin, E = torch.tensor(0), torch.tensor(4)
    x, ids, tw = torch.zeros(6, 128, dtype=torch.int8), torch.zeros(6, 2, dtype=torch.int32), torch.ones(6, 2)
    w2, w2s = torch.zeros(2, 128, 128, dtype=torch.int8), torch.ones(2, 128)
    layer = (x, s, ids, tw, w, ws, w2, w2s)
    space = torch.empty(256, dtype=torch.uint8)
    ops.moe_w8a8_forward(*layer, num_experts=E, expert_begin=begin, workspace=space)
    begin.fill_(2)
    ops.moe_w8a8_forward(*layer, num_experts=E, expert_begin=begin, workspace=space)
    got = [args[0]._obj for name, args in library.calls]
    assert [(s.num_tokens, s.num_experts, s.expert_begin) for s in got] == [(3, 2, 0), (6, 8, 0), (6, 4, 0), (6, 4, 2)]


class Stream:
    """Stands for a torch.cuda.Stream of a device."""

    def __init__(self, index):
        self.device_index = index
        self.device = torch.device("cuda", index)


def test_a_stream_of_another_device_is_refused(monkeypatch):
    """What ran there instead was the current stream of the tensors' device, without a word."""
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: ("on", s))
    monkeypatch.setattr(ops, "_on_gpu", lambda t, name: 0)
    here, other = Stream(0), Stream(1)
    assert ops._elsewhere(0, here) == ("on", here)
    x, w = torch.zeros(2, 128, dtype=torch.bfloat16), torch.ones(128, dtype=torch.bfloat16)
    q, s, ids = torch.zeros(2, 128, dtype=torch.int8), torch.ones(2), torch.zeros(2, 1, dtype=torch.int32)
    off, w3, ws3 = torch.zeros(2, dtype=torch.int32), torch.zeros(1, 256, 128, dtype=torch.int8), torch.ones(1, 256)
    for call in (lambda: ops.rms_norm(x, w, stream=other), lambda: ops.add_rms_norm(x, x, w, stream=other),
                 lambda: ops.rms_norm_int8(x, w, stream=other), lambda: ops.add_rms_norm_int8(x, x, w, stream=other),
                 lambda: ops.int8_quantize(x, stream=other), lambda: ops.route_scored(x.float(), 2, stream=other),
                 lambda: ops.dense_gemm_w8a8(q, s, w3[0], ws3[0], stream=other),
                 lambda: ops.grouped_gemm_w8a8(ops.W13_SWIGLU, q, s, off, w3, ws3, num_tokens=2, top_k=1, stream=other),
                 lambda: ops.moe_w8a8_forward(q, s, ids, ids.float(), w3, ws3, w3, ws3, stream=other)):
        with pytest.raises(ValueError, match="stream"):
            call()
