"""What the binding of include/e2ttt_layer.h refuses before it calls the library.
No GPU is needed: the tensors are fake ones, which have a device and no memory."""
import contextlib
from types import SimpleNamespace

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import chunk_weight_rnn_amd as e2


@pytest.fixture
def t():
    """Arguments of every operator, on cuda:0."""
    with FakeTensorMode():
        z = lambda *s, d=torch.float32: torch.empty(*s, device="cuda", dtype=d)
        yield SimpleNamespace(z=z, q=z(8, 4, 64), k=z(8, 2, 64), lse=z(8, 4), cu=z(3, d=torch.int32),
                              cache=z(5, 2, 16, 64), table=z(2, 3, d=torch.int32), cached=z(2, d=torch.int32),
                              x=z(6, 32), w=z(32), rstd=z(6))


def calls(t):
    return [lambda **a: e2.attention_forward(t.q, t.k, t.k, t.cu, **a),
            lambda **a: e2.attention_backward(t.q, t.k, t.k, t.q, t.lse, t.q, t.cu, **a),
            lambda **a: e2.paged_attention(t.q, t.k, t.k, t.cache, t.cache, t.table, t.cu, t.cached, **a),
            lambda **a: e2.norm_forward(t.x, t.w, **a),
            lambda **a: e2.norm_backward(t.x, t.x, t.w, t.rstd, **a)]


def test_a_stream_of_another_device_is_refused(t, monkeypatch):
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    other = SimpleNamespace(device=torch.device("cuda", 1))
    for call in calls(t):
        with pytest.raises(ValueError, match="stream must be on the tensors' device"):
            call(stream=other)


def test_cpu_tensors_are_refused_with_a_stream_too():
    s = SimpleNamespace(device=torch.device("cuda", 0))
    x = torch.zeros(2, 4)
    with pytest.raises(ValueError, match="GPU"):
        e2.norm_forward(x, x[0], stream=s)


def test_a_workspace_with_gaps_or_repeats_is_refused(t):
    for ws in (t.z(1, d=torch.uint8).expand(1 << 24), t.z(1 << 24, 2, d=torch.uint8)[:, 0]):
        for i in (0, 1, 2, 4):
            with pytest.raises(ValueError, match="workspace must be contiguous"):
                calls(t)[i](workspace=ws)
