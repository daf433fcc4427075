"""What the Python binding of the operators around a hybrid model's layers refuses
before it calls the library.  No GPU is needed: the tensors are fake ones, which have
a device and no memory."""
import contextlib
from types import SimpleNamespace

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import chunk_weight_rnn_amd as e2

BF, F32, I32, I64 = torch.bfloat16, torch.float32, torch.int32, torch.int64
F8, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu


@pytest.fixture
def z():
    with FakeTensorMode():
        yield lambda *s, d=F32: torch.empty(*s, device="cuda", dtype=d)


def calls(z):
    cu = z(3, d=I32)
    return [lambda **a: e2.gated_scan_forward(z(600, 32), z(600, 32), cu, **a),
            lambda **a: e2.gated_scan_backward(z(600, 32), z(600, 32), z(600, 32), z(6, 32), cu, **a),
            lambda **a: e2.embedding_forward(z(5, d=I64), z(9, 8), **a),
            lambda **a: e2.embedding_backward(z(5, 8), z(5, d=I64), 9, **a),
            lambda **a: e2.sample(z(4, 50), z(4), **a),
            lambda **a: e2.paged_attention(z(8, 4, 64, d=BF), None, None, z(5, 2, 16, 64, d=F8), z(5, 2, 16, 64, d=F8), z(2, 3, d=I32),
                                           cu, z(2, d=I32), k_scale=z(5, 2, 16, d=E8), v_scale=z(5, 2, 16, d=E8), **a)]


def test_a_stream_of_another_device_is_refused(z, monkeypatch):
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    for call in calls(z):
        with pytest.raises(ValueError, match="stream must be on the tensors' device"):
            call(stream=SimpleNamespace(device=torch.device("cuda", 1)))


def test_cpu_tensors_are_refused():
    c = torch.zeros
    for call in (lambda: e2.gated_scan_forward(c(4, 2), c(4, 2), c(2, dtype=I32)), lambda: e2.embedding_forward(c(3, dtype=I64), c(4, 2)),
                 lambda: e2.embedding_backward(c(3, 2), c(3, dtype=I64), 4), lambda: e2.sample(c(2, 5), c(2)),
                 lambda: e2.gated_scan(c(4, 2), c(4, 2), c(2, dtype=I32)), lambda: e2.embedding(c(3, dtype=I64), c(4, 2))):
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_a_workspace_with_gaps_or_repeats_is_refused(z):
    for ws in (z(1, d=torch.uint8).expand(1 << 24), z(1 << 24, 2, d=torch.uint8)[:, 0]):
        for i in (0, 1, 3):
            with pytest.raises(ValueError, match="workspace must be contiguous"):
                calls(z)[i](workspace=ws)


def refused(error, text, call):
    with pytest.raises(error, match=text):
        call()


def test_scan_arguments(z):
    x, cu = z(10, 8, d=BF), z(3, d=I32)
    f = e2.gated_scan_forward
    refused(ValueError, r"x must have shape", lambda: f(z(10), z(10), cu))
    refused(TypeError, "float32 or bfloat16", lambda: f(z(10, 8, d=torch.float16), z(10, 8), cu))
    refused(ValueError, "a must have shape", lambda: f(x, z(10, 7), cu))
    refused(TypeError, "a must be", lambda: f(z(10, 8), z(10, 8, d=BF), cu))
    refused(ValueError, "contiguous", lambda: f(z(8, 10, d=BF).t(), z(10, 8), cu))
    refused(ValueError, "cu_seqlens", lambda: f(x, z(10, 8), z(3, d=I64)))
    refused(ValueError, "cu_seqlens", lambda: f(x, z(10, 8), z(0, d=I32)))
    refused(ValueError, "h0 must have shape", lambda: f(x, z(10, 8), cu, h0=z(3, 8)))
    refused(TypeError, "h0 must be", lambda: f(x, z(10, 8), cu, h0=z(2, 8, d=BF)))
    refused(ValueError, "state must be contiguous", lambda: f(x, z(10, 8), cu, state=z(2, 16)[:, ::2]))
    refused(TypeError, "out must be", lambda: f(x, z(10, 8), cu, out=z(10, 8)))
    b = e2.gated_scan_backward
    refused(ValueError, "starts must have shape", lambda: b(x, x, z(10, 8), z(3, 8), cu))
    refused(TypeError, "dout must be", lambda: b(z(10, 8), x, z(10, 8), z(2, 8), cu))
    refused(ValueError, "dstate must have shape", lambda: b(x, x, z(10, 8), z(2, 8), cu, dstate=z(8)))


def test_embedding_arguments(z):
    t, w = z(5, d=I64), z(9, 8)
    refused(TypeError, "tokens must be int32 or int64", lambda: e2.embedding_forward(z(5), w))
    refused(ValueError, "weight must be", lambda: e2.embedding_forward(t, z(8)))
    refused(ValueError, "weight must be", lambda: e2.embedding_forward(t, z(8, 9).t()))
    refused(ValueError, "contiguous", lambda: e2.embedding_forward(z(5, 2, d=I64)[:, 0], w))
    refused(TypeError, "float32 or bfloat16", lambda: e2.embedding_forward(t, w, dtype=torch.float16))
    refused(ValueError, "out must have shape", lambda: e2.embedding_forward(t, w, out=z(5, 9)))
    refused(ValueError, "dout must have shape", lambda: e2.embedding_backward(z(4, 8), t, 9))
    refused(ValueError, "contiguous", lambda: e2.embedding_backward(z(8, 5).t(), t, 9))
    refused(TypeError, "out must be", lambda: e2.embedding_backward(z(5, 8), t, 9, out=z(9, 8, d=BF)))


def test_sample_arguments(z):
    x, u = z(4, 50), z(4)
    refused(ValueError, "logits must have shape", lambda: e2.sample(z(50), z(1)))
    refused(TypeError, "float32 or bfloat16", lambda: e2.sample(z(4, 50, d=torch.float64), u))
    refused(ValueError, "contiguous", lambda: e2.sample(z(50, 4).t(), u))
    refused(ValueError, "u must have shape", lambda: e2.sample(x, z(5)))
    refused(TypeError, "u must be", lambda: e2.sample(x, z(4, d=torch.float64)))
    refused(TypeError, "top_k must be", lambda: e2.sample(x, u, top_k=z(4, d=I64)))
    refused(ValueError, "top_p must have shape", lambda: e2.sample(x, u, top_p=z(1)))
    refused(TypeError, "temperature must be", lambda: e2.sample(x, u, temperature=z(4, d=BF)))
    refused(TypeError, "token must be", lambda: e2.sample(x, u, token=z(4, d=I32)))
    refused(ValueError, "logprob must have shape", lambda: e2.sample(x, u, logprob=z(3)))


def test_paged8_arguments(z):
    q, k, table, cu, cached = z(8, 4, 64, d=BF), z(8, 2, 64, d=BF), z(2, 3, d=I32), z(3, d=I32), z(2, d=I32)
    c8, s8 = z(5, 2, 16, 64, d=F8), z(5, 2, 16, d=E8)
    f = lambda kc=c8, vc=c8, ks=s8, vs=s8: e2.paged_attention(q, k, k, kc, vc, table, cu, cached, k_scale=ks, v_scale=vs)
    refused(ValueError, "both be given", lambda: f(vs=None))
    refused(TypeError, "must be torch.bfloat16", lambda: f(ks=None, vs=None))
    refused(TypeError, "must be torch.float8_e4m3fn", lambda: f(kc=z(5, 2, 16, 64, d=BF), vc=z(5, 2, 16, 64, d=BF)))
    refused(TypeError, "k_scale must be", lambda: f(ks=z(5, 2, 16)))
    refused(ValueError, "v_scale must have shape", lambda: f(vs=z(5, 16, 2, d=E8)))
    refused(ValueError, "k_scale must be contiguous", lambda: f(ks=z(5, 16, 2, d=E8).transpose(1, 2)))


def test_leaves_of_a_live_graph_are_refused_in_a_capture(monkeypatch):
    """The check behind embedding and gated_scan, on the CPU with the stream and the capture given."""
    from chunk_weight_rnn_amd import layer
    stream, capturing = [1], [False]
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: stream[0], raising=False)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing[0])
    w = torch.ones(3, requires_grad=True)
    alive = w * 2
    layer._one_stream(alive, 0)
    stream[0] = 2
    layer._one_stream(w * 3, 0)  # not captured: torch orders the streams
    capturing[0] = True
    with pytest.raises(RuntimeError, match="another stream"):
        layer._one_stream(w * 3, 0)
    layer._one_stream(torch.ones(3), 0)  # no gradients
    layer._one_stream((w * 2) * 3, 0)  # not a leaf
    del alive
    layer._one_stream(w * 3, 0)
