"""Captures beside live eager graphs on the GPU: gradients behind a projection are refused in
the forward of the lookup and the recurrence, and forwards alone of the other operators are
captured as ever."""
import pytest
import torch

from tests.gpu_util import note
from tests.test_gpu_model_streams import _cu, _same

pytestmark = pytest.mark.gpu


def _setup():
    g = torch.Generator(device="cuda").manual_seed(8)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x, weight, inp = r(300, 64).bfloat16(), r(64).requires_grad_(), (r(64, 128) / 8).requires_grad_()
    return x, weight, inp, _cu([100, 200])


def test_leaves_behind_a_projection_are_refused():
    note("a capture of the recurrence behind a projection, beside a live graph")
    import chunk_weight_rnn_amd as e2
    x, weight, inp, cu = _setup()

    def forward():
        y, _ = e2.rms_norm(x, weight)
        z = y.float() @ inp
        return e2.gated_scan(z[:, :64].contiguous(), torch.sigmoid(z[:, 64:]).contiguous(), cu)[0]

    def grads():
        return torch.autograd.grad(forward().square().sum(), (weight, inp))

    want = grads()
    alive = forward()
    torch.cuda.synchronize()
    with pytest.raises(RuntimeError, match="another stream"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            forward()
    del alive
    got = grads()
    torch.cuda.synchronize()
    assert _same(got, want)


def test_forwards_alone_are_captured_beside_a_live_graph():
    note("captured forwards beside a live graph")
    import chunk_weight_rnn_amd as e2
    x, weight, inp, cu = _setup()

    def forward():
        y, _ = e2.rms_norm(x, weight)
        q = y.view(300, 1, 64)
        return y, e2.attention(q, q, q, cu)

    alive = forward()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        forward()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = forward()
    for _ in range(3):
        graph.replay()
        torch.randn(1 << 20, device="cuda").sum().item()
        assert _same([t.detach() for t in held], [t.detach() for t in alive])
