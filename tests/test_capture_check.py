"""The check that keeps a captured backward pass from leaves which an eager graph, still
alive, holds on another stream (CPU only: the streams are numbers, and whether one is being
captured is told).  Such a capture ends the process, so that only its refusal is run."""
import pytest
import torch

from chunk_weight_rnn_amd import layer


class Streams:
    now, capturing = 1, False


@pytest.fixture
def on(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: Streams.now, raising=False)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: Streams.capturing)

    def on(stream, capturing=False):
        Streams.now, Streams.capturing = stream, capturing
    on(1)
    return on


class Op(torch.autograd.Function):
    """An operator of a few tensors."""

    @staticmethod
    def forward(ctx, *xs):
        return sum(xs)

    @staticmethod
    def backward(ctx, g):
        return g, g


def leaf():
    return torch.randn(3, requires_grad=True)


def test_leaves_given_directly(on):
    w, x = leaf(), leaf()
    alive = Op.apply(w, x)
    layer._one_stream_behind(alive, 0)
    on(2, True)
    with pytest.raises(RuntimeError, match="another stream"):
        layer._one_stream_behind(Op.apply(leaf(), w), 0)
    del alive  # the graph goes, and what it knew of its leaves
    layer._one_stream_behind(Op.apply(leaf(), w), 0)


def test_leaves_behind_other_operations(on):
    """A projection's weight stands between the call and the leaf that an eager call was given."""
    w, p = leaf(), leaf()
    alive = Op.apply(w, leaf())
    layer._mark_leaves(alive, 0)
    on(2, True)
    with pytest.raises(RuntimeError, match="another stream"):
        layer._one_stream_behind(Op.apply((w * 2).exp() * p, leaf()), 0)


def test_one_stream_and_eager_calls_pass(on):
    w = leaf()
    alive = [Op.apply(w, leaf())]
    layer._one_stream_behind(alive[0], 0)
    on(1, True)  # the same stream
    layer._one_stream_behind(Op.apply(w * 2, leaf()), 0)
    on(2)  # no capture
    layer._one_stream_behind(Op.apply(w * 2, leaf()), 0)
    on(2, True)
    layer._one_stream_behind(Op.apply(leaf() * 2, leaf()), 0)  # other leaves


def test_nothing_to_differentiate(on):
    on(1, True)
    layer._one_stream_behind(torch.zeros(3), 0)
    with torch.no_grad():
        layer._one_stream_behind(Op.apply(leaf(), leaf()), 0)


def test_a_long_chain_is_walked_once(on):
    """Every node has two ways on: walked by paths there would be 2^200."""
    w = leaf()
    on(1, True)
    x = w
    for _ in range(200):
        x = x + x
    layer._one_stream_behind(Op.apply(x, leaf()), 0)
