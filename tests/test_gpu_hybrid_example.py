"""examples/hybrid_layer.py: training runs through the differentiable
operators, serving through the paged cache and the streamed chunk update, and
serving computes what the training forward does.

Tolerances.  The two forwards round at the same places (projections, branch
outputs, the stream, all bf16, unit roundoff u = 2^-8) and differ in the order
of sums and in which of a row's probabilities are rounded as operands, so each
rounding can fall to the other side: about eight of them per layer at u each,
two layers, in the root of the sum of squares 4 u, and a factor of 4 for the
gates' and fast weights' response: 16 u = 1/16 of the logits' norm.  A token at
a wrong position, a stale state or a wrong page changes its logits by their own
size.  With 8-bit projections (e4m3, half a spacing is 2^-4 of a value at most,
2^-5 on average over a binade, in both operands, independent over a row): 2 / 32
per projection and layer, times the same 4: 1/2.
"""
import importlib.util
import os

import pytest
import torch

from tests.gpu_util import note

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "hybrid_layer.py")
    spec = importlib.util.spec_from_file_location("hybrid_layer", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _relative(got, want):
    return float((got.float() - want.float()).norm() / want.float().norm())


def test_training_lowers_the_loss(ex):
    note("hybrid example, training")
    torch.manual_seed(0)
    model = ex.Model().cuda()
    losses = ex.train(model, 30, 4, 512)  # two chunks: the first one's outputs do not depend on its keys
    assert all(x == x for x in losses)
    assert losses[-1] < losses[0]
    for name, p in model.named_parameters():
        assert p.grad is not None and bool(torch.isfinite(p.grad).all()), name
        assert float(p.grad.abs().max()) > 0, name


@pytest.mark.parametrize("bits8,tol", [(False, 1 / 16), (True, 1 / 2)])
@pytest.mark.parametrize("prompt", [0, 200, 512, 530])
def test_serving_equals_the_training_forward(ex, prompt, bits8, tol):
    note(f"hybrid example, prompt {prompt}, bits8 {bits8}")
    torch.manual_seed(1)
    model = ex.Model().cuda()
    T = prompt + 6 if prompt else 260  # token by token across a chunk's end
    tokens = torch.randint(256, (3, T), generator=torch.Generator().manual_seed(2)).cuda()
    with torch.no_grad():
        want = model(torch.nn.functional.pad(tokens, (0, -T % ex.CHUNK)))[:, :T]
    got = ex.serve(model, tokens, prompt, bits8)
    for i in range(T):
        assert _relative(got[:, i], want[:, i]) < tol, f"token {i}"
