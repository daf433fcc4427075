"""examples/hybrid_layer.py with the gated recurrence as a third branch, the 8-bit
cache and sampling: lookup, recurrence, attention over the cache and the choice of
tokens used together, trained and served.

Tolerances.  Training's and serving's forward round at the same places, the branch of
the recurrence among them (its inputs and outputs in bf16, its state in fp32 in both):
of the logits' norm 16 u = 1/16, as tests/test_gpu_hybrid_example.py derives it.  With
the 8-bit cache keys and values are rounded to e4m3, by 2^-5 of a value on average, two
of them per layer, two layers, the same factor of 4 for the response: 1/2.
"""
import numpy as np
import pytest
import torch

from tests import model_ref as ref
from tests.gpu_util import note
from tests.test_gpu_hybrid_example import _relative, ex  # noqa: F401  (ex is a fixture)

pytestmark = pytest.mark.gpu


def _model(ex, seed):  # noqa: F811
    torch.manual_seed(seed)
    return ex.Model(recur=200).cuda()


def test_a_training_step(ex):  # noqa: F811
    note("hybrid example with the recurrence, training")
    model = _model(ex, 0)
    losses = ex.train(model, 2, 3, 512)
    assert all(x == x for x in losses)
    for name, p in model.named_parameters():
        assert p.grad is not None and bool(torch.isfinite(p.grad).all()), name
        assert float(p.grad.abs().max()) > 0, name


def test_the_lookup_is_the_tables_rows(ex):  # noqa: F811
    note("hybrid example, lookup")
    model = _model(ex, 4)
    tokens = torch.randint(256, (3, 40), device="cuda")
    assert torch.equal(model.embedded(tokens), model.embed(tokens.reshape(-1)).bfloat16())
    assert torch.equal(model.embedded(tokens[:, 7:8]), model.embed(tokens[:, 7]).bfloat16())


@pytest.mark.parametrize("cache8,tol", [(False, 1 / 16), (True, 1 / 2)])
@pytest.mark.parametrize("prompt", [0, 300, 512])
def test_serving_equals_the_training_forward(ex, prompt, cache8, tol):  # noqa: F811
    note(f"hybrid example with the recurrence, prompt {prompt}, cache8 {cache8}")
    model = _model(ex, 1)
    T = prompt + 5 if prompt else 60
    tokens = torch.randint(256, (3, T), generator=torch.Generator().manual_seed(2)).cuda()
    with torch.no_grad():
        want = model(torch.nn.functional.pad(tokens, (0, -T % ex.CHUNK)))[:, :T]
    got = ex.serve(model, tokens, prompt, cache8=cache8)
    for i in range(T):
        assert _relative(got[:, i], want[:, i]) < tol, f"token {i}"


def test_drawn_tokens_are_those_of_the_definition(ex):  # noqa: F811
    """Served again, the drawn tokens' logits are the same bits, and each token the one that
    the plain sampling draws from them."""
    note("hybrid example, generation")
    model = _model(ex, 3)
    prompt = torch.randint(256, (3, 250), generator=torch.Generator().manual_seed(5)).cuda()
    kw = dict(temperature=0.8, top_k=50, top_p=0.95, min_p=0.001)
    tokens, logprobs = ex.generate(model, prompt, 12, torch.Generator().manual_seed(6), cache8=True, **kw)  # past a chunk's end
    u = torch.rand(12, 3, generator=torch.Generator().manual_seed(6)).double().numpy()
    logits = ex.serve(model, torch.cat([prompt, tokens], dim=1), 250, cache8=True)[:, 249:].double().cpu().numpy()
    settings = [float(np.float32(kw[n])) for n in ("temperature",)] + [50] + [float(np.float32(kw[n])) for n in ("top_p", "min_p")]
    for r in range(3):
        for i in range(12):
            token, lp, bound, far = ref.sample(logits[r, i], u[i, r], *settings)
            if far < 1e-9:
                continue  # the draw is at a border
            assert int(tokens[r, i]) == token, (r, i)
            assert abs(float(logprobs[r, i]) - lp) <= bound, (r, i)
