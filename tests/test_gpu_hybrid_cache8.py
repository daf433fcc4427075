"""examples/hybrid_layer.py served from the 8-bit cache, against itself served from a bf16
cache of keys and values that plain torch has rounded the same way.

An 8-bit value times its scale is a bf16 number, so both see the same keys and values, and
differ in the order of their sums alone: of the logits' norm 1/16, as
tests/test_gpu_hybrid_example.py derives it for a bf16 cache."""
import pytest
import torch

from tests.gpu_util import note
from tests.test_gpu_hybrid_example import _relative, ex  # noqa: F401  (ex is a fixture)

pytestmark = pytest.mark.gpu


def rounded(x):
    """Rows to e4m3 with the smallest power of two as scale that brings their largest magnitude to 448 = 0.875 2^9."""
    f, e = torch.frexp(x.float().abs().amax(dim=-1, keepdim=True))
    e = torch.where(f > 0, e - 9 + (f > 0.875).int(), torch.zeros_like(e))
    return torch.ldexp(torch.ldexp(x.float(), -e).to(torch.float8_e4m3fn).float(), e).to(x.dtype)


@pytest.mark.parametrize("recur", [0, 200])
@pytest.mark.parametrize("prompt", [0, 300, 512])
def test_the_cache_holds_rounded_keys_and_values(ex, prompt, recur, monkeypatch):  # noqa: F811
    note(f"hybrid example from the 8-bit cache, prompt {prompt}, recur {recur}")
    torch.manual_seed(1)
    model = ex.Model(recur=recur).cuda()
    T = prompt + 5 if prompt else 60
    tokens = torch.randint(256, (3, T), generator=torch.Generator().manual_seed(2)).cuda()
    got = ex.serve(model, tokens, prompt, cache8=True)
    real, calls = ex.e2.paged_attention, []

    def on_rounded(q, k, v, *a, **kw):
        assert "k_scale" not in kw
        calls.append(1)
        return real(q, rounded(k), rounded(v), *a, **kw)
    monkeypatch.setattr(ex.e2, "paged_attention", on_rounded)
    want = ex.serve(model, tokens, prompt)
    assert len(calls) >= 2 * (T - prompt)
    for i in range(T):
        assert _relative(got[:, i], want[:, i]) < 1 / 16, f"token {i}"
