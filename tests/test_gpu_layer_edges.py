"""Edges of the layer's operators on the GPU: windows wider than every context."""
import pytest
import torch

from tests.gpu_util import note
from tests.test_gpu_attention import TYPES, make, offsets
from tests.test_gpu_layer_streams import _paged

pytestmark = pytest.mark.gpu


def bits(ts):
    return [t.contiguous().view(torch.uint8) for t in ts]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 70])
def test_a_window_wider_than_every_context_is_none(window, dtype):
    """The same plan, the same sums: the same bits, in calls whose keys are split too."""
    import chunk_weight_rnn_amd as e2
    note(f"window {window} {dtype}")
    q, k, v, dout = make([500, 130], 2, 1, 64, dtype)
    cu = offsets([500, 130])
    got = []
    for w in (0, window):
        out, lse = e2.attention_forward(q, k, v, cu, window=w)
        got.append(bits([out, lse, *e2.attention_backward(q, k, v, out, lse, dout, cu, window=w).values()]))
    assert all(torch.equal(a, b) for a, b in zip(*got))
    for new, cached in (([1, 1], [3000, 5]), ([100, 60], [2000, 0])):
        m = _paged(TYPES[dtype], new, 4, 2, 64, 16, cached)
        assert torch.equal(*(e2.paged_attention(*m, window=w) for w in (0, window)))
