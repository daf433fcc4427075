"""Edges of the norm on the GPU."""
import pytest
import torch

from tests.gpu_util import note
from tests.test_gpu_attention import TYPES

pytestmark = pytest.mark.gpu

# a wave's row, a workgroup's row and re-read rows, in 16-byte units and one value at a time
WIDTHS = [64, 999, 2048, 2052, 4095, 8192, 9001, 20000]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("W", WIDTHS)
def test_a_nan_in_the_weight_reaches_the_scale(W, dtype):
    """scale = max|y| / 448, and a maximum over a NaN is one: the row's 8-bit
    values, which are y over it, with it."""
    import chunk_weight_rnn_amd as e2
    note(f"NaN weight W={W} {dtype}")
    x = torch.randn(3, W, generator=torch.Generator(device="cuda").manual_seed(W), device="cuda").to(TYPES[dtype])
    w = torch.ones(W, device="cuda")
    w[W - 3] = float("nan")
    y, scale, _, _ = e2.norm_forward(x, w, bits8=True)
    assert bool(torch.isnan(scale).all()) and bool(torch.isnan(y.float()).all())
    y, _, _, _ = e2.norm_forward(x, w)  # in the stream's type it stays where it is
    assert torch.isnan(y).sum(dim=1).tolist() == [1, 1, 1]
