"""Edges of the norm on the GPU."""
import pytest
import torch

from tests import layer_ref as ref
from tests.gpu_util import note
from tests.test_gpu_attention import TYPES, f64, within
from tests.test_gpu_norm import make, rounder

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


@pytest.mark.parametrize("W", [64, 999, 4095, 9001])
@pytest.mark.parametrize("units", [1, 3, 100, 223, 225, 448, 5000])
def test_rows_whose_scale_is_the_smallest_value(units, W):
    """Rows of zeros and of values of a few times 2^-149: the zeros stay zeros and
    the products with the scale stay within half a step of e4m3, a sixteenth of a
    value, and of 2^-149."""
    import chunk_weight_rnn_amd as e2
    note(f"scale near 2^-149: {units} W={W}")
    tiny = 2.0 ** -149
    x = torch.zeros(2, W, device="cuda", dtype=torch.float64)
    x[:, ::3] = 2.0 ** -126
    w = torch.full((W,), units * 2.0 ** -23, device="cuda")  # x w = units 2^-149, exactly, and rstd is 1
    y, scale, _, _ = e2.norm_forward(x.float(), w, eps=1.0, bits8=True)
    y, scale = y.double(), scale.double()
    assert bool((scale > 0).all())
    assert bool((y[x == 0] == 0).all())
    off = (y * scale[:, None] - torch.where(x > 0, units * tiny, 0.0)).abs()
    # the scale is rounded to whole 2^-149, and a quotient past 448 is 448
    bound = units * tiny / 16 + 0.5 * tiny + (448 * 0.5 * tiny if units >= 224 else 0.0)
    assert float(off.max()) <= bound


def repeated(block, rows):
    """The rows of `block` again and again, `rows` in all."""
    big = torch.empty(rows, block.shape[1], dtype=block.dtype, device="cuda")
    for a in range(0, rows, block.shape[0]):
        n = min(block.shape[0], rows - a)
        big[a:a + n] = block[:n]
    return big


def same_rows(big, block):
    return all(torch.equal(big[a:a + block.shape[0]], block[:big.shape[0] - a])
               for a in range(0, big.shape[0], block.shape[0]))


# more rows than workgroups that one dimension of a grid may have: four rows to a
# workgroup of 256 threads, one to 256, one to 1024
@pytest.mark.parametrize("W,rows", [(8, (1 << 26) + 5), (1025, (1 << 24) + 3), (4097, (1 << 22) + 3)])
def test_more_rows_than_a_dimension_of_a_grid(W, rows):
    import chunk_weight_rnn_amd as e2
    note(f"norm of {rows} rows of {W}")
    block = torch.randn(1 << 19, W, dtype=torch.bfloat16, device="cuda")
    w = torch.rand(W, device="cuda")
    x = repeated(block, rows)
    y, _, _, rstd = e2.norm_forward(x, w)
    want, _, _, want_rstd = e2.norm_forward(block, w)
    assert same_rows(y, want) and same_rows(rstd[:, None], want_rstd[:, None])
    del y
    dx, _ = e2.norm_backward(x, x, w, rstd)
    want, _ = e2.norm_backward(block, block, w, want_rstd)
    assert same_rows(dx, want)
    del x, dx, rstd, block, want, want_rstd
    torch.cuda.empty_cache()


def shifted(t):
    """The same values one element past an allocation's start."""
    flat = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
    flat[1:] = t.flatten()
    return flat[1:].view(t.shape)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("W", [1, 64, 777, 2048, 4104, 9001])
def test_tensors_aligned_to_their_elements_alone(W, dtype):
    import chunk_weight_rnn_amd as e2
    note(f"norm of shifted tensors W={W} {dtype}")
    x, r, w, dy, dh = (shifted(t) for t in make(5, W, dtype, True, seed=W))
    y, _, h, rstd = e2.norm_forward(x, w, residual=r, h=shifted(r))
    dx, dw = e2.norm_backward(dy, h, w, rstd, dh=dh)
    want = ref.norm(f64(x), f64(r), f64(w), 1e-6, dtype, rounder(dtype), f64(dy), f64(dh))
    for n, t in (("h", h), ("rstd", rstd), ("y", y), ("dx", dx), ("dweight", dw)):
        within(n, t, *want[n], f"W={W} {dtype}")
    y8, scale, _, _ = e2.norm_forward(h, w, bits8=True)
    assert bool(torch.isfinite(y8.float()).all())
    # half a step of e4m3, 2^-4 of a value or half of 2^-9, and what y itself is off
    val, bnd = want["y32"]
    within("y8", y8.double() * scale.double()[:, None], val, 1.01 * abs(val) / 16 + f64(scale)[:, None] * 2.0 ** -9 + bnd)


def test_gradients_of_rows_put_together():
    """What arrives from a concatenation are slices of one gradient, which start anywhere."""
    import chunk_weight_rnn_amd as e2
    g = torch.Generator(device="cuda").manual_seed(4)
    a, b, dy = (torch.randn(n, 777, generator=g, device="cuda").bfloat16() for n in (3, 5, 8))
    w = torch.ones(777, device="cuda")
    leaves = [t.clone().requires_grad_(True) for t in (a, b)]
    torch.cat([e2.rms_norm(t, w)[0] for t in leaves]).backward(dy)
    for t, leaf, d in ((a, leaves[0], dy[:3]), (b, leaves[1], dy[3:])):
        rstd = e2.norm_forward(t, w)[3]
        assert torch.equal(leaf.grad, e2.norm_backward(d.clone(), t, w, rstd)[0])
