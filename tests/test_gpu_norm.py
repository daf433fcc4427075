"""RMS norm with the residual's addition on the GPU, against layer_ref."""
import numpy as np
import pytest
import torch

from tests import layer_ref as ref
from tests.gpu_util import note
from tests.test_gpu_attention import TYPES, f64, within

pytestmark = pytest.mark.gpu


def rounder(dtype):
    return lambda a: f64(torch.from_numpy(a).to(TYPES[dtype]))


def make(rows, W, dtype, residual, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = lambda s=1.0: (torch.randn(rows, W, generator=g, device="cuda") * s).to(TYPES[dtype])
    x, r, dy, dh = t(), t(2.0), t(), t()
    w = 1 + 0.1 * torch.randn(W, generator=g, device="cuda")
    return x, (r if residual else None), w, dy, (dh if residual else None)


# widths of every form: a wave's row, a workgroup's row, re-read rows, each in
# 16-byte units and one value at a time
WIDTHS = [1, 3, 8, 64, 520, 999, 1024, 2048, 2052, 4095, 8192, 8200, 9001]


def check(rows, W, dtype, residual):
    import chunk_weight_rnn_amd as e2
    where = f"rows={rows} W={W} {dtype} residual={residual}"
    note("norm " + where)
    x, r, w, dy, dh = make(rows, W, dtype, residual)
    y, scale, h, rstd = e2.norm_forward(x, w, residual=r, eps=1e-5)
    assert scale is None
    dx, dw = e2.norm_backward(dy, h, w, rstd, dh=dh)
    torch.cuda.synchronize()
    want = ref.norm(f64(x), None if r is None else f64(r), f64(w), 1e-5, dtype, rounder(dtype), f64(dy),
                    None if dh is None else f64(dh))
    for n, t in (("h", h), ("rstd", rstd), ("y", y), ("dx", dx), ("dweight", dw)):
        within(n, t, *want[n], where)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("W", WIDTHS)
def test_widths(W, dtype):
    check(5, W, dtype, True)
    check(3, W, dtype, False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 2, 9, 513, 4099])
def test_rows(rows, dtype):
    check(rows, 160, dtype, True)


def e4m3_gap(q):
    """Distance between neighbours of e4m3 at |q|."""
    e = np.floor(np.log2(np.maximum(np.abs(q), 2.0 ** -6)))
    return 2.0 ** (e - 3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("W", WIDTHS)
def test_bits8(W, dtype):
    """Every 8-bit value is within half a step of y / scale (and of what fp32
    errors in it can move), the largest of a row is 448."""
    import chunk_weight_rnn_amd as e2
    x, r, w, _, _ = make(6, W, dtype, True, seed=W)
    y, scale, h, _ = e2.norm_forward(x, w, residual=r, bits8=True)
    torch.cuda.synchronize()
    assert y.dtype == torch.float8_e4m3fn and scale.shape == (6,)
    want = ref.norm(f64(x), f64(r), f64(w), 1e-6, dtype, rounder(dtype))
    val, bnd = want["y32"]
    top = np.abs(val).max(axis=1)
    rel = (bnd / np.maximum(np.abs(val), 1e-300)).max()
    within("scale", scale, top / 448, top / 448 * (rel + 2.0 ** -22))
    q = val / (top / 448)[:, None]
    got = f64(y.float())
    assert np.abs(got).max(axis=1).tolist() == [448.0] * 6
    assert (np.abs(got - q) <= 0.5 * e4m3_gap(q) + 4 * rel * np.abs(q) + 1e-6).all()


def test_rows_of_zeros_nan_and_inf():
    import chunk_weight_rnn_amd as e2
    x = torch.zeros(4, 256, device="cuda", dtype=torch.bfloat16)
    x[1, 3] = float("nan")
    x[2, 5] = float("inf")
    x[3] = 1
    w = torch.ones(256, device="cuda")
    for bits8 in (False, True):
        y, scale, _, _ = e2.norm_forward(x, w, bits8=bits8)
        f = y.float()
        assert (f[0] == 0).all() and torch.isnan(f[1]).all() and torch.isnan(f[2, 5]) and torch.isfinite(f[3]).all()
        if bits8:
            assert scale[0] == 1 and (f[3] == 448).all()


def test_tiny_rows_in_8_bits():
    """Rows so small that the scale is subnormal stay finite."""
    import chunk_weight_rnn_amd as e2
    x = torch.full((3, 64), 1e-38, device="cuda")
    w = torch.full((64,), 3e-5, device="cuda")
    y, scale, _, _ = e2.norm_forward(x, w, eps=1.0, bits8=True)
    assert torch.isfinite(y.float()).all() and torch.isfinite(scale).all()


@pytest.mark.parametrize("W", [2048, 777, 20000])
def test_in_place_stream_and_repeat(W):
    import chunk_weight_rnn_amd as e2
    x, r, w, dy, dh = make(300, W, "bf16", True)
    y, _, h, rstd = e2.norm_forward(x, w, residual=r)
    dx, dw = e2.norm_backward(dy, h, w, rstd, dh=dh)
    r2 = r.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y2, _, h2, rstd2 = e2.norm_forward(x, w, residual=r2, h=r2)
        dx2, dw2 = e2.norm_backward(dy, h2, w, rstd2, dh=dh)
    s.synchronize()
    torch.cuda.synchronize()
    assert h2 is r2
    for a, b in ((y, y2), (h, h2), (rstd, rstd2), (dx, dx2), (dw, dw2)):
        assert torch.equal(a, b)


def test_autograd_and_differences():
    """rms_norm() gives norm_backward's gradients, and in fp32 they match
    central differences: off by h^2 / 6 times the third derivative and by the
    forward's noise over h, both against |dy| |y|'s size."""
    import chunk_weight_rnn_amd as e2
    x, r, w, dy, dh = make(7, 96, "f32", True)
    leaves = [t.clone().requires_grad_(True) for t in (x, w, r)]
    y, h = e2.rms_norm(leaves[0], leaves[1], leaves[2])
    ((y * dy).sum() + (h * dh).sum()).backward()
    y0, _, h0, rstd = e2.norm_forward(x, w, residual=r)
    dx, dw = e2.norm_backward(dy, h0, w, rstd, dh=dh)
    for leaf, g in zip(leaves, (dx, dw, dx)):
        assert torch.equal(leaf.grad, g)
    gen = torch.Generator(device="cuda").manual_seed(3)
    step = 2.0 ** -7
    for i, g in enumerate((dx, dw, dx)):
        d = torch.randn(g.shape, generator=gen, device="cuda") / g.numel() ** 0.5

        def f(t):
            a = [x, w, r]
            a[i] = a[i] + t * d
            yy, _, hh, _ = e2.norm_forward(a[0], a[1], residual=a[2])
            return float((yy.double() * dy.double()).sum() + (hh.double() * dh.double()).sum())
        diff = (f(step) - f(-step)) / (2 * step)
        size = float(dy.norm() * y0.norm() + dh.norm() * h0.norm())
        assert abs(diff - float((g.double() * d.double()).sum())) <= (step * step + 2.0 ** -20 / step) * size
    # without a residual, h is x and y alone has a gradient
    lx = x.clone().requires_grad_(True)
    yy, hh = e2.rms_norm(lx, w)
    assert hh is lx
    (yy * dy).sum().backward()
    _, _, _, rs = e2.norm_forward(x, w)
    assert torch.equal(lx.grad, e2.norm_backward(dy, x, w, rs)[0])


def test_any_leading_dimensions():
    import chunk_weight_rnn_amd as e2
    x, r, w, _, _ = make(12, 64, "bf16", True)
    y, _, h, rstd = e2.norm_forward(x, w, residual=r)
    for lead in ((3, 4), (2, 3, 2), (12,)):
        a = e2.norm_forward(x.view(*lead, 64), w, residual=r.view(*lead, 64))
        assert a[0].shape == (*lead, 64) and a[3].shape == lead
        assert torch.equal(a[0].view(12, 64), y) and torch.equal(a[3].view(12), rstd)
    a = e2.norm_forward(x[0], w, residual=r[0])
    assert a[3].shape == () and torch.equal(a[0], y[0])
    a = e2.norm_forward(x[0], w, residual=r[0], bits8=True)
    assert a[1].shape == () and a[3] is None


def test_no_rows():
    import chunk_weight_rnn_amd as e2
    x = torch.empty(0, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    y, _, h, rstd = e2.norm_forward(x, w)
    assert y.shape == (0, 64) and rstd.shape == (0,)
    dx, dw = e2.norm_backward(x, h, w, rstd)
    torch.cuda.synchronize()
    assert dx.shape == (0, 64) and (dw == 0).all()
