"""Edges of the layer's operators on the GPU: windows wider than every context, tokens
outside every sequence, heads far apart."""
import numpy as np
import pytest
import torch

from tests import layer_ref as ref
from tests.gpu_util import note
from tests.test_gpu_attention import TYPES, f64, make, offsets, within
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


# Tokens before the first offset and past the last one belong to no sequence.
# Their rows see nothing: outputs and gradients are 0, lse is the log of an
# empty sum.  (lens of the sequences, tokens before and after them)
OUTSIDE = [([40, 30], 0, 30), ([40, 30], 17, 3), ([700], 300, 500), ([1], 0, 300), ([0, 0], 64, 65), ([], 0, 33)]


def fill_with_nan(monkeypatch):
    """What the calls allocate holds NaN before the kernels write it."""
    real = torch.empty

    def empty(*a, **k):
        t = real(*a, **k)
        return t.fill_(float("nan")) if t.is_floating_point() else t
    monkeypatch.setattr(torch, "empty", empty)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,K,D", [(4, 2, 64), (16, 16, 128), (3, 1, 32)])
@pytest.mark.parametrize("lens,before,after", OUTSIDE)
def test_tokens_outside_every_sequence(lens, before, after, H, K, D, dtype, monkeypatch):
    import chunk_weight_rnn_amd as e2
    note(f"tokens outside: {lens} {before} {after} H={H} K={K} D={D} {dtype}")
    n = before + sum(lens) + after
    q, k, v, dout = make([n], H, K, D, dtype)
    cu = offsets([before] + lens)[1:].contiguous()
    inside = slice(before, before + sum(lens))
    fill_with_nan(monkeypatch)
    out, lse = e2.attention_forward(q, k, v, cu)
    g = e2.attention_backward(q, k, v, out, lse, dout, cu)
    torch.cuda.synchronize()
    monkeypatch.undo()
    val, bnd = ref.packed(*(f64(t[inside]) for t in (q, k, v)), lens, 0, D ** -0.5, dtype, f64(dout[inside]))
    for name, t, nothing in (("out", out, 0.0), ("lse", lse, -np.inf), ("dq", g["q"], 0.0), ("dk", g["k"], 0.0),
                             ("dv", g["v"], 0.0)):
        within(name, t[inside], val[name], bnd[name])
        for part in (t[:before], t[before + sum(lens):]):
            assert bool((part.double() == nothing).all()), name


def test_padding_adds_nothing_to_a_projections_gradient():
    """A packed buffer with tokens to spare, through autograd."""
    import chunk_weight_rnn_amd as e2
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(200, 64, generator=g, device="cuda")
    w = torch.randn(4 * 32, 64, generator=g, device="cuda", requires_grad=True)
    cu = offsets([90, 60])

    def grad(x):
        q, k, v = (x @ w.t()).view(-1, 4, 32).split([2, 1, 1], dim=1)
        (r,) = torch.autograd.grad(e2.attention(q, k, v, cu).square().sum(), w)
        return r
    want = grad(x[:150])
    torch.full((200, 4, 32), float("nan"), device="cuda")  # what the allocator hands out next
    got = grad(x)
    assert bool(torch.isfinite(got).all())
    assert float((got - want).norm()) <= 1e-5 * float(want.norm())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new,cached", [([1, 1], [3000, 5]), ([1, 1], [30, 5]), ([100, 60], [2000, 0]),
                                        ([400] * 8, [10] * 8)])
@pytest.mark.parametrize("before,after", [(0, 7), (5, 40)])
def test_new_tokens_outside_every_sequence(new, cached, before, after, dtype):
    import chunk_weight_rnn_amd as e2
    note(f"paged tokens outside: {new} {cached} {before} {after} {dtype}")
    q, k, v, kc, vc, table, cu, held = _paged(TYPES[dtype], new, 16, 4, 64, 16, cached)
    pad = [torch.nn.functional.pad(t, (0, 0, 0, 0, before, after), value=float("nan")) for t in (q, k, v)]
    caches = [(kc.clone(), vc.clone()) for _ in range(2)]
    want = e2.paged_attention(q, k, v, *caches[0], table, cu, held)
    got = torch.full_like(pad[0], float("nan"))
    e2.paged_attention(*pad, *caches[1], table, cu + before, held, out=got)
    inside = got[before:before + sum(new)]
    assert bool(torch.isfinite(inside).all())
    # the number of key ranges may be another: twice the error of the rounded probabilities and of the result
    u = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -18
    assert float((inside.float() - want.float()).abs().max()) <= 4 * u * float(torch.stack([v.abs().max(), vc.abs().max()]).max())
    assert bool((got[:before] == 0).all()) and bool((got[before + sum(new):] == 0).all())
    assert all(torch.equal(a, b) for a, b in zip(*caches))  # and their keys and values go nowhere


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,K", [(4, 2), (3, 1), (2, 2)])
@pytest.mark.parametrize("far", [1 << 23, (1 << 25) + 8])
def test_heads_far_apart(far, H, K, dtype):
    """Head-major tensors of long sequences: heads 2^23 values apart and more, whose
    offsets within a tile leave 31 bits."""
    import chunk_weight_rnn_amd as e2
    note(f"heads {far} apart H={H} K={K} {dtype}")

    def spread(t):
        n, h, d = t.shape
        s = torch.empty((h - 1) * (far + 8) + n * d, dtype=t.dtype, device="cuda").as_strided(t.shape, (d, far + 8, 1))
        return s.copy_(t)
    q, k, v, dout = make([300, 41], H, K, 64, dtype, view=False)
    cu = offsets([300, 41])
    got = []
    for x in ((q, k, v), tuple(spread(t) for t in (q, k, v))):
        out, lse = e2.attention_forward(*x, cu)
        got.append([out, lse, *e2.attention_backward(*x, out, lse, dout, cu).values()])
    assert all(torch.equal(a, b) for a, b in zip(*got))
    m = _paged(TYPES[dtype], [1, 100], H, K, 64, 16, [700, 90])
    assert torch.equal(e2.paged_attention(*m), e2.paged_attention(*(spread(t) for t in m[:3]), *m[3:]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_paged_call_of_no_sequences(dtype):
    import chunk_weight_rnn_amd as e2
    note(f"paged, no sequences, {dtype}")
    q, k, v, kc, vc, *_ = _paged(TYPES[dtype], [5], 4, 2, 64, 16, [3])
    none = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    before = kc.clone(), vc.clone()
    out = torch.full_like(q, float("nan"))
    assert e2.paged_attention(q, k, v, kc, vc, none(0, 4), none(1), none(0), out=out) is out
    assert bool((out == 0).all()) and torch.equal(kc, before[0]) and torch.equal(vc, before[1])
