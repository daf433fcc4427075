"""Token lookup and its gradient on the GPU, against model_ref."""
import numpy as np
import pytest
import torch

from tests import model_ref as ref
from tests.gpu_util import note
from tests.test_gpu_attention import f64, within

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "f32": torch.float32}
TYPES = [(a, b) for a in T for b in T]


def tokens_of(n, vocab, kind, seed=0):
    rng = np.random.default_rng(seed)
    if kind == "even":
        t = rng.integers(0, vocab, n)
    elif kind == "words":  # a few of them make up most of the text
        t = np.minimum(rng.zipf(1.3, n) - 1, vocab - 1)
        t = rng.permutation(vocab)[t]
    elif kind == "one":
        t = np.full(n, vocab // 2)
    else:  # "outside": some are not in the table
        t = rng.integers(-vocab, 2 * vocab, n)
    return torch.from_numpy(t.astype(np.int64)).cuda()


def check(n, vocab, W, table="f32", dtype="bf16", kind="even", scale=1.0, index=torch.int64, seed=0):
    import chunk_weight_rnn_amd as e2
    where = f"n={n} vocab={vocab} W={W} {table}->{dtype} {kind} scale={scale} {index}"
    note("embedding " + where)
    g = torch.Generator(device="cuda").manual_seed(seed)
    tok = tokens_of(n, vocab, kind, seed).to(index)
    w = torch.randn(vocab, W, generator=g, device="cuda").to(T[table])
    d = torch.randn(n, W, generator=g, device="cuda").to(T[dtype])
    out = e2.embedding_forward(tok, w, scale=scale, dtype=T[dtype])
    dw = e2.embedding_backward(d, tok, vocab, scale=scale, dtype=T[table])
    torch.cuda.synchronize()
    t, s = tok.cpu().numpy(), float(np.float32(scale))
    within("out", out, *ref.lookup(t, f64(w), s, dtype), where)
    within("dweight", dw, *ref.lookup_gradient(t, f64(d), vocab, s, table), where)
    assert torch.equal(dw, e2.embedding_backward(d, tok, vocab, scale=scale, dtype=T[table])), where


@pytest.mark.parametrize("table,dtype", TYPES)
@pytest.mark.parametrize("W", [1, 7, 8, 64, 65, 100, 512, 516, 2048, 2056, 4100])
def test_widths(W, table, dtype):
    check(70, 40, W, table, dtype)


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 1000, 1025, 5000])
@pytest.mark.parametrize("kind", ["even", "words", "one", "outside"])
def test_counts(n, kind):
    """Rows with one place to thousands, pieces that begin and end inside rows."""
    check(n, 50, 40, kind=kind, seed=n)
    check(n, 50, 24, "bf16", "f32", kind=kind, seed=n)


@pytest.mark.parametrize("vocab", [1, 2, 3, 511, 512, 513, 1025, 32000, 262145, 300001])
def test_vocabularies(vocab):
    check(900, vocab, 8, kind="words")
    check(900, vocab, 8, kind="outside")


@pytest.mark.parametrize("table,dtype", TYPES)
@pytest.mark.parametrize("scale", [0.0, -1.5, 45.254833995939045, 1e-20])
def test_scales(scale, table, dtype):
    check(300, 20, 48, table, dtype, scale=scale)


@pytest.mark.parametrize("kind", ["even", "words", "outside"])
def test_int32_tokens(kind):
    check(777, 100, 64, kind=kind, index=torch.int32)


def test_the_lookup_is_exact():
    """Without a scale the values are the table's, cast."""
    import chunk_weight_rnn_amd as e2
    w = torch.randn(100, 512, device="cuda")
    t = torch.randint(100, (5, 6, 7), device="cuda")
    assert torch.equal(e2.embedding_forward(t, w), w[t])
    assert torch.equal(e2.embedding_forward(t, w, dtype=torch.bfloat16), w[t].bfloat16())
    assert torch.equal(e2.embedding_forward(t, w.bfloat16(), dtype=torch.float32), w.bfloat16()[t].float())
    out = torch.empty(5, 6, 7, 512, device="cuda")
    assert e2.embedding_forward(t, w, out=out) is out and torch.equal(out, w[t])


@pytest.mark.parametrize("table,dtype", TYPES)
def test_tensors_that_begin_at_an_odd_element(table, dtype):
    import chunk_weight_rnn_amd as e2
    n, vocab, W = 200, 30, 64
    t = tokens_of(n, vocab, "words")
    w, d = torch.randn(vocab, W, device="cuda").to(T[table]), torch.randn(n, W, device="cuda").to(T[dtype])
    want = e2.embedding_forward(t, w, dtype=T[dtype]), e2.embedding_backward(d, t, vocab, dtype=T[table])
    odd = lambda x: torch.empty(x.numel() + 1, dtype=x.dtype, device="cuda")[1:].view(x.shape).copy_(x)
    assert torch.equal(e2.embedding_forward(t, odd(w), dtype=T[dtype], out=odd(want[0])), want[0])
    assert torch.equal(e2.embedding_backward(odd(d), t, vocab, dtype=T[table], out=odd(want[1])), want[1])


def test_no_tokens():
    import chunk_weight_rnn_amd as e2
    t = torch.empty(0, dtype=torch.int64, device="cuda")
    assert e2.embedding_forward(t, torch.randn(3, 4, device="cuda")).shape == (0, 4)
    assert torch.equal(e2.embedding_backward(torch.empty(0, 4, device="cuda"), t, 3), torch.zeros(3, 4, device="cuda"))


def test_not_finite_rows_reach_their_tokens_alone():
    import chunk_weight_rnn_amd as e2
    t = tokens_of(3000, 20, "words")
    d = torch.randn(3000, 64, device="cuda")
    want = e2.embedding_backward(d, t, 20)
    d[1234] = float("nan")
    got = e2.embedding_backward(d, t, 20)
    v = int(t[1234])
    assert torch.isnan(got[v]).all()
    got[v] = want[v]
    assert torch.equal(got, want)


def test_autograd():
    import chunk_weight_rnn_amd as e2
    w = torch.randn(40, 48, device="cuda", requires_grad=True)
    t = tokens_of(500, 40, "words").view(5, 100)
    out = e2.embedding(t, w, scale=3.0, dtype=torch.bfloat16)
    d = torch.randn(out.shape, device="cuda").bfloat16()
    out.backward(d)
    assert out.dtype == torch.bfloat16 and w.grad.dtype == torch.float32
    assert torch.equal(w.grad, e2.embedding_backward(d, t, 40, scale=3.0, dtype=torch.float32))
    # differences: the map is linear, so one step of any size
    v = torch.randn(40, 48, device="cuda")
    change = e2.embedding_forward(t, v, scale=3.0).double()
    want = float((change * d.double()).sum())
    size = float((change * d.double()).abs().sum())
    assert abs(float((w.grad.double() * v.double()).sum()) - want) < 2 ** -16 * size
    (g,) = torch.autograd.grad(e2.embedding(t, w).sum(), w, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


def test_rows_past_32_bit_offsets():
    """A table and outputs of more than 2^32 bytes."""
    import chunk_weight_rnn_amd as e2
    V, W = (1 << 32) // 8192 + 100, 4096
    w = torch.zeros(V, W, dtype=torch.bfloat16, device="cuda")
    rows = [0, 5, V // 2, V - 2, V - 1]
    vals = torch.randn(len(rows), W, device="cuda").bfloat16()
    w[rows] = vals
    t = torch.tensor(rows, device="cuda").repeat(20)
    assert torch.equal(e2.embedding_forward(t, w), vals.repeat(20, 1))
    d = torch.ones(len(t), W, device="cuda").bfloat16()
    g = e2.embedding_backward(d, t, V)
    assert (g[rows] == 20).all() and int(torch.count_nonzero(g)) == len(rows) * W
