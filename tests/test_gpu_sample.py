"""Sampling on the GPU, against model_ref: the same token for every row and every
random number that is not within 2^-36 of a border (weights may be off by a unit
of 2^-44, 2^8 of them together are at most that), and its log probability."""
import numpy as np
import pytest
import torch

from tests import model_ref as ref
from tests.gpu_util import note
from tests.test_gpu_attention import f64

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "f32": torch.float32}
FILTERS = {"none": {}, "k1": dict(top_k=1), "k": dict(top_k=20), "k_all": dict(top_k=10 ** 6), "p": dict(top_p=0.7),
           "p0": dict(top_p=0.0), "p_most": dict(top_p=0.9999), "m": dict(min_p=0.05), "m1": dict(min_p=1.0),
           "cold": dict(temperature=0.2, top_p=0.9), "hot": dict(temperature=5.0, top_k=100, top_p=0.5, min_p=0.01),
           "greedy": dict(temperature=0.0)}
DEFAULT = dict(temperature=1.0, top_k=0, top_p=1.0, min_p=0.0)
NEAR = 2.0 ** -36


def compare(logits, u, settings, where):
    import chunk_weight_rnn_amd as e2
    note("sample " + where)
    kw = dict(DEFAULT, **settings)
    token, logprob = e2.sample(logits, u, **settings)
    torch.cuda.synchronize()
    x, uu = f64(logits), f64(u)
    col = {k: (v.double().cpu().numpy() if torch.is_tensor(v) else np.full(len(uu), np.float64(np.float32(v)))) for k, v in kw.items()}
    skipped = 0
    for r in range(len(uu)):
        s = [float(col[k][r]) for k in ("temperature", "top_k", "top_p", "min_p")]
        want, lp, bound, far = ref.sample(x[r], uu[r], s[0], int(s[1]), s[2], s[3])
        if far < NEAR and uu[r] != 0:
            skipped += 1
            continue
        assert int(token[r]) == want, f"{where} row {r}"
        assert (np.isnan(lp) and torch.isnan(logprob[r])) or abs(float(logprob[r]) - lp) <= bound, f"{where} row {r}: {float(logprob[r])} {lp}"
    assert skipped <= len(uu) // 8, where
    return token


def logits_of(rows, V, dtype, seed=0, kind="peaks"):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = 2 * torch.randn(rows, V, generator=g, device="cuda")
    if kind == "peaks":
        x.scatter_add_(1, torch.randint(V, (rows, 8), generator=g, device="cuda"), 8 * torch.rand(rows, 8, generator=g, device="cuda"))
    elif kind == "coarse":  # few different values: ties everywhere
        x = torch.round(x)
    elif kind == "flat":
        x = torch.zeros_like(x) - 3.25
    return x.to(T[dtype]), torch.rand(rows, generator=g, device="cuda")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name", list(FILTERS))
@pytest.mark.parametrize("kind", ["peaks", "coarse", "flat", "plain"])
def test_filters(kind, name, dtype):
    for V in (1, 2, 9, 300, 1111):
        x, u = logits_of(8, V, dtype, seed=V, kind=kind)
        compare(x, u, FILTERS[name], f"{kind} {name} {dtype} V={V}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [4095, 4096, 4097, 8192, 8193, 16385, 32000, 32769, 65537, 128257, 262136])
def test_vocabularies(V, dtype):
    """Rows of every form: in the LDS, and read again for each pass; odd strides."""
    x, u = logits_of(3, V, dtype, seed=V)
    for name in ("none", "k", "p", "hot"):
        compare(x, u, FILTERS[name], f"{name} {dtype} V={V}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_every_token_at_its_share(dtype):
    """Random numbers over the whole range: each token between its borders."""
    x, _ = logits_of(1, 37, dtype, seed=5)
    u = (torch.arange(2048, device="cuda") + 0.5) / 2048
    for name in ("none", "k", "p", "m"):
        token = compare(x.expand(2048, 37).contiguous(), u, FILTERS[name], f"{name} {dtype} all u")
        assert (token[1:] >= token[:-1]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_border_cases_as_defined(dtype):
    """Equal weights, whose sums meet the targets exactly."""
    import chunk_weight_rnn_amd as e2
    x = torch.zeros(64, 64, device="cuda").to(T[dtype])
    u = torch.arange(64, device="cuda") / 64
    assert e2.sample(x, u)[0].tolist() == list(range(64))  # u = k / 64: more than k weights
    below = torch.nextafter(u, torch.zeros_like(u))
    assert e2.sample(x, below)[0].tolist() == [0] + list(range(63))
    last = torch.full_like(u, 1 - 2 ** -24)
    assert e2.sample(x, last, top_p=0.5)[0].tolist() == [31] * 64  # half of them, and no more
    assert e2.sample(x, last, top_p=0.5 + 2 ** -20)[0].tolist() == [32] * 64
    assert e2.sample(x, last, top_k=7)[0].tolist() == [6] * 64
    assert e2.sample(x, last, top_k=7, top_p=0.5)[0].tolist() == [3] * 64
    assert e2.sample(x, last, min_p=1.0)[0].tolist() == [63] * 64
    y = x.clone()
    y[:, ::2] = -0.0  # zeros of either sign are equal
    assert e2.sample(y, last, top_k=3)[0].tolist() == [2] * 64


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name", ["none", "k", "p", "m", "hot", "greedy"])
def test_values_that_are_not_finite(name, dtype):
    inf, nan = float("inf"), float("nan")
    rows = [[0.0, nan, 1.0, -inf, 0.5], [-inf] * 5, [nan] * 5, [inf, 0.0, inf, nan, -inf], [-inf, -inf, 2.0, nan, -inf],
            [3e38, 1.0, 3e38, -3e38, 0.0], [-3e38, -3e38, -3e38, nan, -inf]]
    x = torch.tensor(rows, device="cuda").to(T[dtype])
    for u in (0.0, 0.3, 0.6, 0.999):
        compare(x, torch.full((len(rows),), u, device="cuda"), FILTERS[name], f"{name} {dtype} u={u}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_random_numbers_and_temperatures_at_the_ends(dtype):
    import chunk_weight_rnn_amd as e2
    x, _ = logits_of(6, 500, dtype, seed=9)
    u = torch.tensor([0.0, 2.0 ** -149, 2.0 ** -30, 1 - 2.0 ** -24, 0.5, 1e-7], device="cuda")
    for t in (1e-38, 1e-6, 0.01, 1.0, 100.0, 1e30):
        compare(x, u, dict(temperature=t, top_p=0.95), f"{dtype} T={t}")
        compare(x, u, dict(temperature=t), f"{dtype} T={t}")
    odd = torch.tensor([1.0, 1.5, float("inf"), float("nan"), -0.5, -float("inf")], device="cuda")
    near = torch.tensor([1 - 2.0 ** -24, 1 - 2.0 ** -24, 1 - 2.0 ** -24, 0, 0, 0], device="cuda")
    assert torch.equal(e2.sample(x, odd)[0], e2.sample(x, near)[0])


def test_settings_of_each_row():
    x, u = logits_of(12, 700, "f32", seed=3)
    c = lambda *v, d=torch.float32: torch.tensor(v * (12 // len(v)), device="cuda", dtype=d)
    s = dict(temperature=c(0.0, 0.5, 1.0, 2.0), top_k=c(0, 5, 1000, -1, d=torch.int32), top_p=c(1.0, 0.9, 0.3), min_p=c(0.0, 0.1))
    compare(x, u, s, "settings of each row")
    for k, v in s.items():
        compare(x, u, {k: v}, f"{k} of each row")


def test_settings_out_of_range_are_taken_as_written():
    """NaN switches a filter off; as a temperature it takes the largest."""
    import chunk_weight_rnn_amd as e2
    x, u = logits_of(4, 300, "f32", seed=4)
    c = lambda v: torch.full((4,), v, device="cuda")
    same = lambda a, b: all(torch.equal(p, q) for p, q in zip(e2.sample(x, u, **a), e2.sample(x, u, **b)))
    nan = float("nan")
    assert same(dict(top_p=c(nan)), {}) and same(dict(min_p=c(nan)), {}) and same(dict(top_p=c(7.0)), {})
    assert same(dict(temperature=c(nan)), dict(temperature=0.0)) and same(dict(temperature=c(-2.0)), dict(temperature=0.0))
    assert same(dict(top_p=c(-1.0)), dict(top_k=1)) and same(dict(min_p=c(-1.0)), {}) and same(dict(min_p=c(9.0)), dict(min_p=1.0))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strides_and_alignment(dtype):
    import chunk_weight_rnn_amd as e2
    for V in (5, 1001, 40003):
        x, u = logits_of(9, V, dtype, seed=V)
        want = e2.sample(x, u, top_p=0.9)
        for off, wide in ((0, V + 8), (1, V + 1), (3, V + 11)):
            y = torch.full((9, wide), float("inf"), device="cuda").to(x.dtype)
            y[:, off:off + V] = x
            got = e2.sample(y[:, off:off + V], u, top_p=0.9)
            assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_large_batch_and_no_rows():
    import chunk_weight_rnn_amd as e2
    x, u = logits_of(1, 40, "f32", seed=8)
    n = 5000
    us = torch.rand(n, device="cuda")
    token, _ = e2.sample(x.expand(n, 40).contiguous(), us)
    share = torch.softmax(x[0].double(), 0).cumsum(0)
    assert torch.equal(token, torch.searchsorted(share, us.double(), right=True).clamp(max=39))
    token, lp = e2.sample(x[:0], u[:0])
    assert token.shape == lp.shape == (0,)
