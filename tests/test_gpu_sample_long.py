"""Sampling from rows of more logits than the kernel's list holds (8192), against
model_ref: ties and level rows under every filter, borders deep in the row, logits that
rise along it, infinities and NaN far apart.  Rows are taken by the rules of
tests/test_gpu_sample.py, whose comparison this is.

Where no filter but top_p is set, such a row's weights are summed unrounded, each within
2^-45 of the largest one's, so a draw may differ within 2^-45 V of a border: 2^-27 for the
longest row, and `NEAR` for the rest."""
import pytest
import torch

from tests import test_gpu_sample as base
from tests.test_gpu_sample import T, compare

pytestmark = pytest.mark.gpu

FILTERS = {
    "none": {}, "greedy": dict(temperature=0.0), "k20": dict(top_k=20), "k1000": dict(top_k=1000), "k1001": dict(top_k=1001),
    "k5000": dict(top_k=5000), "k_most": dict(top_k=8192), "k1001_p": dict(top_k=1001, top_p=0.6), "k5000_p": dict(top_k=5000, top_p=0.97),
    "k20_p_m": dict(top_k=20, top_p=0.9, min_p=0.01), "k5000_m": dict(top_k=5000, min_p=0.3), "p0": dict(top_p=0.0), "p": dict(top_p=0.7),
    "p_most": dict(top_p=0.9999), "p_m": dict(top_p=0.99, min_p=0.05), "m": dict(min_p=0.05), "m_low": dict(min_p=1e-6), "m1": dict(min_p=1.0),
    "cold": dict(temperature=0.05, top_p=0.9), "hot": dict(temperature=20.0, top_p=0.9), "hot_k": dict(temperature=20.0, top_k=3000, min_p=0.5),
}
KINDS = ["flat", "coarse", "level", "plain", "rising", "falling"]


def logits_of(kind, rows, V, dtype, seed, rise=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = 2 * torch.randn(rows, V, generator=g, device="cuda")
    if kind == "coarse":  # few different values
        x = torch.round(x)
    elif kind == "flat":  # one
        x = torch.zeros_like(x) - 3.25
    elif kind == "level":  # weights that differ little
        x = 0.01 * x
    elif kind in ("rising", "falling"):  # by some 500 powers of two, or as told
        up = torch.linspace(0, 350.0 if rise is None else rise, V, device="cuda")
        x = x + (up if kind == "rising" else up.flip(0))
    return x.to(T[dtype]), torch.rand(rows, generator=g, device="cuda")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("name", list(FILTERS))
def test_filters(name, kind, dtype):
    for V, rows in ((8193, 3), (40003, 1)):
        x, u = logits_of(kind, rows, V, dtype, seed=V + 1)
        compare(x, u, FILTERS[name], f"{kind} {name} {dtype} V={V}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name", ["k1001", "p", "p_most", "k5000_p", "m_low", "none"])
@pytest.mark.parametrize("rise", [190.0, 240.0, 320.0])
def test_bins_that_count_anew(rise, name, dtype):
    """Maxima that rise by less than the bins' depth from step to step, and by more than
    bins count in all, over the row."""
    V = 131075
    x, u = logits_of("rising", 1, V, dtype, seed=int(rise), rise=rise)
    compare(x, u, FILTERS[name], f"rising by {rise} {name} {dtype} V={V}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind,name", [("flat", "none"), ("flat", "p"), ("flat", "k5000"), ("coarse", "k1001_p"), ("coarse", "p_most"),
                                       ("level", "m_low"), ("level", "p"), ("plain", "k5000_p"), ("plain", "m")])
def test_the_longest_rows(kind, name, dtype, monkeypatch):
    monkeypatch.setattr(base, "NEAR", 2.0 ** -27)
    V = 262136
    x, u = logits_of(kind, 1, V, dtype, seed=11)
    compare(x, u, FILTERS[name], f"{kind} {name} {dtype} V={V}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("u", [0.0, 2.0 ** -24, 0.37, 0.5, 1 - 2.0 ** -24])
@pytest.mark.parametrize("name", ["none", "k20", "k1001", "p", "m_low", "k5000_p"])
def test_random_numbers_at_the_ends(name, u, dtype):
    for kind in ("flat", "coarse"):
        x, _ = logits_of(kind, 1, 8200, dtype, seed=3)
        compare(x, torch.full((1,), u, device="cuda"), FILTERS[name], f"{kind} {name} {dtype} u={u}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name", ["none", "greedy", "k20", "k1001", "k5000_p", "p", "m", "k20_p_m", "hot"])
def test_values_that_are_not_finite(name, dtype):
    inf, nan = float("inf"), float("nan")
    V = 40003
    x, u = logits_of("plain", 5, V, dtype, seed=21)
    x[0, ::7] = nan
    x[0, 512 * 16 * 2:512 * 16 * 2 + 1024] = nan  # tiles of nothing else
    x[1, ::3] = -inf
    x[1, 9000:20000] = -inf
    x[2, 5::4001] = inf  # ten of them, tiles apart
    x[2, 7::100] = nan
    x[3] = nan
    x[3, 33333] = -2.5
    x[4] = -inf
    compare(x, u, FILTERS[name], f"not finite {name} {dtype}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_infinities(dtype):
    V = 40003
    x, _ = logits_of("plain", 4, V, dtype, seed=22)
    x[:, 3::3] = float("inf")
    u = torch.tensor([0.0, 0.3, 0.77, 1 - 2.0 ** -24], device="cuda")
    for name in ("none", "k20", "k5000", "k5000_p", "p", "p0", "m1", "greedy"):
        compare(x, u, FILTERS[name], f"infinities {name} {dtype}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_greedy_takes_the_first_of_equal_ones(dtype):
    import chunk_weight_rnn_amd as e2
    V = 100003
    x, u = logits_of("plain", 6, V, dtype, seed=23)
    want = [V - 1, 0, 8192, 65537, 511, 512]
    for r, i in enumerate(want):
        x[r, i] = 50.0
        x[r, i + 1::997] = 50.0
    token, logprob = e2.sample(x, u, temperature=0.0)
    assert token.tolist() == want and bool((logprob == 0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_settings_of_each_long_row(dtype):
    """Rows of one call that go each their way."""
    names = list(FILTERS)
    x, u = logits_of("coarse", len(names), 9001, dtype, seed=31)
    x[1::2] = logits_of("plain", len(names), 9001, dtype, seed=32)[0][1::2]
    col = lambda k, off, d=torch.float32: torch.tensor([FILTERS[n].get(k, off) for n in names], device="cuda", dtype=d)
    compare(x, u, dict(temperature=col("temperature", 1.0), top_k=col("top_k", 0, torch.int32), top_p=col("top_p", 1.0),
                       min_p=col("min_p", 0.0)), f"settings of each row {dtype}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [300, 9001])
def test_temperatures_of_each_row_at_the_ends(V, dtype):
    """Infinite (every finite logit alike), and so small that 1 / T overflows."""
    x, u = logits_of("plain", 8, V, dtype, seed=V)
    x[:, ::5] = -float("inf")
    t = torch.tensor([float("inf"), 1e-45, 3e38, 1e-30] * 2, device="cuda")
    for name in ("none", "k20", "k1001", "p", "m", "k5000_p"):
        compare(x, u, dict(FILTERS[name], temperature=t), f"temperatures at the ends {name} {dtype} V={V}")
