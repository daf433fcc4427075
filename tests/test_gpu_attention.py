"""Causal attention over packed sequences on the GPU, forward and backward,
against the 64-bit implementation in layer_ref (values and bounds)."""
import numpy as np
import pytest
import torch

from tests import layer_ref as ref
from tests.gpu_util import note

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def offsets(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


def f64(t):
    return t.detach().double().cpu().numpy()


def within(name, got, val, bnd, where=""):
    got = f64(got)
    assert got.shape == val.shape, (name, got.shape, val.shape)
    same = (got == val) | (np.isnan(got) & np.isnan(val))
    with np.errstate(invalid="ignore"):
        off = np.where(same, 0.0, np.abs(got - val))
    bad = ~(off <= bnd)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, off / np.maximum(bnd, 1e-300), 0)), off.shape)
        raise AssertionError(f"{where} {name}: {int(bad.sum())} of {bad.size} outside; worst at {i}: "
                             f"{got[i]} for {val[i]}, bound {bnd[i]}")


def make(lens, H, K, D, dtype, seed=0, view=True, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    N = sum(lens)
    x = (torch.randn(N, H + 2 * K, D, generator=g, device="cuda") * std).to(TYPES[dtype])
    q, k, v = x[:, :H], x[:, H:H + K], x[:, H + K:]
    if not view:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    dout = torch.randn(N, H, D, generator=g, device="cuda").to(TYPES[dtype])
    return q, k, v, dout


def check(lens, H, K, D, dtype, window, view=True, scale=None, seed=0, std=1.0):
    import chunk_weight_rnn_amd as e2
    where = f"lens={lens} H={H} K={K} D={D} {dtype} window={window}"
    note("attention " + where)
    q, k, v, dout = make(lens, H, K, D, dtype, seed, view, std)
    cu = offsets(lens)
    kw = dict(window=window, scale=scale)
    out, lse = e2.attention_forward(q, k, v, cu, **kw)
    torch.cuda.synchronize()
    val, bnd = ref.packed(f64(q), f64(k), f64(v), lens, window, scale or D ** -0.5, dtype, f64(dout))
    within("out", out, val["out"], bnd["out"], where)
    within("lse", lse, val["lse"], bnd["lse"], where)
    g = e2.attention_backward(q, k, v, out, lse, dout, cu, **kw)
    torch.cuda.synchronize()
    for n in ("q", "k", "v"):
        assert g[n].dtype == q.dtype
        within("d" + n, g[n], val["d" + n], bnd["d" + n], where)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[1], [2], [31], [32], [33], [63, 64, 65], [1, 0, 129, 1, 0, 7], [300, 5]])
def test_lengths(lens, dtype):
    check(lens, 4, 2, 64, dtype, 0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,K", [(1, 1), (3, 1), (6, 2), (5, 5), (8, 1), (16, 4), (40, 1)])
def test_head_groups(H, K, dtype):
    check([70, 3, 45], H, K, 64 if H > 8 else 128, dtype, 0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [8, 16, 24, 32, 56, 64, 72, 96, 120, 128])
def test_head_dims(D, dtype):
    check([97, 40], 4, 2, D, dtype, 0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window", [1, 2, 31, 64, 65, 127, 1000, 2 ** 31 - 1])
def test_windows(window, dtype):
    check([260, 90], 4, 2, 64, dtype, window)


@pytest.mark.parametrize("window", [0, 100])
def test_long_sequence_of_few_heads(window):
    """One sequence whose row tiles alone would not fill the chip (the keys are
    split and joined), over many key tiles."""
    check([1500], 2, 1, 128, "bf16", window)


@pytest.mark.parametrize("H,K,D,window", [(16, 16, 128, 0), (32, 16, 64, 0), (48, 16, 128, 0), (16, 16, 64, 150)])
def test_many_key_blocks(H, K, D, window):
    """Enough key blocks to fill the chip, with groups that divide a tile and
    one that does not."""
    check([700, 0, 900, 505], H, K, D, "bf16", window)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_sequences(dtype):
    """More sequences than a wave has lanes, some empty."""
    check([(i * 7) % 13 for i in range(150)], 2, 1, 32, dtype, 0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_contiguous_inputs_and_scale(dtype):
    check([130, 61], 4, 4, 64, dtype, 0, view=False, scale=0.31)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_steep_scores(dtype):
    """Scores of some hundreds: the running maximum rises by more than the lazy
    threshold again and again, and most probabilities vanish."""
    check([200, 77], 2, 2, 64, dtype, 0, std=5.0)


def test_head_major_views():
    """[H, N, D] tensors passed as [N, H, D] views."""
    import chunk_weight_rnn_amd as e2
    lens, H, K, D = [90, 33], 4, 2, 64
    q, k, v, _ = make(lens, H, K, D, "bf16", view=False)
    hm = [t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k, v)]
    assert not hm[0].is_contiguous()
    a = e2.attention_forward(q, k, v, offsets(lens))
    b = e2.attention_forward(*hm, offsets(lens))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_same_bits_again_and_on_another_stream():
    import chunk_weight_rnn_amd as e2
    lens = [700, 400, 123]
    q, k, v, dout = make(lens, 8, 2, 128, "bf16")
    cu = offsets(lens)

    def both(stream=None):
        out, lse = e2.attention_forward(q, k, v, cu, stream=stream)
        return [out, lse, *e2.attention_backward(q, k, v, out, lse, dout, cu, stream=stream).values()]
    a = both()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = both()
    s.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_a_sequence_does_not_reach_its_neighbours():
    """NaN and Inf in one packed sequence leave the others' results as they are."""
    import chunk_weight_rnn_amd as e2
    lens = [70, 90, 50]
    q, k, v, dout = make(lens, 4, 2, 64, "bf16", view=False)
    cu = offsets(lens)
    want, lse = e2.attention_forward(q, k, v, cu)
    gw = e2.attention_backward(q, k, v, want, lse, dout, cu)
    for t in (q, k, v):
        t[70:160] = float("nan")
    k[100] = float("inf")
    got, lse = e2.attention_forward(q, k, v, cu)
    gg = e2.attention_backward(q, k, v, got, lse, dout, cu)
    keep = torch.ones(210, dtype=torch.bool, device="cuda")
    keep[70:160] = False
    assert torch.equal(got[keep], want[keep])
    assert torch.isnan(got[70:160]).all()
    for n in ("q", "k", "v"):
        assert torch.equal(gg[n][keep], gw[n][keep])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,K,D,window", [(4, 2, 64, 0), (2, 2, 128, 50), (8, 1, 96, 0)])
@pytest.mark.parametrize("what", ["v_nan", "v_inf", "k_nan", "q_nan", "dout_inf"])
def test_not_finite_values_in_masked_places(what, H, K, D, window, dtype):
    """A NaN or Inf reaches the results that depend on it and no others: what
    the masked terms would bring stays out, exactly as without them."""
    import chunk_weight_rnn_amd as e2
    n, at = 190, 100
    note(f"not finite: {what} H={H} K={K} D={D} window={window} {dtype}")
    q, k, v, dout = make([n], H, K, D, dtype, seed=3, view=False)
    cu = offsets([n])
    x = {"v_nan": v, "v_inf": v, "k_nan": k, "q_nan": q, "dout_inf": dout}[what]
    x[at, 0, 5] = float("inf") if what.endswith("inf") else float("nan")
    out, lse = e2.attention_forward(q, k, v, cu, window=window)
    g = e2.attention_backward(q, k, v, out, lse, dout, cu, window=window)
    x[at, 0, 5] = 1.0  # what does not depend on the value may be compared with any other
    val, bnd = ref.packed(f64(q), f64(k), f64(v), [n], window, D ** -0.5, dtype, f64(dout))
    # what each result depends on, by position
    i = np.arange(n)
    sees = (i >= at) & ((i < at + window) if window else True)   # queries that see position `at`
    seen = (i <= at) & ((i > at - window) if window else True)   # keys that it sees
    G = H // K
    clean = {}
    if what[0] in "vk":
        hit = np.zeros((n, H), bool)
        hit[sees, :G] = True
        clean["out"] = ~hit
        clean["dq"] = ~hit
        # a key's gradients come from every row that sees it and is hit
        key_hit = np.array([any(sees[r] for r in range(j, min(n, j + window) if window else n)) for j in range(n)])
        clean["dk"] = clean["dv"] = ~np.stack([key_hit if h == 0 else np.zeros(n, bool) for h in range(K)], 1)
        if what[0] == "v":
            clean["dv"] = np.ones((n, K), bool)  # dv does not depend on v
    else:
        hit = np.zeros((n, H), bool)
        hit[at, 0] = True
        clean["out"] = ~hit if what == "q_nan" else np.ones((n, H), bool)
        clean["dq"] = ~hit
        clean["dk"] = clean["dv"] = ~np.stack([seen if h == 0 else np.zeros(n, bool) for h in range(K)], 1)
    for name, t in (("out", out), ("dq", g["q"]), ("dk", g["k"]), ("dv", g["v"])):
        c = clean[name]
        got = f64(t)
        assert np.isfinite(got[c]).all(), f"{what}: {name} is not finite where it should be"
        assert (np.abs(got[c] - val[name][c]) <= bnd[name][c]).all(), f"{what}: {name}"
    assert not np.isfinite(f64(out)[at, 0]).all() or what == "dout_inf"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_autograd_and_differences(dtype):
    """attention() under torch.autograd gives attention_backward's gradients; in
    fp32 they also match central differences of the forward along a random
    direction.  With step h the difference is off by h^2 / 6 times the third
    derivative (of the order of the function's own magnitude for directions of
    unit scores) and by the forward's noise over h."""
    import chunk_weight_rnn_amd as e2
    lens, H, K, D = [61, 20], 4, 2, 32
    q, k, v, dout = make(lens, H, K, D, dtype, view=False)
    cu = offsets(lens)
    leaves = [t.clone().requires_grad_(True) for t in (q, k, v)]
    out = e2.attention(*leaves, cu, window=40)
    (out.float() * dout.float()).sum().backward()
    o, lse = e2.attention_forward(q, k, v, cu, window=40)
    g = e2.attention_backward(q, k, v, o, lse, dout, cu, window=40)
    for leaf, n in zip(leaves, ("q", "k", "v")):
        assert torch.equal(leaf.grad, g[n])
    if dtype == "bf16":
        return
    gen = torch.Generator(device="cuda").manual_seed(5)
    h = 2.0 ** -7
    for i, n in enumerate(("q", "k", "v")):
        d = torch.randn(g[n].shape, generator=gen, device="cuda") / g[n].numel() ** 0.5
        def f(t):
            x = [q, k, v]
            x[i] = x[i] + t * d
            return float((e2.attention_forward(*x, cu, window=40)[0].double() * dout.double()).sum())
        diff = (f(h) - f(-h)) / (2 * h)
        size = float(dout.double().norm() * v.double().norm()) / D ** 0.5
        assert abs(diff - float((g[n].double() * d.double()).sum())) <= (h * h + 2.0 ** -20 / h) * size


def test_empty_calls():
    import chunk_weight_rnn_amd as e2
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    k = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    out, lse = e2.attention_forward(q, k, k, offsets([0, 0]))
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    g = e2.attention_backward(q, k, k, out, lse, out, offsets([0, 0]))
    assert g["k"].shape == (0, 2, 64)


def test_wrong_offsets_stay_inside():
    """Offsets that do not fit the tensors are clamped: no access outside, no
    result promised."""
    import chunk_weight_rnn_amd as e2
    q, k, v, dout = make([100], 4, 2, 64, "bf16", view=False)
    for cu in ([0, 1 << 30], [50, 20, 100], [-5, 60], [200, 300]):
        c = torch.tensor(cu, dtype=torch.int32, device="cuda")
        out, lse = torch.zeros_like(q), torch.zeros(100, 4, device="cuda")
        e2.attention_forward(q, k, v, c, out=out, lse=lse)
        e2.attention_backward(q, k, v, out, lse, dout, c)
    torch.cuda.synchronize()
