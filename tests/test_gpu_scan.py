"""The gated linear recurrence and its gradients on the GPU, against model_ref."""
import numpy as np
import pytest
import torch

from tests import model_ref as ref
from tests.gpu_util import note
from tests.test_gpu_attention import f64, offsets, within

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "f32": torch.float32}
TYPES = [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")]


def make(lens, C, dtype, gate, seed=0, before=0, after=0, low=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = before + sum(lens) + after
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    a = low + (1 - low) * torch.rand(n, C, generator=g, device="cuda") ** 0.25  # many near 1
    cu = offsets(lens) + before
    return dict(x=r(n, C).to(T[dtype]), a=a.to(T[gate]), h0=r(len(lens), C), cu=cu.to(torch.int32), dout=r(n, C).to(T[dtype]),
                dstate=r(len(lens), C))


def check(lens, C, dtype, gate, **kw):
    import chunk_weight_rnn_amd as e2
    where = f"lens={lens if len(lens) < 9 else len(lens)} C={C} {dtype} {gate} {kw}"
    note("scan " + where)
    m = make(lens, C, dtype, gate, **kw)
    out, state, starts = e2.gated_scan_forward(m["x"], m["a"], m["cu"], h0=m["h0"], save=True)
    g = e2.gated_scan_backward(m["dout"], m["x"], m["a"], starts, m["cu"], dstate=m["dstate"])
    torch.cuda.synchronize()
    r = ref.scan(f64(m["x"]), f64(m["a"]), f64(m["h0"]), lens, kw.get("before", 0), dtype, gate, f64(m["dout"]), f64(m["dstate"]))
    for name, got in (("out", out), ("state", state), ("dx", g["x"]), ("da", g["a"]), ("dh0", g["h0"])):
        within(name, got, *r[name], where)
    return m, out, state, starts, g


@pytest.mark.parametrize("dtype,gate", TYPES)
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 127, 128, 129, 255, 256, 257, 1000])
def test_lengths(n, dtype, gate):
    check([n], 70, dtype, gate)


@pytest.mark.parametrize("dtype,gate", TYPES)
@pytest.mark.parametrize("C", [1, 2, 63, 64, 65, 128, 130, 257])
def test_widths(C, dtype, gate):
    check([150, 3], C, dtype, gate)


@pytest.mark.parametrize("dtype,gate", TYPES)
@pytest.mark.parametrize("lens", [[0], [0, 0, 5], [5, 0, 300, 1, 0, 128, 40], [1] * 130, [17] * 70, [3000, 1, 1, 700]])
def test_packed_sequences(lens, dtype, gate):
    check(lens, 33, dtype, gate)
    check(lens, 66, dtype, gate)


@pytest.mark.parametrize("dtype,gate", TYPES)
@pytest.mark.parametrize("S,n,C", [(1, 5000, 64), (2, 3000, 200), (3, 700, 34)])
def test_sequences_in_parts(S, n, C, dtype, gate):
    """Few sequences and channels: a sequence is cut into parts."""
    check([n - 37 * i for i in range(S)], C, dtype, gate, low=0.9)


@pytest.mark.parametrize("dtype,gate", TYPES)
def test_many_sequences_and_channels(dtype, gate):
    """Enough workgroups without parts."""
    check([40 + i % 200 for i in range(70)], 260, dtype, gate)


@pytest.mark.parametrize("dtype,gate", TYPES)
@pytest.mark.parametrize("lens,before,after", [([40, 30], 0, 30), ([40, 30], 17, 3), ([700], 300, 500), ([1], 0, 300),
                                               ([1, 1, 1], 5, 5), ([0, 0], 64, 65), ([], 0, 33)])
def test_tokens_outside_every_sequence(lens, before, after, dtype, gate, monkeypatch):
    real = torch.empty

    def empty(*a, **k):  # what the calls allocate holds NaN before the kernels write it
        t = real(*a, **k)
        return t.fill_(float("nan") if t.is_floating_point() else 255)
    monkeypatch.setattr(torch, "empty", empty)
    for C in (31, 64):
        check(lens, C, dtype, gate, before=before, after=after)


@pytest.mark.parametrize("dtype,gate", TYPES)
def test_gates_of_zero_and_one(dtype, gate):
    """A gate of 0 forgets everything before it, one of 1 keeps all of it."""
    import chunk_weight_rnn_amd as e2
    m = make([400], 64, dtype, gate)
    m["a"][:] = 1
    m["a"][130] = 0
    m["x"][:129] = 1e30
    out, state, starts = e2.gated_scan_forward(m["x"], m["a"], m["cu"], h0=m["h0"], save=True)
    assert torch.equal(out[130], m["x"][130])
    r = ref.scan(f64(m["x"][130:]), f64(m["a"][130:]), np.zeros((1, 64)), [270], 0, dtype, gate)
    within("out", out[130:], *r["out"], "after the gate of 0")
    g = e2.gated_scan_backward(m["dout"], m["x"], m["a"], starts, m["cu"])
    assert torch.isfinite(g["a"][131:]).all() and torch.isfinite(g["x"]).all()


@pytest.mark.parametrize("dtype,gate", TYPES)
@pytest.mark.parametrize("lens", [[1] * 9, [600], [100] * 40])
def test_not_finite_values_stay_in_their_channel_and_after(lens, dtype, gate):
    import chunk_weight_rnn_amd as e2
    m = make(lens, 66, dtype, gate)
    want, ws, _ = e2.gated_scan_forward(m["x"], m["a"], m["cu"], h0=m["h0"])
    t = sum(lens) // 2
    m["x"][t, 7] = float("nan")
    out, state, _ = e2.gated_scan_forward(m["x"], m["a"], m["cu"], h0=m["h0"])
    seq = int(torch.searchsorted(m["cu"], torch.tensor(t, dtype=torch.int32, device="cuda"), right=True)) - 1
    end = int(m["cu"][seq + 1])
    assert torch.isnan(out[t:end, 7]).all() and torch.isnan(state[seq, 7])
    keep = torch.ones_like(out, dtype=torch.bool)
    keep[t:end, 7] = False
    assert torch.equal(out[keep], want[keep])
    state[seq, 7] = ws[seq, 7]
    assert torch.equal(state, ws)


@pytest.mark.parametrize("dtype,gate", TYPES)
@pytest.mark.parametrize("lens", [[1] * 6, [9, 0, 600], [300] * 3, [60] * 70])
def test_state_carries_over_calls_in_place(lens, dtype, gate):
    """Two calls with the state in place give what one call over both gives."""
    import chunk_weight_rnn_amd as e2
    a, b = make(lens, 130, dtype, gate, seed=1), make(lens, 130, dtype, gate, seed=2)
    join = lambda k: torch.cat([t[i] for s in range(len(lens)) for t, i in
                                ((a[k], slice(int(a["cu"][s]), int(a["cu"][s + 1]))), (b[k], slice(int(b["cu"][s]), int(b["cu"][s + 1]))))])
    state = a["h0"].clone()
    oa, s1, _ = e2.gated_scan_forward(a["x"], a["a"], a["cu"], h0=state, state=state)
    assert s1 is state
    ob, _, _ = e2.gated_scan_forward(b["x"], b["a"], b["cu"], h0=state, state=state)
    whole = ref.scan(f64(join("x")), f64(join("a")), f64(a["h0"]), [2 * n for n in lens], 0, dtype, gate)
    within("state", state, *whole["state"], str(lens))
    at = 0
    for s, n in enumerate(lens):
        for o, i in ((oa, int(a["cu"][s])), (ob, int(b["cu"][s]))):
            within("out", o[i:i + n], whole["out"][0][at:at + n], whole["out"][1][at:at + n], f"seq {s}")
            at += n


@pytest.mark.parametrize("dtype,gate", TYPES)
@pytest.mark.parametrize("lens", [[1] * 20, [500, 60], [129] * 70])
def test_strides_and_alignment(lens, dtype, gate):
    """Views of a wider tensor, and tensors that begin at an odd element: the same bits
    as contiguous ones wherever the same channels go together."""
    import chunk_weight_rnn_amd as e2
    m = make(lens, 62, dtype, gate)
    want = e2.gated_scan_forward(m["x"], m["a"], m["cu"], h0=m["h0"], save=True)
    n = sum(lens)
    for off, wide in ((0, 200), (2, 64), (1, 63), (3, 71)):
        x, a = torch.full((n, wide), 7.0, device="cuda").to(m["x"].dtype), torch.full((n, wide), 7.0, device="cuda").to(m["a"].dtype)
        x[:, off:off + 62], a[:, off:off + 62] = m["x"], m["a"]
        x, a = x[:, off:off + 62], a[:, off:off + 62]
        out, state, starts = e2.gated_scan_forward(x, a, m["cu"], h0=m["h0"], save=True)
        assert torch.equal(out, want[0]) and torch.equal(state, want[1])
        g = e2.gated_scan_backward(m["dout"], x, a, starts, m["cu"], dstate=m["dstate"])
        w = e2.gated_scan_backward(m["dout"], m["x"], m["a"], want[2], m["cu"], dstate=m["dstate"])
        assert all(torch.equal(g[k], w[k]) for k in g)


def test_no_states_given():
    import chunk_weight_rnn_amd as e2
    m = make([100, 5], 40, "f32", "f32")
    out, state, starts = e2.gated_scan_forward(m["x"], m["a"], m["cu"])
    zero = torch.zeros_like(m["h0"])
    want = e2.gated_scan_forward(m["x"], m["a"], m["cu"], h0=zero, save=True)
    assert starts is None and torch.equal(out, want[0]) and torch.equal(state, want[1])
    g, w = (e2.gated_scan_backward(m["dout"], m["x"], m["a"], want[2], m["cu"], dstate=d) for d in (None, zero))
    assert all(torch.equal(g[k], w[k]) for k in g)


@pytest.mark.parametrize("lens", [[7, 0, 3], [140]])
def test_gradients_against_differences(lens):
    """Central differences of the 64-bit definition along random directions."""
    import chunk_weight_rnn_amd as e2
    C = 6
    m = make(lens, C, "f32", "f32", low=0.5)
    x, a, h0 = (m[k].clone().requires_grad_(True) for k in ("x", "a", "h0"))
    out, state = e2.gated_scan(x, a, m["cu"], h0)
    ((out * m["dout"]).sum() + (state * m["dstate"]).sum()).backward()
    f = {k: f64(m[k]) for k in ("x", "a", "h0", "dout", "dstate")}

    def loss(x, a, h0):
        r = ref.scan(x, a, h0, lens, 0, "f32", "f32")
        return (r["out"][0] * f["dout"]).sum() + (r["state"][0] * f["dstate"]).sum()
    rng = np.random.default_rng(0)
    for name, t in (("x", x), ("a", a), ("h0", h0)):
        v = rng.standard_normal(f[name].shape)
        h = 1e-6
        args = lambda s: [f[k] + (s * h * v if k == name else 0) for k in ("x", "a", "h0")]
        want = (loss(*args(1)) - loss(*args(-1))) / (2 * h)
        got = float((t.grad.double().cpu().numpy() * v).sum())
        assert abs(got - want) < 1e-4 * max(1.0, abs(want)), name  # 1e-10 / 1e-6 of differences, fp32 sums


def test_autograd_needs_only_what_is_used():
    import chunk_weight_rnn_amd as e2
    m = make([50], 8, "bf16", "f32")
    x, a = m["x"].clone().requires_grad_(True), m["a"].clone().requires_grad_(True)
    out, state = e2.gated_scan(x, a, m["cu"])
    out.float().sum().backward()  # nothing arrives at the state, h0 is not there
    gx = x.grad.clone()
    x.grad = a.grad = None
    out, state = e2.gated_scan(x, a, m["cu"], torch.zeros(1, 8, device="cuda"))
    out.float().sum().backward()
    assert torch.equal(gx, x.grad)
    x.grad = None
    out, state = e2.gated_scan(x, a, m["cu"])
    state.sum().backward()
    assert torch.equal(x.grad[-1].float(), torch.ones(8, device="cuda"))
    x2 = m["x"].clone().requires_grad_(True)
    (g,) = torch.autograd.grad(e2.gated_scan(x2, a, m["cu"])[0].float().sum(), x2, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


def test_wrong_offsets_stay_inside():
    """Offsets that fall, or lie outside, are clamped: no access outside, no result promised."""
    import chunk_weight_rnn_amd as e2
    for lens in ([50, 60, 70], [900, 900], [1, 1, 1]):
        m = make(lens, 64, "bf16", "f32")
        for cu in (m["cu"].flip(0).contiguous(), m["cu"] + 10 ** 6, m["cu"] - 10 ** 6, m["cu"] * 0 + sum(lens),
                   torch.tensor([0] + [sum(lens)] * len(lens), dtype=torch.int32, device="cuda")):
            _, _, starts = e2.gated_scan_forward(m["x"], m["a"], cu, h0=m["h0"], save=True)
            e2.gated_scan_backward(m["dout"], m["x"], m["a"], starts, cu, dstate=m["dstate"])
    torch.cuda.synchronize()
