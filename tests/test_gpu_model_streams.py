"""The operators around a hybrid model's layers on streams and in graphs:
``stream=`` runs a call on that stream with what it allocates belonging to it;
captured calls, replayed with eager work and other inputs between, give the
eager call's bits; a serving step of all of them is one graph; a workspace is
taken over by the next call, whatever it holds."""
import pytest
import torch

from tests.gpu_util import note

pytestmark = pytest.mark.gpu


def _cu(lens):
    return torch.tensor([0] + [sum(lens[:i + 1]) for i in range(len(lens))], dtype=torch.int32, device="cuda")


def _cache8(seqs, ctx, K=2, D=64, page=16):
    import chunk_weight_rnn_amd as e2
    g = torch.Generator(device="cuda").manual_seed(5)
    per = -(-(ctx + 200) // page)
    kc, vc = (torch.zeros(seqs * per, K, page, D, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = (torch.zeros(seqs * per, K, page, dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu) for _ in range(2))
    table = torch.randperm(seqs * per, generator=g, device="cuda").to(torch.int32).view(seqs, per)
    q, k = (torch.randn(seqs * ctx, K, D, generator=g, device="cuda").bfloat16() for _ in range(2))
    e2.paged_attention(q, k, k.flip(0), kc, vc, table, _cu([ctx] * seqs), torch.zeros(seqs, dtype=torch.int32, device="cuda"),
                       k_scale=ks, v_scale=vs)
    return kc, vc, table, ks, vs


def _calls():
    """Calls with workspaces and without, by name, and the tensors that they read."""
    import chunk_weight_rnn_amd as e2
    g = torch.Generator(device="cuda").manual_seed(1)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device="cuda").to(dtype)

    tokens, weight, d = torch.randint(300, (700,), generator=g, device="cuda"), normal(300, 520, dtype=torch.float32), normal(700, 520)
    x, dout = normal(2500, 200), normal(2500, 200)
    a = torch.rand(2500, 200, generator=g, device="cuda")
    cu, ones = _cu([1800, 5, 0, 695]), _cu([1] * 6)
    starts = e2.gated_scan_forward(x, a, cu, save=True)[2]
    logits, u = normal(5, 40000), torch.rand(5, generator=g, device="cuda")
    few = normal(5, 90)

    def paged(n, ctx):
        kc, vc, table, ks, vs = _cache8(2, ctx)
        q, k, v = (normal(2 * n, h, 64) for h in (4, 2, 2))
        cached = torch.full((2,), ctx, dtype=torch.int32, device="cuda")
        return lambda **s: (e2.paged_attention(q, k, v, kc, vc, table, _twos[n], cached, k_scale=ks, v_scale=vs, **s),
                            kc.view(torch.uint8), ks.view(torch.uint8)), (q, k, v)

    _twos = {n: _cu([n] * 2) for n in (1, 100)}
    decode, chunk = paged(1, 900), paged(100, 900)
    return {
        "lookup": (lambda **s: (e2.embedding_forward(tokens, weight, dtype=torch.bfloat16, **s),), (weight,)),
        "lookup_backward": (lambda **s: (e2.embedding_backward(d, tokens, 300, dtype=torch.float32, **s),), (d,)),
        "scan": (lambda **s: e2.gated_scan_forward(x, a, cu, save=True, **s)[:2], (x,)),
        "scan_step": (lambda **s: e2.gated_scan_forward(x[:6], a[:6], ones, **s)[:2], (x,)),
        "scan_backward": (lambda **s: tuple(e2.gated_scan_backward(dout, x, a, starts, cu, **s).values()), (dout,)),
        "decode": decode,
        "chunk": chunk,
        "sample": (lambda **s: e2.sample(logits, u, temperature=0.8, top_k=1000, top_p=0.9, **s), (logits,)),
        "sample_few": (lambda **s: e2.sample(few, u, top_p=0.9, **s), (few,)),
    }


NAMES = ["lookup", "lookup_backward", "scan", "scan_step", "scan_backward", "decode", "chunk", "sample", "sample_few"]


def _same(a, b):
    return all(torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8)) for x, y in zip(a, b))


def _copy(ts):
    return tuple(t.clone() for t in ts)


@pytest.mark.parametrize("name", NAMES)
def test_stream_argument_owns_what_is_allocated(name, monkeypatch):
    note(f"{name} with stream=")
    call = _calls()[name][0]
    want = _copy(call())
    torch.cuda.synchronize()
    s, seen = torch.cuda.Stream(), []
    for fn in ("empty", "empty_like"):
        real = getattr(torch, fn)
        monkeypatch.setattr(torch, fn, lambda *a, _real=real, **k: (seen.append(torch.cuda.current_stream()), _real(*a, **k))[1])
    got = call(stream=s)
    monkeypatch.undo()
    assert seen and all(x == s for x in seen)
    s.synchronize()
    assert _same(got, want)


@pytest.mark.parametrize("name", NAMES)
def test_graph_replay(name):
    note(f"{name} captured")
    call, inputs = _calls()[name]
    call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = call()
    for i in range(4):
        for t in inputs:
            t.copy_(t.flip(0) if i % 2 else t * 0.5)
        want = _copy(call())
        torch.cuda.synchronize()
        graph.replay()
        torch.randn(1 << 20, device="cuda").sum().item()
        assert _same(held, want), i


def test_a_serving_step_in_one_graph():
    """Token -> vector -> recurrence -> attention over the 8-bit cache -> logits -> token, the
    state and the cache carried from replay to replay, as the eager loop gives them."""
    note("a serving step in one graph")
    import chunk_weight_rnn_amd as e2
    S, K, D, V = 3, 2, 64, 500
    W = K * D
    g = torch.Generator(device="cuda").manual_seed(2)
    weight = torch.randn(V, W, generator=g, device="cuda")
    head = torch.randn(W, V, generator=g, device="cuda").bfloat16()
    cu = _cu([1] * S)

    def fresh():
        kc, vc, table, ks, vs = _cache8(S, 50, K, D)
        return dict(token=torch.tensor([3, 4, 5], device="cuda"), state=torch.zeros(S, W, device="cuda"), cache=(kc, vc, table, ks, vs),
                    cached=torch.full((S,), 50, dtype=torch.int32, device="cuda"), u=torch.zeros(S, device="cuda"))

    def step(s):
        x = e2.embedding_forward(s["token"], weight, dtype=torch.bfloat16)
        h = e2.gated_scan_forward(x, torch.sigmoid(x.float()), cu, h0=s["state"], state=s["state"])[0]
        kc, vc, table, ks, vs = s["cache"]
        q = h.view(S, K, D)
        o = e2.paged_attention(q, q, q, kc, vc, table, cu, s["cached"], k_scale=ks, v_scale=vs)
        e2.sample(o.view(S, W) @ head, s["u"], temperature=0.7, top_k=40, top_p=0.95, token=s["token"])
        s["cached"] += 1

    us = torch.rand(20, S, generator=g, device="cuda")
    eager, tokens = fresh(), []
    for u in us:
        eager["u"].copy_(u)
        step(eager)
        tokens.append(eager["token"].clone())
    held = fresh()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(held)
    torch.cuda.current_stream().wait_stream(side)
    start = fresh()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(held)
    for name in ("token", "state", "cached"):
        held[name].copy_(start[name])
    for a, b in zip(held["cache"], start["cache"]):
        a.view(torch.uint8).copy_(b.view(torch.uint8))
    for i, u in enumerate(us):
        held["u"].copy_(u)
        graph.replay()
        assert torch.equal(held["token"], tokens[i]), i
    assert torch.equal(held["state"], eager["state"])
    for a, b in zip(held["cache"], eager["cache"]):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("fill", [0, 255])
@pytest.mark.parametrize("name", NAMES)
def test_a_workspace_may_hold_anything(name, fill):
    note(f"{name}, a workspace full of {fill}")
    call = _calls()[name][0]
    if name in ("lookup",):
        return  # takes none
    want = _copy(call())
    ws = torch.full((1 << 24,), fill, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        assert _same(call(workspace=ws), want)


def test_captured_gradients():
    """Forward and backward in one graph; refused in the forward while an eager graph of the
    same leaves is alive, since the backward would end the process."""
    note("captured gradients")
    import chunk_weight_rnn_amd as e2
    g = torch.Generator(device="cuda").manual_seed(3)
    tokens = torch.randint(90, (400,), generator=g, device="cuda")
    weight = torch.randn(90, 72, generator=g, device="cuda").requires_grad_()
    gates = torch.rand(400, 72, generator=g, device="cuda").requires_grad_()
    dout = torch.randn(400, 72, generator=g, device="cuda").bfloat16()
    cu = _cu([150, 250])

    def forward():
        return e2.gated_scan(e2.embedding(tokens, weight, dtype=torch.bfloat16), gates, cu)[0]

    def grads():
        return torch.autograd.grad(forward(), (weight, gates), dout)

    want = grads()
    alive = forward()
    torch.cuda.synchronize()
    refused = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError, match="another stream"):
        with torch.cuda.graph(refused):
            forward()
    del alive
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        grads()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = grads()
    for i in range(4):
        graph.replay()
        torch.randn(1 << 20, device="cuda").sum().item()
        assert _same(held, want), i
        assert _same(grads(), want), i


def test_second_derivatives_are_refused():
    import chunk_weight_rnn_amd as e2
    weight = torch.randn(9, 8, device="cuda").requires_grad_()
    x = e2.embedding(torch.arange(9, device="cuda"), weight)
    a = torch.rand(9, 8, device="cuda").requires_grad_()
    for y, leaf in ((x, weight), (e2.gated_scan(x, a, _cu([9]))[0], a)):
        (g,) = torch.autograd.grad((y * y).sum(), leaf, create_graph=True)
        with pytest.raises(RuntimeError):
            torch.autograd.grad(g.sum(), leaf)


def test_recurrences_on_several_streams_at_once():
    """Tiles wait for tiles of their own call alone, however the calls share the chip."""
    note("recurrences on four streams")
    import chunk_weight_rnn_amd as e2
    g = torch.Generator(device="cuda").manual_seed(7)
    calls = []
    for n in (9000, 6000, 4097, 8191):
        x, d = (torch.randn(n, 1000, generator=g, device="cuda").bfloat16() for _ in range(2))
        a, cu = torch.rand(n, 1000, generator=g, device="cuda"), _cu([n // 3, n - n // 3])
        out, state, starts = e2.gated_scan_forward(x, a, cu, save=True)
        grads = e2.gated_scan_backward(d, x, a, starts, cu)
        calls.append((x, a, cu, d, (out, state, starts), tuple(grads.values())))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = []
    for _ in range(3):
        for s, (x, a, cu, d, *_rest) in zip(streams, calls):
            f = e2.gated_scan_forward(x, a, cu, save=True, stream=s)
            got.append((f, tuple(e2.gated_scan_backward(d, x, a, f[2], cu, stream=s).values())))
    torch.cuda.synchronize()
    for i, (f, b) in enumerate(got):
        want = calls[i % len(calls)]
        assert _same(f[:2], want[4][:2]) and _same(b, want[5]), i
