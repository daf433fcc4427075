"""The layer operators on streams and in graphs: ``stream=`` runs a call on
that stream with what it allocates belonging to it; captured calls, replayed
with eager work between, give the eager call's bits; second derivatives, which
the operators do not have, are refused."""
import pytest
import torch

from tests.gpu_util import note

pytestmark = pytest.mark.gpu


def _packed(dtype, lens, H, K, D, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = sum(lens)
    q, k, v, dout = (torch.randn(n, h, D, generator=g, device="cuda").to(dtype) for h in (H, K, K, H))
    cu = torch.tensor([0] + [sum(lens[:i + 1]) for i in range(len(lens))], dtype=torch.int32, device="cuda")
    return q, k, v, dout, cu


def _paged(dtype, news, H, K, D, page, cached, seed=0):
    q, k, v, _, cu = _packed(dtype, news, H, K, D, seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    per = -(-(max(cached) + max(news)) // page)
    kc, vc = (torch.randn(per * len(news), K, page, D, generator=g, device="cuda").to(dtype) for _ in range(2))
    table = torch.arange(per * len(news), dtype=torch.int32, device="cuda").view(len(news), per)
    return q, k, v, kc, vc, table, cu, torch.tensor(cached, dtype=torch.int32, device="cuda")


def _calls(dtype):
    """Calls with workspaces and without, by name."""
    import chunk_weight_rnn_amd as e2
    q, k, v, dout, cu = _packed(dtype, [300, 1, 77], 4, 2, 64)
    out, lse = e2.attention_forward(q, k, v, cu)
    decode, chunk = (_paged(dtype, n, 4, 2, 64, 16, c) for n, c in (([1, 1], [3000, 5]), ([100, 60], [2000, 0])))
    x, r, dy = (torch.randn(33, 520, device="cuda").to(dtype) for _ in range(3))
    w = torch.rand(520, device="cuda")
    rstd = e2.norm_forward(x, w)[3]
    return {
        "forward": lambda **s: e2.attention_forward(q, k, v, cu, window=50, **s),
        "backward": lambda **s: tuple(e2.attention_backward(q, k, v, out, lse, dout, cu, **s).values()),
        "decode": lambda **s: (e2.paged_attention(*decode, **s),),
        "chunk": lambda **s: (e2.paged_attention(*chunk, **s),),
        "norm": lambda **s: e2.norm_forward(x, w, residual=r, **s)[::2],
        "norm8": lambda **s: e2.norm_forward(x, w, bits8=True, **s)[:2],
        "norm_backward": lambda **s: e2.norm_backward(dy, x, w, rstd, **s),
    }


NAMES = ["forward", "backward", "decode", "chunk", "norm", "norm8", "norm_backward"]


def _same(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b) if x is not None)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("name", NAMES)
def test_stream_argument_owns_what_is_allocated(name, dtype, monkeypatch):
    note(f"{name} {dtype} with stream=")
    call = _calls(dtype)[name]
    want = call()
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


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("name", NAMES)
def test_graph_replay(name, dtype):
    note(f"{name} {dtype} in a graph")
    call = _calls(dtype)[name]
    want = call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for rep in range(4):
        other = call()  # eager work between replays
        for t in got:
            if t is not None:
                t.view(torch.uint8).zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert _same(got, want), f"replay {rep}"
        assert _same(other, want), f"eager call {rep}"


def test_second_derivatives_are_refused():
    import chunk_weight_rnn_amd as e2
    q, k, v, dout, cu = _packed(torch.float32, [9], 2, 1, 32)
    q.requires_grad_(True)
    (g,) = torch.autograd.grad((e2.attention(q, k, v, cu) * dout).sum(), q, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()
