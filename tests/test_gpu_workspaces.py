"""Workspaces of the operators around a hybrid model's layers: calls that need one give the
same bits whatever it holds, from one of exactly the size asked for, and leave what follows
it alone."""
import pytest
import torch

from tests.gpu_util import note
from tests.test_gpu_model_streams import _cache8, _copy, _cu, _same

pytestmark = pytest.mark.gpu


def _calls():
    """Calls that need a workspace, by name."""
    import chunk_weight_rnn_amd as e2
    g = torch.Generator(device="cuda").manual_seed(1)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device="cuda").to(dtype)

    tokens, d = torch.randint(300, (5000,), generator=g, device="cuda"), normal(5000, 520)
    many = tokens % 3  # rows of many places, which are summed in pieces
    x, dout = normal(6100, 200), normal(6100, 200)
    a = torch.rand(6100, 200, generator=g, device="cuda")
    cu = _cu([5400, 5, 0, 695])
    starts = e2.gated_scan_forward(x, a, cu, save=True)[2]

    def paged(n, ctx, seqs):
        kc, vc, table, ks, vs = _cache8(seqs, ctx)
        q, k, v = (normal(seqs * n, h, 64) for h in (4, 2, 2))
        cached, at = torch.full((seqs,), ctx, dtype=torch.int32, device="cuda"), _cu([n] * seqs)
        return lambda **s: (e2.paged_attention(q, k, v, kc, vc, table, at, cached, k_scale=ks, v_scale=vs, **s), kc.view(torch.uint8),
                            vc.view(torch.uint8), ks.view(torch.uint8), vs.view(torch.uint8))

    return {
        "lookup_backward": lambda **s: (e2.embedding_backward(d, tokens, 300, dtype=torch.float32, **s),),
        "lookup_backward_pieces": lambda **s: (e2.embedding_backward(d, many, 300, dtype=torch.bfloat16, **s),),
        "lookup_backward_few": lambda **s: (e2.embedding_backward(d[:5], tokens[:5], 300, **s),),
        "scan": lambda **s: e2.gated_scan_forward(x, a, cu, save=True, **s)[:2],
        "scan_backward": lambda **s: tuple(e2.gated_scan_backward(dout, x, a, starts, cu, **s).values()),
        "decode": paged(1, 2500, 2),
        "decode_batch": paged(1, 900, 40),
        "chunk": paged(100, 1900, 2),
    }


NAMES = ["lookup_backward", "lookup_backward_pieces", "lookup_backward_few", "scan", "scan_backward", "decode", "decode_batch", "chunk"]
GUARD = 1 << 16


@pytest.mark.parametrize("name", NAMES)
def test_what_it_holds_and_what_follows_it(name, monkeypatch):
    note(f"{name} in a workspace of its size")
    from chunk_weight_rnn_amd import layer, tokens
    call, need, real = _calls()[name], [], layer._workspace

    def asked(workspace, size, like):
        need.append(size)
        return real(workspace, size, like)
    monkeypatch.setattr(layer, "_workspace", asked)
    monkeypatch.setattr(tokens, "_workspace", asked)
    want = _copy(call())
    monkeypatch.undo()
    assert len(need) == 1 and need[0] > 0
    for fill in (0, 255, 0x7f):
        held = torch.full((need[0] + GUARD,), fill, dtype=torch.uint8, device="cuda")
        for _ in range(2):  # the second call finds what the first one left
            assert _same(call(workspace=held[:need[0]]), want), fill
        assert bool((held[need[0]:] == fill).all()), fill


@pytest.mark.parametrize("name", NAMES)
def test_one_that_is_too_small_is_refused(name):
    import chunk_weight_rnn_amd as e2
    call = _calls()[name]
    with pytest.raises((e2.E2TTTError, ValueError)):
        call(workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
