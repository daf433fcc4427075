"""Attention of new tokens over a paged cache on the GPU, against layer_ref."""
import numpy as np
import pytest
import torch

from tests import layer_ref as ref
from tests.gpu_util import note
from tests.test_gpu_attention import TYPES, f64, offsets, within

pytestmark = pytest.mark.gpu


def make(ctx, new, H, K, D, page, dtype, seed=0, fill=float("nan"), spare=3):
    """A pool whose unused slots hold `fill`, pages in random order, and the
    64-bit keys and values of every sequence."""
    rng = np.random.default_rng(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = TYPES[dtype]
    need = [-(-(a + b) // page) for a, b in zip(ctx, new)]
    pool = sum(need) + spare
    order = rng.permutation(pool).astype(np.int32)
    kc = torch.full((pool, K, page, D), fill, dtype=dt, device="cuda")
    vc = torch.full((pool, K, page, D), fill, dtype=dt, device="cuda")
    table = np.full((len(ctx), max(need + [1]) + 1), -1, dtype=np.int32)
    N = sum(new)
    t = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dt)
    q, k, v = t(N, H, D), t(N, K, D), t(N, K, D)
    old, at = [], 0
    for s, c in enumerate(ctx):
        table[s, :need[s]] = order[at:at + need[s]]
        at += need[s]
        ok, ov = t(c, K, D), t(c, K, D)
        old.append((ok, ov))
        p = torch.arange(c, device="cuda")
        pages = torch.from_numpy(table[s]).cuda().long()[p // page]
        kc[pages, :, p % page] = ok
        vc[pages, :, p % page] = ov
    return dict(q=q, k=k, v=v, kc=kc, vc=vc, table=torch.from_numpy(table).cuda(), cu=offsets(new),
                cached=torch.tensor(ctx, dtype=torch.int32, device="cuda"), old=old, need=need, order=order)


def check(ctx, new, H, K, D, page, dtype, window=0, seed=0, append=True):
    import chunk_weight_rnn_amd as e2
    where = f"ctx={ctx} new={new} H={H} K={K} D={D} page={page} {dtype} window={window} append={append}"
    note("paged " + where)
    m = make(ctx, new, H, K, D, page, dtype, seed)
    before = m["kc"].clone(), m["vc"].clone()
    args = (m["q"], m["k"], m["v"])
    if not append:  # a first call leaves the new tokens in the cache
        e2.paged_attention(*args, m["kc"], m["vc"], m["table"], m["cu"], m["cached"], window=window)
        args = (m["q"], None, None)
    out = e2.paged_attention(*args, m["kc"], m["vc"], m["table"], m["cu"], m["cached"], window=window)
    torch.cuda.synchronize()
    a = 0
    for s, (c, n) in enumerate(zip(ctx, new)):
        ks = np.concatenate([f64(m["old"][s][0]), f64(m["k"][a:a + n])])
        vs = np.concatenate([f64(m["old"][s][1]), f64(m["v"][a:a + n])])
        for h in range(H):
            r = ref.attention(f64(m["q"][a:a + n, h]), ks[:, h * K // H], vs[:, h * K // H], c, window, D ** -0.5, dtype)
            within("out", out[a:a + n, h], *r["out"], f"{where} seq {s} head {h}")
        # the new tokens are in their slots
        p = np.arange(c, c + n)
        pages = m["table"][s].cpu().numpy()[p // page]
        before[0][pages, :, p % page] = m["k"][a:a + n]
        before[1][pages, :, p % page] = m["v"][a:a + n]
        a += n
    for x, y in zip(before, (m["kc"], m["vc"])):  # and nothing else was written
        assert torch.equal(torch.nan_to_num(x.float(), nan=7e4), torch.nan_to_num(y.float(), nan=7e4)), where


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page", [1, 2, 16, 64, 256])
def test_single_tokens(page, dtype):
    check([0, 1, 15, 16, 17, 63, 64, 200, 700], [1] * 9, 8, 2, 64, page, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,K", [(1, 1), (6, 2), (7, 1), (4, 4), (16, 1), (40, 1)])
def test_head_groups(H, K, dtype):
    check([130, 0, 37], [1, 1, 1], H, K, 64, 16, dtype)
    check([130, 0, 37], [3, 40, 9], H, K, 64, 16, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [8, 32, 64, 96, 128])
def test_head_dims(D, dtype):
    check([300, 5], [1, 1], 4, 2, D, 32, dtype)
    check([100, 5], [30, 20], 4, 2, D, 32, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window", [1, 2, 16, 63, 100, 5000])
def test_windows(window, dtype):
    """Slots below every window hold NaN like the unused ones."""
    import chunk_weight_rnn_amd as e2
    check([400, 90, 3], [1, 1, 1], 4, 2, 64, 16, dtype, window)
    check([400, 90, 3], [33, 70, 5], 4, 2, 64, 16, dtype, window)
    m = make([400], [1], 4, 2, 64, 16, dtype)
    want = e2.paged_attention(m["q"], m["k"], m["v"], m["kc"], m["vc"], m["table"], m["cu"], m["cached"], window=window)
    p = torch.arange(max(0, 400 - window + 1), device="cuda")
    pages = m["table"][0].long()[p // 16]
    m["kc"][pages, :, p % 16] = float("nan")
    m["vc"][pages, :, p % 16] = float("inf")
    got = e2.paged_attention(m["q"], m["k"], m["v"], m["kc"], m["vc"], m["table"], m["cu"], m["cached"], window=window)
    assert torch.equal(got, want) and torch.isfinite(got).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_chunks_and_mixed_batches(dtype):
    """Chunks of a prompt, single tokens and idle sequences in one call."""
    check([0, 256, 100, 511, 64], [256, 1, 0, 77, 130], 8, 2, 64, 64, dtype)
    check([0], [300], 4, 1, 128, 64, dtype)
    check([900], [64], 16, 4, 128, 64, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_new_tokens_already_in_the_cache(dtype):
    check([50, 0, 200], [1, 20, 64], 4, 2, 64, 16, dtype, append=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new", [3, 100])
def test_not_finite_new_tokens_do_not_reach_earlier_ones(new, dtype):
    """A NaN in one new token's value or key leaves the rows before it as they are."""
    import chunk_weight_rnn_amd as e2
    for which in ("k", "v"):
        m = make([70], [new], 4, 2, 64, 16, dtype)
        run = lambda: e2.paged_attention(m["q"], m["k"], m["v"], m["kc"], m["vc"], m["table"], m["cu"], m["cached"])
        want = run()
        m[which][new // 2, 0, 7] = float("nan")
        got = run()
        note(f"not finite: new={new} {dtype} {which}")
        assert torch.isnan(got[new // 2:, :2]).any(-1).all()  # the two query heads of that key head
        assert torch.isfinite(got[:new // 2]).all() and torch.isfinite(got[:, 2:]).all()
        # the same sums, term by term where the fast ones were not finite
        assert (got[:new // 2].float() - want[:new // 2].float()).abs().max() <= 2 ** -6
        assert torch.equal(got[:, 2:], want[:, 2:])


def test_many_sequences():
    check([(i * 37) % 90 for i in range(140)], [1 + (i % 3 == 0) for i in range(140)], 2, 1, 32, 16, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_other_strides(dtype):
    """One tensor that holds keys and values slot by slot, [pages, page, 2, K, D]."""
    import chunk_weight_rnn_amd as e2
    m = make([200, 33], [1, 1], 4, 2, 64, 16, dtype)
    want = e2.paged_attention(m["q"], m["k"], m["v"], m["kc"].clone(), m["vc"].clone(), m["table"], m["cu"], m["cached"])
    both = torch.stack([m["kc"], m["vc"]], dim=0).permute(1, 3, 0, 2, 4).contiguous()
    kc, vc = both[:, :, 0].transpose(1, 2), both[:, :, 1].transpose(1, 2)
    got = e2.paged_attention(m["q"], m["k"], m["v"], kc, vc, m["table"], m["cu"], m["cached"])
    assert torch.equal(got, want)
    p = int(m["cached"][0])
    assert torch.equal(kc[m["table"][0, p // 16].long(), :, p % 16], m["k"][0])


def test_shared_pages():
    """Two sequences with the same first pages."""
    import chunk_weight_rnn_amd as e2
    m = make([64, 64], [1, 1], 4, 2, 64, 16, "bf16")
    t = m["table"].clone()
    t[1, :4] = t[0, :4]
    q = m["q"].clone()
    q[1] = q[0]
    k, v = m["k"].clone(), m["v"].clone()
    k[1], v[1] = k[0], v[0]
    out = e2.paged_attention(q, k, v, m["kc"], m["vc"], t, m["cu"], m["cached"])
    assert torch.equal(out[0], out[1])


def test_pool_past_32_bit_offsets():
    """A pool of more than 2^32 bytes, with pages at both ends of it."""
    import chunk_weight_rnn_amd as e2
    m = make([300], [1], 4, 2, 128, 64, "bf16")
    want = e2.paged_attention(m["q"], m["k"], m["v"], m["kc"], m["vc"], m["table"], m["cu"], m["cached"])
    pages = (1 << 32) // (2 * 64 * 128 * 2) + 1000
    kc = torch.empty(pages, 2, 64, 128, dtype=torch.bfloat16, device="cuda")
    vc = torch.empty(pages, 2, 64, 128, dtype=torch.bfloat16, device="cuda")
    t = m["table"].clone()
    for i in range(5):
        at = pages - 1 - i if i % 2 else i
        kc[at], vc[at] = m["kc"][m["table"][0, i].long()], m["vc"][m["table"][0, i].long()]
        t[0, i] = at
    got = e2.paged_attention(m["q"], m["k"], m["v"], kc, vc, t, m["cu"], m["cached"])
    assert torch.equal(got, want)


def test_streamed_chunks_equal_the_whole_prompt():
    """A prompt fed a chunk per call gives what attention_forward gives for the
    whole of it, within twice the bound of one."""
    import chunk_weight_rnn_amd as e2
    n, H, K, D, page = 500, 8, 2, 64, 32
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn(n, h, D, generator=g, device="cuda").bfloat16() for h in (H, K, K))
    whole, _ = e2.attention_forward(q, k, v, offsets([n]), window=200)
    _, bnd = ref.packed(f64(q), f64(k), f64(v), [n], 200, D ** -0.5, "bf16")
    kc = torch.full((20, K, page, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    table = torch.randperm(20, device="cuda").to(torch.int32)[None, :].contiguous()
    at = 0
    for step in (1, 64, 100, 1, 200, 134):
        sl = slice(at, at + step)
        out = e2.paged_attention(q[sl], k[sl], v[sl], kc, vc, table, offsets([step]),
                                 torch.tensor([at], dtype=torch.int32, device="cuda"), window=200)
        within("out", out, f64(whole[sl]), 2 * bnd["out"][sl], f"chunk at {at}")
        at += step


def test_wrong_pages_and_lengths_stay_inside():
    """Page indices and lengths that do not fit are clamped: no access outside,
    no result promised."""
    import chunk_weight_rnn_amd as e2
    m = make([100, 40], [2, 30], 4, 2, 64, 16, "bf16")
    cases = [(m["table"] * 0 + 10 ** 6, m["cached"]), (m["table"] * 0 - 7, m["cached"]),
             (m["table"], m["cached"] + 10 ** 6), (m["table"], m["cached"] - 10 ** 6)]
    for t, c in cases:
        e2.paged_attention(m["q"], m["k"], m["v"], m["kc"], m["vc"], t, m["cu"], c)
        e2.paged_attention(m["q"], None, None, m["kc"], m["vc"], t, m["cu"], c)
    torch.cuda.synchronize()


def test_a_captured_step_replays():
    """One decoding step in a HIP graph: replays see what the buffers hold then."""
    import chunk_weight_rnn_amd as e2
    m = make([100, 40], [1, 1], 8, 2, 64, 16, "bf16")
    out = torch.empty_like(m["q"])
    call = lambda: e2.paged_attention(m["q"], m["k"], m["v"], m["kc"], m["vc"], m["table"], m["cu"], m["cached"], out=out)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    g = torch.Generator(device="cuda").manual_seed(9)
    for i in range(4):
        m["q"].copy_(torch.randn(m["q"].shape, generator=g, device="cuda"))
        m["cached"].add_(1)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        call()
        torch.cuda.synchronize()
        assert torch.equal(got, out), i
