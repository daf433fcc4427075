"""Attention over a paged cache in 8 bits on the GPU: what is written against
model_ref.quantise, bit for bit, and the outputs against layer_ref on what the cache
holds (an 8-bit value times its scale is a bf16 number, so the bounds are the bf16
ones)."""
import numpy as np
import pytest
import torch

from tests import layer_ref as ref
from tests import model_ref
from tests.gpu_util import note
from tests.test_gpu_attention import f64, offsets, within

pytestmark = pytest.mark.gpu

F8, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu


def make(ctx, new, H, K, D, page, seed=0, spread=0, spare=3):
    """A pool whose unused slots hold NaN, pages in random order, and the 64-bit keys
    and values of every sequence, as the cache holds or will hold them.  `spread`:
    rows' magnitudes differ by up to that many powers of two."""
    rng = np.random.default_rng(seed)
    need = [-(-(a + b) // page) for a, b in zip(ctx, new)]
    pool = sum(need) + spare
    order = rng.permutation(pool).astype(np.int32)
    table = np.full((len(ctx), max(need + [1]) + 1), -1, dtype=np.int32)
    at = 0
    for s, m in enumerate(need):
        table[s, :m] = order[at:at + m]
        at += m
    bf = lambda x: torch.from_numpy(x).to(torch.bfloat16)

    def rows(n, h):
        return bf(rng.standard_normal((n, h, D)) * 2.0 ** rng.integers(-spread, spread + 1, (n, h, 1)))
    N = sum(new)
    m = dict(q=bf(rng.standard_normal((N, H, D))).cuda(), cu=offsets(new), table=torch.from_numpy(table).cuda(),
             cached=torch.tensor(ctx, dtype=torch.int32, device="cuda"), held={}, bits={})
    for name in ("k", "v"):
        x = rows(N, K)
        m[name] = x.cuda()
        vals, b = model_ref.quantise(x.double().numpy())
        m["bits"][name] = b
        cache = torch.full((pool, K, page, D), 0x7f, dtype=torch.uint8)
        scale = torch.full((pool, K, page), 255, dtype=torch.uint8)
        held, a = [], 0
        for s, (c, n) in enumerate(zip(ctx, new)):
            old, ob = model_ref.quantise(rows(c, K).double().numpy())
            p = np.arange(c)
            pages = torch.from_numpy(table[s][p // page]).long()
            x8 = torch.from_numpy(old / 2.0 ** (ob[..., None] - 127.0)).float().to(F8).view(torch.uint8)
            cache[pages, :, p % page] = x8
            scale[pages, :, p % page] = torch.from_numpy(ob.astype(np.uint8))
            held.append(np.concatenate([old, vals[a:a + n]]))
            a += n
        m[name + "c"], m[name + "s"], m["held"][name] = cache.view(F8).cuda(), scale.view(E8).cuda(), held
    return m


def call(m, window=0, append=True, **kw):
    import chunk_weight_rnn_amd as e2
    k, v = (m["k"], m["v"]) if append else (None, None)
    return e2.paged_attention(m["q"], k, v, m["kc"], m["vc"], m["table"], m["cu"], m["cached"], window=window,
                              k_scale=m["ks"], v_scale=m["vs"], **kw)


def u8(t):
    return t.view(torch.uint8)


def check(ctx, new, H, K, D, page, window=0, seed=0, append=True, spread=0):
    where = f"ctx={ctx} new={new} H={H} K={K} D={D} page={page} window={window} append={append} spread={spread}"
    note("paged8 " + where)
    m = make(ctx, new, H, K, D, page, seed, spread)
    before = {n: u8(m[n]).clone() for n in ("kc", "vc", "ks", "vs")}
    if not append:
        call(m, window)
    out = call(m, window, append)
    torch.cuda.synchronize()
    a = 0
    for s, (c, n) in enumerate(zip(ctx, new)):
        ks, vs = m["held"]["k"][s], m["held"]["v"][s]
        for h in range(H):
            r = ref.attention(f64(m["q"][a:a + n, h]), ks[:, h * K // H], vs[:, h * K // H], c, window, D ** -0.5, "bf16")
            within("out", out[a:a + n, h], *r["out"], f"{where} seq {s} head {h}")
        p = np.arange(c, c + n)
        pages = m["table"][s].cpu().numpy()[p // page]
        for name in ("k", "v"):
            b = m["bits"][name][a:a + n]
            x8 = torch.from_numpy(m["held"][name][s][c:] / 2.0 ** (b[..., None] - 127.0)).float().to(F8)
            before[name + "c"][pages, :, p % page] = u8(x8.cuda())
            before[name + "s"][pages, :, p % page] = torch.from_numpy(b.astype(np.uint8)).cuda()
        a += n
    for n, x in before.items():  # the new tokens are in their slots, and nothing else was written
        assert torch.equal(x, u8(m[n])), f"{where} {n}"


@pytest.mark.parametrize("page", [1, 2, 16, 64, 256])
def test_single_tokens(page):
    check([0, 1, 15, 16, 17, 63, 64, 200, 700], [1] * 9, 8, 2, 64, page)


@pytest.mark.parametrize("H,K", [(1, 1), (6, 2), (7, 1), (4, 4), (16, 1), (40, 1)])
def test_head_groups(H, K):
    check([130, 0, 37], [1, 1, 1], H, K, 64, 16)
    check([130, 0, 37], [3, 40, 9], H, K, 64, 16)


@pytest.mark.parametrize("D", [16, 32, 48, 64, 80, 96, 128])
def test_head_dims(D):
    check([300, 5], [1, 1], 4, 2, D, 32)
    check([100, 5], [30, 20], 4, 2, D, 32)


@pytest.mark.parametrize("window", [1, 2, 16, 63, 100, 5000])
def test_windows(window):
    """Slots below every window may hold anything."""
    check([400, 90, 3], [1, 1, 1], 4, 2, 64, 16, window)
    check([400, 90, 3], [33, 70, 5], 4, 2, 64, 16, window)
    m = make([400], [1], 4, 2, 64, 16)
    want = call(m, window)
    p = torch.arange(max(0, 400 - window + 1), device="cuda")
    pages = m["table"][0].long()[p // 16]
    for n in ("kc", "vc"):
        u8(m[n])[pages, :, p % 16] = 0x7f
    for n in ("ks", "vs"):
        u8(m[n])[pages, :, p % 16] = 255
    got = call(m, window)
    assert torch.equal(got, want) and torch.isfinite(got).all()


def test_chunks_and_mixed_batches():
    check([0, 256, 100, 511, 64], [256, 1, 0, 77, 130], 8, 2, 64, 64)
    check([0], [300], 4, 1, 128, 64)
    check([900], [64], 16, 4, 128, 64)
    check([2500, 3], [70, 1], 4, 1, 128, 16)


@pytest.mark.parametrize("D,page,ctx", [(128, 64, [2600]), (64, 16, [3000, 9]), (128, 1, [1500]), (128, 256, [1023, 0, 1400])])
def test_long_contexts_of_single_tokens(D, page, ctx):
    """More units per workgroup than it has stages."""
    check(ctx, [1] * len(ctx), 4, 2, D, page)
    check(ctx, [2] * len(ctx), 4, 2, D, page, window=1000)


def test_many_sequences():
    check([(i * 37) % 90 for i in range(140)], [1 + (i % 3 == 0) for i in range(140)], 2, 1, 32, 16)


def test_new_tokens_already_in_the_cache():
    check([50, 0, 200], [1, 20, 64], 4, 2, 64, 16, append=False)


@pytest.mark.parametrize("new", [[1, 1], [20, 40]])
def test_magnitudes_of_every_size(new):
    check([150, 40], new, 4, 2, 64, 16, spread=6)


def test_rounding_into_the_cache():
    """Rows of every magnitude that bf16 has, at the border of a scale, zeros, and rows that
    are not finite."""
    D = 32
    tops = [2.0 ** e * f for e in range(-133, 128, 9) for f in (1.0, 1.75, 1.7578125, 1.9921875)] + [448.0, 450.0, 0.0, 3.3895e38, 1e-40]
    rng = np.random.default_rng(0)
    x = np.stack([np.concatenate([[t], t * rng.uniform(-1, 1, D - 1)]) for t in tops])
    x = torch.from_numpy(x).to(torch.bfloat16)
    bad = x[:3].clone()
    bad[0, 3], bad[1, 31], bad[2, 0] = float("nan"), float("inf"), -float("inf")
    x = torch.cat([x, bad])[:, None]
    n = len(x)
    want, b = model_ref.quantise(x.double().numpy())
    m = make([0], [n], 1, 1, D, 16)
    m["k"] = m["v"] = x.cuda()
    call(m)
    torch.cuda.synchronize()
    p = np.arange(n)
    pages = m["table"][0].cpu().numpy()[p // 16]
    for name in ("k", "v"):
        got = u8(m[name + "s"])[pages, :, p % 16].cpu().numpy()
        assert (got == b).all()
        x8 = m[name + "c"].view(torch.uint8)[pages, :, p % 16].view(F8).double().cpu().numpy()
        with np.errstate(invalid="ignore"):
            y = x8 * np.where(b < 255, 2.0 ** (b - 127.0), np.nan)[..., None]
        assert np.array_equal(y, want, equal_nan=True)
        assert np.isnan(x8[-3:]).all()


@pytest.mark.parametrize("new", [3, 100])
def test_not_finite_new_tokens_do_not_reach_earlier_ones(new):
    for which in ("k", "v"):
        m = make([70], [new], 4, 2, 64, 16)
        want = call(m)
        m[which][new // 2, 0, 7] = float("nan")
        got = call(m)
        note(f"not finite: new={new} {which}")
        assert torch.isnan(got[new // 2:, :2]).any(-1).all()  # the two query heads of that key head
        assert torch.isfinite(got[:new // 2]).all() and torch.isfinite(got[:, 2:]).all()
        assert (got[:new // 2].float() - want[:new // 2].float()).abs().max() <= 2 ** -6
        assert torch.equal(got[:, 2:], want[:, 2:])


def test_other_strides():
    """One tensor that holds keys and values slot by slot, [pages, page, 2, K, D]."""
    m = make([200, 33], [1, 1], 4, 2, 64, 16)
    kc, vc = m["kc"], m["vc"]
    both = torch.stack([u8(kc), u8(vc)], dim=0).permute(1, 3, 0, 2, 4).contiguous()
    want = call(m)
    m["kc"], m["vc"] = both[:, :, 0].transpose(1, 2).view(F8), both[:, :, 1].transpose(1, 2).view(F8)
    assert torch.equal(call(m), want)
    assert torch.equal(u8(m["kc"].contiguous()), u8(kc)) and torch.equal(u8(m["vc"].contiguous()), u8(vc))


def test_tokens_fed_one_by_one_and_in_chunks_leave_the_same_cache():
    """And see the same keys: outputs within twice the bound of one."""
    import chunk_weight_rnn_amd as e2
    n, H, K, D, page = 200, 4, 2, 64, 32
    m = make([0], [n], H, K, D, page, spread=3)
    whole = call(m)
    first = {k: u8(m[k]).clone() for k in ("kc", "vc", "ks", "vs")}
    at = 0
    for step in (1, 64, 100, 1, 34):
        sl = slice(at, at + step)
        out = e2.paged_attention(m["q"][sl], m["k"][sl], m["v"][sl], m["kc"], m["vc"], m["table"], offsets([step]),
                                 torch.tensor([at], dtype=torch.int32, device="cuda"), k_scale=m["ks"], v_scale=m["vs"])
        for h in range(H):
            r = ref.attention(f64(m["q"][sl, h]), m["held"]["k"][0][:at + step, h // 2], m["held"]["v"][0][:at + step, h // 2],
                              at, 0, D ** -0.5, "bf16")
            within("out", out[:, h], f64(whole[sl, h]), 2 * r["out"][1], f"chunk at {at}")
        at += step
    assert all(torch.equal(first[k], u8(m[k])) for k in first)


def test_wrong_pages_and_lengths_stay_inside():
    m = make([100, 40], [2, 30], 4, 2, 64, 16)
    table, cached = m["table"], m["cached"]
    for t, c in ((table * 0 + 10 ** 6, cached), (table * 0 - 7, cached), (table, cached + 10 ** 6), (table, cached - 10 ** 6)):
        m["table"], m["cached"] = t, c
        call(m)
        call(m, append=False)
    one = make([100, 40], [1, 1], 4, 2, 64, 16)
    for t, c in ((table * 0 + 10 ** 6, cached), (table * 0 - 7, cached), (table, cached + 10 ** 6), (table, cached - 10 ** 6)):
        one["table"], one["cached"] = t, c
        call(one)
    torch.cuda.synchronize()


def test_tokens_outside_every_sequence():
    m = make([30, 50], [4, 6], 4, 2, 64, 16)
    want = call(m)
    keep = {k: u8(m[k]).clone() for k in ("kc", "vc", "ks", "vs")}
    for n in ("q", "k", "v"):
        m[n] = torch.cat([torch.full_like(m[n][:3], float("nan")), m[n], torch.full_like(m[n], float("nan"))])
    m["cu"] = m["cu"] + 3
    out = torch.full_like(m["q"], float("nan"))
    call(m, out=out)
    assert torch.equal(out[3:13], want) and not out[:3].any() and not out[13:].any()
    assert all(torch.equal(keep[k], u8(m[k])) for k in keep)


def test_pool_past_32_bit_offsets():
    m = make([300], [1], 4, 2, 128, 64)
    want = call(m)
    pages = (1 << 32) // (2 * 64 * 128) + 1000
    t = m["table"].clone()
    new = {}
    for n in ("kc", "vc", "ks", "vs"):
        new[n] = torch.empty(pages, *m[n].shape[1:], dtype=torch.uint8, device="cuda")
    for i in range(5):
        at = pages - 1 - i if i % 2 else i
        for n in new:
            new[n][at] = u8(m[n])[m["table"][0, i].long()]
        t[0, i] = at
    m.update({n: x.view(F8 if n[1] == "c" else E8) for n, x in new.items()}, table=t)
    assert torch.equal(call(m), want)
