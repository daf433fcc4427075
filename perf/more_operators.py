"""What is measured of the operators that a hybrid model runs around its layers.

* ``embed`` / ``embed_train``: token lookup with a scale; its gradient, a dense
  tensor in which the rows of equal tokens are summed;
* ``scan`` / ``scan_train``: the gated linear recurrence
  h_t = a_t h_{t-1} + x_t of every channel over packed sequences, with the state
  carried in and out; forward alone or forward and backward;
* ``paged8``: attention of new tokens over a paged cache of 8-bit keys and
  values, which the call first extends by the new ones, quantised;
* ``sample``: one token per row of logits by temperature, top-k, top-p and
  min-p, from given random numbers, and the log of its probability.

``run`` computes them in elementary torch operations in 32 bits (weights of the
sampling in whole multiples of 2^-44), or, where ``own`` is true, through the
package's entry points.  ``exact`` is the definition in 64 bits.
"""
import random

import numpy as np
import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f32": 4}
_F8 = torch.float8_e4m3fn
_E8 = torch.float8_e8m0fnu
_F8_MAX = 448.0
_ONE = 1 << 44  # the largest weight of a row of logits


# ------------------------------------------------------------------- cases
def listed():
    return [
        # the next tokens of eight streams: latency counts
        _embed("embed_decode", "embed", "bf16", "bf16", tokens=8, vocab=32000, width=2048),
        # a training step's lookup and gradient, 8 rows of 2K tokens of text, fp32 master weights
        _embed("embed_train_2k", "embed_train", "f32", "bf16", tokens=16384, vocab=32000, width=2048),
        # a model over bytes: few rows, each of them summed over many tokens
        _embed("embed_train_bytes", "embed_train", "f32", "bf16", tokens=16384, vocab=256, width=512),
        # one new token of each stream of a serving batch, states updated in place
        _scan("scan_step", "scan", "bf16", "f32", seqs=64, longest=1, width=2048),
        # a training step: 8 packed rows of up to 2K tokens, gates in fp32
        _scan("scan_train_2k", "scan_train", "bf16", "f32", seqs=8, longest=2048, width=2048),
        # the 16K sequence read at once: a single chain of tokens
        _scan("scan_16k", "scan", "bf16", "bf16", seqs=1, longest=16384, width=2048),
        # one user's next token over a short 8-bit cache: latency counts
        _paged8("decode8_one", 16, 4, 128, page=16, seqs=1, new=1, context=513, window=0),
        # the next tokens of a full serving batch, contexts of every length up to 16K
        _paged8("decode8_batch", 16, 4, 128, page=64, seqs=64, new=1, context=16383, window=0),
        # eight streams, a 256-token chunk each, window of 2K
        _paged8("chunk8_batch", 16, 4, 128, page=64, seqs=8, new=256, context=8191, window=2048),
        # one user's next token, all filters
        _sample("sample_one", "bf16", rows=1, vocab=32000, filters="all"),
        # a serving batch whose users each set their own
        _sample("sample_batch", "bf16", rows=64, vocab=32000, filters="mixed"),
        # a batch of samples from a large vocabulary of odd size, by probability alone
        _sample("sample_wide", "f32", rows=256, vocab=128257, filters="top_p"),
    ]


def draw(rng):
    op = rng.choice(["embed", "embed_train", "scan", "scan_train", "paged8", "decode8", "sample", "sample"])
    if op in ("embed", "embed_train"):
        tokens, vocab, width = _log(rng, 1, 32768), _log(rng, 2, 131072), _log(rng, 8, 4096)
        tokens = min(tokens, max(1, (1 << 25) // width))
        vocab = min(vocab, max(2, (1 << 26) // width))
        return _embed(None, op, rng.choice(["f32", "bf16"]), rng.choice(["bf16", "bf16", "f32"]), tokens, vocab, width,
                      scale=rng.choice([1.0, round(width ** 0.5, 3)]))
    if op in ("scan", "scan_train"):
        dtype, gate = rng.choice([("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32")])
        longest, width = _log(rng, 1, 16384 if op == "scan" else 4096), _log(rng, 8, 4096)
        seqs = _log(rng, 1, max(1, min(128, (1 << 25) // (longest * width))))
        return _scan(None, op, dtype, gate, seqs, longest, width, rng.randrange(1 << 20))
    if op == "sample":
        vocab = _log(rng, 2, 200000)
        rows = _log(rng, 1, max(1, min(256, (1 << 25) // vocab)))
        return _sample(None, rng.choice(["bf16", "f32"]), rows, vocab,
                       rng.choice(["all", "mixed", "none", "top_k", "top_p", "min_p"]))
    heads, kv = rng.choice([(16, 4), (16, 16), (16, 2), (8, 8), (8, 1), (4, 2), (12, 4), (6, 2)])
    dim, page = rng.choice([128, 128, 64, 96, 32]), rng.choice([1, 16, 32, 64, 256])
    window = rng.choice([0, 0, _log(rng, 16, 4096)])
    if op == "decode8":
        context, seqs, new = _log(rng, 1, 16383), _log(rng, 1, 64), rng.choice([1, 1, 1, 2, 5])
    else:
        context, seqs, new = _log(rng, 1, 8191), _log(rng, 1, 8), _log(rng, 6, 300)
    seqs = max(1, min(seqs, (1 << 28) // (context * kv * dim)))
    return _paged8(None, heads, kv, dim, page, seqs, new, context, window, rng.randrange(1 << 20))


def _log(rng, lo, hi):
    """A whole number spread evenly over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def _named(name, c):
    return c if name is None else dict(c, name=name)


def _embed(name, op, weight, dtype, tokens, vocab, width, scale=1.0):
    return _named(name, dict(op=op, weight=weight, dtype=dtype, tokens=tokens, vocab=vocab, width=width, scale=scale))


def _scan(name, op, dtype, gate, seqs, longest, width, lens=7):
    return _named(name, dict(op=op, dtype=dtype, gate=gate, seqs=seqs, longest=longest, width=width, lens=lens))


def _paged8(name, heads, kv, dim, page, seqs, new, context, window, lens=7):
    return _named(name, dict(op="paged8", heads=heads, kv=kv, dim=dim, page=page, seqs=seqs, new=new, context=context,
                             window=window, lens=lens))


def _sample(name, dtype, rows, vocab, filters):
    return _named(name, dict(op="sample", dtype=dtype, rows=rows, vocab=vocab, filters=filters))


def _lengths(case):
    """Sequence lengths: the first one the longest, the others between an
    eighth of it and all of it."""
    r = random.Random(case["lens"])
    top = case["longest"]
    return [top] + [max(1, int(top * r.uniform(0.125, 1.0))) for _ in range(case["seqs"] - 1)]


def _contexts(case):
    """(tokens in the cache, new tokens) of each sequence of a paged case."""
    r = random.Random(case["lens"])
    ctx = [case["context"]] + [int(case["context"] * r.uniform(0.05, 1.0)) for _ in range(case["seqs"] - 1)]
    new = [case["new"]] + [max(1, int(case["new"] * r.uniform(0.5, 1.0))) for _ in range(case["seqs"] - 1)]
    return list(zip(ctx, new))


def work(case):
    op = case["op"]
    if op in ("embed", "embed_train"):
        n, w, es, ws = case["tokens"], case["width"], _BYTES[case["dtype"]], _BYTES[case["weight"]]
        fwd = n * 8 + min(n, case["vocab"]) * w * ws + n * w * es
        if op == "embed":
            return {"bytes": fwd, "flops": n * w}
        return {"bytes": fwd + n * w * es + case["vocab"] * w * ws, "flops": 3 * n * w}
    if op in ("scan", "scan_train"):
        n, w, es, gs = sum(_lengths(case)), case["width"], _BYTES[case["dtype"]], _BYTES[case["gate"]]
        fwd = n * w * (2 * es + gs) + 8 * case["seqs"] * w
        if op == "scan":
            return {"bytes": fwd, "flops": 2 * n * w}
        return {"bytes": fwd + n * w * (2 * es + gs) + 8 * case["seqs"] * w, "flops": 5 * n * w}
    if op == "sample":
        n = case["rows"] * case["vocab"]
        return {"bytes": n * _BYTES[case["dtype"]] + 32 * case["rows"], "flops": 16 * n}
    H, K, D, W = case["heads"], case["kv"], case["dim"], case["window"]
    cs = _contexts(case)
    new = sum(n for _, n in cs)
    seen = min(sum(min(c, n + W - 1 if W else c) for c, n in cs), sum(c for c, _ in cs))  # cached keys some query sees
    pairs = sum(min(p + 1, W) if W else p + 1 for c, n in cs for p in range(c, c + n))
    # queries and outputs, new keys and values in and, in 8 bits with a scale, out; cached ones
    return {"bytes": 4 * D * new * H + 2 * K * new * (2 * D + D + 1) + 2 * K * seen * (D + 1), "flops": 4 * D * H * pairs}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=g, device=dev) * std).to(dtype)

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device=dev)

    s, op = {"case": case}, case["op"]
    if op in ("embed", "embed_train"):
        n, v, w = case["tokens"], case["vocab"], case["width"]
        # words' frequencies fall with their rank: the commonest is one token in twelve
        upto = torch.cumsum((1 << 32) // torch.arange(1, v + 1, device=dev), dim=0)
        words = torch.randperm(v, generator=g, device=dev)
        at = torch.randint(int(upto[-1]), (n,), generator=g, device=dev)
        s["tokens"] = words[torch.searchsorted(upto, at, right=True)]
        s["weight"] = normal(v, w, std=0.02, dtype=_TYPES[case["weight"]])
        if op == "embed_train":
            s["dout"] = normal(n, w, dtype=_TYPES[case["dtype"]])
        return s
    if op in ("scan", "scan_train"):
        lens, w, dt = _lengths(case), case["width"], _TYPES[case["dtype"]]
        n = sum(lens)
        s.update(x=normal(n, w, std=0.5, dtype=dt), a=torch.sigmoid(3 + normal(n, w)).to(_TYPES[case["gate"]]),
                 h0=normal(case["seqs"], w), cu=_offsets(lens, dev), longest=max(lens))
        s["state"] = torch.empty_like(s["h0"])
        if op == "scan_train":
            s.update(dout=normal(n, w, dtype=dt), dstate=normal(case["seqs"], w))
        return s
    if op == "sample":
        n, v = case["rows"], case["vocab"]
        x = normal(n, v, std=2.0)
        peaks = torch.randint(v, (n, 32), generator=g, device=dev)  # the tokens that the context asks for
        s["logits"] = x.scatter_add_(1, peaks, 10 * uniform(n, 32)).to(_TYPES[case["dtype"]])
        s["u"] = uniform(n)
        s.update(_filters(case["filters"], n, uniform))
        return s
    H, K, D, page = case["heads"], case["kv"], case["dim"], case["page"]
    cs = _contexts(case)
    n = sum(b for _, b in cs)
    need = [-(-(a + b) // page) for a, b in cs]
    pool, wide = sum(need) + 3, max(need) + 2
    order = torch.randperm(pool, generator=g, device=dev).to(torch.int32).cpu()
    table = torch.zeros(len(cs), wide, dtype=torch.int32)
    at = 0
    for i, m in enumerate(need):
        table[i, :m] = order[at:at + m]
        at += m
    bf = torch.bfloat16
    s.update(q=normal(n, H, D, dtype=bf), k=normal(n, K, D, dtype=bf), v=normal(n, K, D, dtype=bf),
             table=table.to(dev), longest=max(a + b for a, b in cs), most=max(b for _, b in cs),
             cached=torch.tensor([a for a, _ in cs], dtype=torch.int32, device=dev))
    s["cu"] = _offsets([b for _, b in cs], dev)
    for name in ("k", "v"):
        s[name + "_cache"], e = _quantise(normal(pool, K, page, D, dtype=bf))
        s[name + "_scale"] = e.view(_E8)
    return s


def _offsets(lens, dev):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device=dev)


def _filters(kind, n, uniform):
    """The settings of `n` rows: numbers, or a tensor of one each."""
    if kind == "none":
        return dict(temperature=1.0, top_k=0, top_p=1.0, min_p=0.0)
    if kind == "all":
        return dict(temperature=0.8, top_k=50, top_p=0.95, min_p=0.02)
    if kind == "top_k":
        return dict(temperature=1.0, top_k=40, top_p=1.0, min_p=0.0)
    if kind == "top_p":
        return dict(temperature=1.0, top_k=0, top_p=0.9, min_p=0.0)
    if kind == "min_p":
        return dict(temperature=1.2, top_k=0, top_p=1.0, min_p=0.05)
    some = lambda share, x, off: torch.where(uniform(n) < share, x, torch.full_like(x, off))
    return dict(temperature=some(0.9, 0.3 + uniform(n), 0.0),  # 0: the largest
                top_k=some(0.5, torch.floor(1 + 200 * uniform(n)), 0).to(torch.int32),
                top_p=some(0.7, 0.5 + 0.5 * uniform(n), 1.0), min_p=some(0.3, 0.1 * uniform(n), 0.0))


def _quantise(x):
    """Rows of 8-bit floats and the exponents (plus 127) of their scales: the
    smallest power of two that brings the row's largest magnitude to 448 at most."""
    f, e = torch.frexp(x.float().abs().amax(dim=-1))
    e = torch.where(f > 0, (e - 9 + (f > _F8_MAX / 512).int()).clamp(min=-127), torch.zeros_like(e))
    y = torch.ldexp(x.float(), -e[..., None]).clamp(-_F8_MAX, _F8_MAX)
    return y.to(_F8), (e + 127).to(torch.uint8)


def _dequantise(x, e, dtype=torch.float32):
    return torch.ldexp(x.to(dtype), e[..., None].int() - 127)


# ---------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state, op)
    if op in ("embed", "embed_train"):
        return _plain_embed(state, op)
    if op in ("scan", "scan_train"):
        return _plain_scan(state, op)
    return _plain_sample(state) if op == "sample" else _plain_paged(state)


def _own(s, op):
    import chunk_weight_rnn_amd as e2
    c = s["case"]
    if op in ("embed", "embed_train"):
        out = e2.embedding_forward(s["tokens"], s["weight"], scale=c["scale"], dtype=_TYPES[c["dtype"]])
        if op == "embed":
            return {"out": out}
        dw = e2.embedding_backward(s["dout"], s["tokens"], c["vocab"], scale=c["scale"], dtype=_TYPES[c["weight"]])
        return {"out": out, "dweight": dw}
    if op == "scan":
        out, state, _ = e2.gated_scan_forward(s["x"], s["a"], s["cu"], h0=s["h0"], state=s["state"])
        return {"out": out, "state": state}
    if op == "scan_train":
        out, state, starts = e2.gated_scan_forward(s["x"], s["a"], s["cu"], h0=s["h0"], save=True)
        g = e2.gated_scan_backward(s["dout"], s["x"], s["a"], starts, s["cu"], dstate=s["dstate"])
        return {"out": out, "state": state, "dx": g["x"], "da": g["a"], "dh0": g["h0"]}
    if op == "sample":
        token, logprob = e2.sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"],
                                   top_p=s["top_p"], min_p=s["min_p"])
        return {"token": token, "logprob": logprob}
    out = e2.paged_attention(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["cu"], s["cached"],
                             window=c["window"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    return _with_cache(s, out)


def _with_cache(s, out):
    return {"out": out, "k_cache": s["k_cache"], "v_cache": s["v_cache"],
            "k_scale": s["k_scale"].view(torch.uint8), "v_scale": s["v_scale"].view(torch.uint8)}


def _plain_embed(s, op):
    c = s["case"]
    r = {"out": (s["weight"][s["tokens"]].float() * c["scale"]).to(_TYPES[c["dtype"]])}
    if op == "embed_train":
        d = torch.zeros(c["vocab"], c["width"], device=s["dout"].device)
        d.index_add_(0, s["tokens"], s["dout"].float())
        r["dweight"] = (d * c["scale"]).to(_TYPES[c["weight"]])
    return r


def _doubling(x, a):
    """h_t = a_t h_{t-1} + x_t along dim 1, in place of both, in log2 steps."""
    d = 1
    while d < x.shape[1]:
        x[:, d:] += a[:, d:] * x[:, :-d]
        a[:, d:] = a[:, d:] * a[:, :-d]
        d *= 2
    return x


def _plain_scan(s, op):
    """Padded to [sequence, position, channel]."""
    c, dt, L = s["case"], s["x"].dtype, s["longest"]
    N, dev = s["x"].shape[0], s["x"].device
    cu = s["cu"].long()
    count = cu[1:] - cu[:-1]
    pos = torch.arange(L, device=dev)
    real = (pos < count[:, None])[:, :, None]
    at = (cu[:-1, None] + pos).clamp(max=N - 1)
    seq = torch.searchsorted(cu, torch.arange(N, device=dev), right=True) - 1
    place = torch.arange(N, device=dev) - cu[seq]
    each = torch.arange(c["seqs"], device=dev)

    def pad(t):
        return torch.where(real, t.float()[at], torch.zeros((), device=dev))

    x, a = pad(s["x"]), pad(s["a"])
    x[:, 0] += a[:, 0] * s["h0"]
    h = _doubling(x, a.clone())
    r = {"out": h[seq, place].to(dt), "state": s["state"].copy_(h[each, count - 1])}
    if op == "scan_train":
        r["state"] = r["state"].clone()
        g = pad(s["dout"])
        g[each, count - 1] += s["dstate"]
        after = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], dim=1)
        g = _doubling(g.flip(1), after.flip(1)).flip(1)
        before = torch.cat([s["h0"][:, None], h[:, :-1]], dim=1)
        r["dx"], r["da"] = g[seq, place].to(dt), (g * before)[seq, place].to(s["a"].dtype)
        r["dh0"] = a[:, 0] * g[:, 0]
    return r


def _plain_sample(s):
    """Weights are whole multiples of 2^-44 of the largest, so that their sums
    are exact.  Tokens in order of falling logit, equal ones by index: the first
    top_k of them; of those, as many as are needed for top_p of their weight; of
    those, the ones with at least min_p of the largest weight.  Of what is left,
    by index, the first at which the sum exceeds u of the whole, and the log of
    its share of it."""
    x = s["logits"].double()
    n, v = x.shape
    col = lambda t: torch.as_tensor(t, device=x.device).expand(n)[:, None]
    T, top_k, top_p, min_p, u = (col(s[k]) for k in ("temperature", "top_k", "top_p", "min_p", "u"))
    x, order = torch.sort(x, dim=1, descending=True, stable=True)
    p = torch.exp((x - x[:, :1]) / torch.where(T > 0, T, torch.ones_like(T)).double())
    w = torch.round(p * _ONE).long()
    rank = torch.arange(v, device=x.device)
    w = torch.where((rank >= top_k) & (top_k > 0) | (rank > 0) & (T <= 0), torch.zeros_like(w), w)
    upto = torch.cumsum(w, dim=1)
    before, total = (upto - w).double(), upto[:, -1:].double()
    w = torch.where((top_p < 1) & (before >= top_p.double() * total) & (rank > 0), torch.zeros_like(w), w)
    w = torch.where(p < min_p.double(), torch.zeros_like(w), w)
    w = torch.zeros_like(w).scatter_(1, order, w)
    upto = torch.cumsum(w, dim=1)
    total = upto[:, -1:].double()
    token = (upto.double() > u.double() * total).int().argmax(dim=1)
    share = w.gather(1, token[:, None]).double() / total
    return {"token": token, "logprob": torch.log(share[:, 0]).float()}


def _plain_paged(s):
    c, dt = s["case"], s["q"].dtype
    H, K, D, W, page = c["heads"], c["kv"], c["dim"], c["window"], c["page"]
    G, L, M = H // K, s["longest"], s["most"]
    N, dev = s["q"].shape[0], s["q"].device
    cu, cached, table = s["cu"].long(), s["cached"].long(), s["table"].long()
    S = cu.numel() - 1
    seq = torch.searchsorted(cu, torch.arange(N, device=dev), right=True) - 1
    place = torch.arange(N, device=dev) - cu[seq]
    where = cached[seq] + place
    pos = torch.arange(L, device=dev)
    held = table[:, pos // page]  # [S, L]
    new = torch.arange(M, device=dev)
    mine = cached[:, None] + new  # [S, M]: the queries' positions
    real = new < (cu[1:] - cu[:-1])[:, None]
    sees = real[:, :, None] & (pos <= mine[:, :, None]) & ((pos > mine[:, :, None] - W) if W else True)

    def written(name):
        """The cache with the new tokens in it, read back: [S, K, L, D], zeros where no query looks."""
        x, e = _quantise(s[name])
        at = table[seq, where // page]
        s[name + "_cache"].view(torch.uint8)[at, :, where % page] = x.view(torch.uint8)
        s[name + "_scale"].view(torch.uint8)[at, :, where % page] = e
        x = s[name + "_cache"].view(torch.uint8)[held, :, pos % page].view(_F8)
        y = _dequantise(x, s[name + "_scale"].view(torch.uint8)[held, :, pos % page])
        y = torch.where(sees.any(dim=1)[:, :, None, None], y, torch.zeros((), device=dev))
        return y.permute(0, 2, 1, 3).contiguous()

    k, v = written("k"), written("v")
    at = (cu[:-1, None] + new).clamp(max=N - 1)
    q = s["q"].float()[at].reshape(S, M, K, G, D).permute(0, 2, 3, 1, 4).reshape(S, K, G * M, D)
    p = torch.matmul(q, k.transpose(2, 3)).mul_(D ** -0.5).reshape(S, K, G, M, L)
    p.masked_fill_(~sees[:, None, None], float("-inf"))
    top = p.amax(dim=-1, keepdim=True)
    p.sub_(torch.where(torch.isfinite(top), top, torch.zeros_like(top))).exp_()
    total = p.sum(dim=-1, keepdim=True)
    p.div_(torch.where(total > 0, total, torch.ones_like(total)))
    out = torch.matmul(p.reshape(S, K, G * M, L), v)
    out = out.reshape(S, K, G, M, D).permute(0, 3, 1, 2, 4)[seq, place].reshape(N, H, D).to(dt)
    return _with_cache(s, out)


# ------------------------------------------------- the definition, 64 bits
def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    f8 = torch.float64
    if op in ("embed", "embed_train"):
        w = s["weight"].to(f8).requires_grad_(op == "embed_train")
        out = torch.index_select(w, 0, s["tokens"]) * case["scale"]
        if op == "embed":
            return {"out": out}
        (dw,) = torch.autograd.grad(out, w, s["dout"].to(f8))
        return {"out": out.detach(), "dweight": dw}
    if op in ("scan", "scan_train"):
        return _exact_scan(case, s)
    if op == "sample":
        return _exact_sample(s)
    H, K, D, page = case["heads"], case["kv"], case["dim"], case["page"]
    G, cu = H // K, s["cu"].tolist()
    out = torch.zeros(cu[-1], H, D, dtype=f8, device="cuda")

    def rounded(x):
        """A row of keys or values as the cache holds it."""
        x = x.to(f8)
        step = torch.full_like(x[:, :1], 2.0 ** -127)
        top = x.abs().amax(dim=1, keepdim=True)
        for e in range(-126, 128):  # the scale grows until the largest fits
            step = torch.where(top > _F8_MAX * step, torch.full_like(step, 2.0 ** e), step)
        return (x / step).float().to(_F8).to(f8) * step

    for i, (a, b) in enumerate(zip(cu, cu[1:])):
        kept = int(s["cached"][i])
        slot = torch.arange(kept, device="cuda")
        held = s["table"][i].long()[slot // page]
        at = torch.arange(kept, kept + b - a, device="cuda")[:, None]
        key = torch.arange(kept + b - a, device="cuda")[None, :]
        hidden = key > at
        if case["window"]:
            hidden = hidden | (key <= at - case["window"])
        for j in range(K):
            kv = []
            for name in ("k", "v"):
                e = s[name + "_scale"].view(torch.uint8)[held, j, slot % page].to(f8) - 127
                old = s[name + "_cache"].view(torch.uint8)[held, j, slot % page].view(_F8).to(f8) * torch.exp2(e)[:, None]
                kv.append(torch.cat([old, rounded(s[name][a:b, j])]))
            for h in range(j * G, (j + 1) * G):
                scores = (s["q"][a:b, h].to(f8) @ kv[0].T / D ** 0.5).masked_fill(hidden, float("-inf"))
                out[a:b, h] = torch.softmax(scores, 1) @ kv[1]
    return {"out": out, "k_cache": None, "v_cache": None, "k_scale": None, "v_scale": None}


def _exact_scan(case, s):
    f8 = torch.float64
    train = case["op"] == "scan_train"
    cu = s["cu"].tolist()
    x, a, h0 = (s[n].to(f8) for n in ("x", "a", "h0"))
    out, state = torch.empty_like(x), torch.empty_like(h0)
    before = torch.empty_like(x) if train else None
    # sequences side by side, as long as they last
    order = sorted(range(case["seqs"]), key=lambda i: cu[i] - cu[i + 1])
    lens = [cu[i + 1] - cu[i] for i in order]
    first, h = torch.tensor([cu[i] for i in order], device="cuda"), h0[order]
    for t in range(lens[0]):
        live = sum(n > t for n in lens)
        rows = first[:live] + t
        if train:
            before[rows] = h[:live]
        h[:live] = a[rows] * h[:live] + x[rows]
        out[rows] = h[:live]
    state[order] = h
    if not train:
        return {"out": out, "state": state}
    g, da, dout = s["dstate"].to(f8)[order], torch.empty_like(a), s["dout"].to(f8)
    dx, dh0 = torch.empty_like(x), torch.empty_like(h0)
    for t in reversed(range(lens[0])):
        live = sum(n > t for n in lens)
        rows = first[:live] + t
        dx[rows] = g[:live] + dout[rows]  # what reaches the state after token t
        da[rows] = dx[rows] * before[rows]
        g[:live] = dx[rows] * a[rows]
    dh0[order] = g
    return {"out": out, "state": state, "dx": dx, "da": da, "dh0": dh0}


def _exact_sample(s):
    x = s["logits"].double().cpu().numpy()
    n = x.shape[0]
    num = lambda k: np.broadcast_to(s[k].double().cpu().numpy() if torch.is_tensor(s[k]) else np.float64(np.float32(s[k])), n)
    T, top_k, top_p, min_p, u = (num(k) for k in ("temperature", "top_k", "top_p", "min_p", "u"))
    token, logprob = np.empty(n, dtype=np.int64), np.zeros(n)
    for i in range(n):
        if T[i] <= 0:
            token[i] = int(np.argmax(x[i]))
            continue
        p = np.exp((x[i] - x[i].max()) / T[i])
        w = np.rint(p * _ONE).astype(np.longdouble)
        order = np.lexsort((np.arange(x.shape[1]), -x[i]))
        if top_k[i] > 0:
            order = order[:int(top_k[i])]
        if top_p[i] < 1:
            upto = np.cumsum(w[order])
            order = order[:1 + int(np.searchsorted(upto, np.longdouble(top_p[i]) * upto[-1], side="left"))]
        order = np.sort(order[p[order] >= min_p[i]])
        upto = np.cumsum(w[order])
        token[i] = order[int(np.searchsorted(upto, np.longdouble(u[i]) * upto[-1], side="right"))]
        logprob[i] = np.log(w[token[i]] / upto[-1])
    return {"token": torch.from_numpy(token).cuda(), "logprob": torch.from_numpy(logprob).cuda()}
