"""What is measured of the operators of a hybrid layer beside the chunk update.

A hybrid layer joins the fast-weight branch (``chunk_forward``) with sliding
window attention.  Its operators here are

* ``prompt`` / ``train``: causal attention over packed sequences with grouped
  heads and an optional window, forward alone or forward and backward;
* ``paged``: attention of each sequence's new tokens over a paged key/value
  cache that the call first extends by them (single tokens and chunks);
* ``norm`` / ``norm_train``: root-mean-square norm with the residual's
  addition, in the stream's type or in 8 bits with a scale per row, forward
  alone or forward and backward.

``run`` computes them in elementary torch operations in 32 bits, or, where
``own`` is true, through the package's entry points.  ``exact`` is the
definition in 64 bits.
"""
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_F8 = torch.float8_e4m3fn
_F8_MAX = 448.0
_EPS = 1e-6


# ------------------------------------------------------------------- cases
def listed():
    return [
        # the shortest prompt that a user sends: one sentence, latency counts
        _attn("prompt_short", "prompt", "bf16", 16, 4, 128, seqs=1, longest=77, window=0),
        # a prefill batch of the 1.3B-shaped layer: packed prompts of uneven length, full causal
        _attn("prompt_packed_2k", "prompt", "bf16", 16, 4, 128, seqs=16, longest=2048, window=0),
        # the 16K extrapolation sequence through a sliding window, a key head per query head
        _attn("prompt_16k_window", "prompt", "bf16", 16, 16, 128, seqs=1, longest=16384, window=2048),
        # a training step's attention: packed documents at the 2K training context
        _attn("train_packed_2k", "train", "bf16", 16, 4, 128, seqs=12, longest=2048, window=0),
        # the fp32 layer of four heads of 64, two rows of 2K, two query heads to a key head
        _attn("train_f32", "train", "f32", 4, 2, 64, seqs=2, longest=2048, window=0),
        # one user's next token at a short context: latency counts
        _paged("decode_one", "bf16", 16, 4, 128, page=16, seqs=1, new=1, context=513, window=0),
        # the next tokens of a full serving batch, contexts of every length up to 16K
        _paged("decode_batch", "bf16", 16, 4, 128, page=64, seqs=64, new=1, context=16383, window=0),
        # eight streams, a 256-token chunk each (the chunk update's call beside it), window of 2K
        _paged("chunk_batch", "bf16", 16, 4, 128, page=64, seqs=8, new=256, context=8191, window=2048),
        # one row of the 16K sequence streamed a 256-token chunk per call, near its end, full causal
        _paged("chunk_16k", "bf16", 16, 4, 128, page=64, seqs=1, new=256, context=16128, window=0),
        # the norm before a decode step's projections in 8 bits: eight rows
        _norm("norm_decode_8bit", "norm", "bf16", rows=8, width=2048, bits8=True, residual=True),
        # the same for a prefill batch of 8 x 2K tokens
        _norm("norm_prompt_8bit", "norm", "bf16", rows=16384, width=2048, bits8=True, residual=True),
        # a training step's norm of 8 x 2K tokens, with its gradients
        _norm("norm_train", "norm_train", "bf16", rows=16384, width=2048, bits8=False, residual=True),
    ]


def draw(rng):
    op = rng.choice(["prompt", "train", "paged", "decode", "norm", "norm_train"])
    if op in ("norm", "norm_train"):
        rows, width = _log(rng, 1, 16384), _log(rng, 64, 8192)
        rows = min(rows, max(1, (1 << 25) // width))
        return _norm(None, op, rng.choice(["bf16", "bf16", "f32"]), rows, width,
                     bits8=op == "norm" and rng.random() < 0.6, residual=rng.random() < 0.75)
    heads, kv = rng.choice([(16, 4), (16, 16), (16, 2), (8, 8), (8, 1), (4, 2), (12, 4), (6, 2)])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    dim = rng.choice([128, 128, 64, 96, 32]) if dtype == "bf16" else rng.choice([64, 32, 128])
    window = rng.choice([0, 0, _log(rng, 16, 4096)])
    lens = rng.randrange(1 << 20)
    if op in ("prompt", "train"):
        longest = _log(rng, 1, 8192 if op == "prompt" and dtype == "bf16" else 2048)
        most = max(1, (16 << 20 if dtype == "bf16" else 4 << 20) // (longest * longest))
        return _attn(None, op, dtype, heads, kv, dim, _log(rng, 1, min(most, 32)), longest, window, lens)
    page = rng.choice([1, 16, 32, 64, 256])
    if op == "decode":
        context, seqs, new = _log(rng, 1, 16383), _log(rng, 1, 64), rng.choice([1, 1, 1, 2, 5])
    else:
        context, seqs, new = _log(rng, 1, 8191), _log(rng, 1, 8), _log(rng, 6, 300)
    room = (1 << 28) if dtype == "bf16" else (1 << 25)  # cached values, keys alone
    seqs = max(1, min(seqs, room // (context * kv * dim)))
    return _paged(None, dtype, heads, kv, dim, page, seqs, new, context, window, lens)


def _log(rng, lo, hi):
    """A whole number spread evenly over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def _attn(name, op, dtype, heads, kv, dim, seqs, longest, window, lens=7):
    c = dict(op=op, dtype=dtype, heads=heads, kv=kv, dim=dim, seqs=seqs, longest=longest, window=window, lens=lens)
    return c if name is None else dict(c, name=name)


def _paged(name, dtype, heads, kv, dim, page, seqs, new, context, window, lens=7):
    c = dict(op="paged", dtype=dtype, heads=heads, kv=kv, dim=dim, page=page, seqs=seqs, new=new, context=context,
             window=window, lens=lens)
    return c if name is None else dict(c, name=name)


def _norm(name, op, dtype, rows, width, bits8, residual):
    c = dict(op=op, dtype=dtype, rows=rows, width=width, bits8=bits8, residual=residual)
    return c if name is None else dict(c, name=name)


def _lengths(case):
    """Sequence lengths of an attention case: the first one the longest, the
    others between an eighth of it and all of it."""
    r = random.Random(case["lens"])
    top = case["longest"]
    return [top] + [max(1, int(top * r.uniform(0.125, 1.0))) for _ in range(case["seqs"] - 1)]


def _contexts(case):
    """(tokens in the cache, new tokens) of each sequence of a paged case."""
    r = random.Random(case["lens"])
    ctx = [case["context"]] + [int(case["context"] * r.uniform(0.05, 1.0)) for _ in range(case["seqs"] - 1)]
    new = [case["new"]] + [max(1, int(case["new"] * r.uniform(0.5, 1.0))) for _ in range(case["seqs"] - 1)]
    return list(zip(ctx, new))


def _pairs(first, count, window):
    """Query-key pairs of `count` queries at positions first, first + 1, ..."""
    return sum(min(p + 1, window) if window else p + 1 for p in range(first, first + count))


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("norm", "norm_train"):
        n, w = case["rows"] * case["width"], case["width"]
        res = 2 * n * es if case["residual"] else 0  # residual read, stream written
        fwd = n * es + res + w * 4 + n * (1 if case["bits8"] else es) + case["rows"] * 4
        if case["op"] == "norm":
            return {"bytes": fwd, "flops": 5 * n}
        return {"bytes": fwd + n * es * 4 + w * 8, "flops": 14 * n}  # dy, stream, its gradient; dx and dweight
    H, K, D = case["heads"], case["kv"], case["dim"]
    if case["op"] == "paged":
        cs = _contexts(case)
        new = sum(n for _, n in cs)
        seen = sum(min(c, n + case["window"] - 1 if case["window"] else c) for c, n in cs)  # cached keys some query sees
        seen = min(seen, sum(c for c, _ in cs))
        pairs = sum(_pairs(c, n, case["window"]) for c, n in cs)
        return {"bytes": es * D * (2 * new * H + 4 * new * K + 2 * seen * K), "flops": 4 * D * H * pairs}
    n = sum(_lengths(case))
    pairs = sum(_pairs(0, s, case["window"]) for s in _lengths(case))
    fwd = es * n * D * (2 * H + 2 * K) + 4 * n * H
    if case["op"] == "prompt":
        return {"bytes": fwd, "flops": 4 * D * H * pairs}
    return {"bytes": fwd + es * n * D * (2 * H + 2 * K), "flops": 14 * D * H * pairs}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = _TYPES[case["dtype"]]

    def normal(*shape, std=1.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device=dev) * std).to(dtype)

    s = {"case": case}
    if case["op"] in ("norm", "norm_train"):
        n, w = case["rows"], case["width"]
        s["x"] = normal(n, w)
        s["weight"] = 1.0 + normal(w, std=0.1, dtype=torch.float32)
        s["residual"] = normal(n, w, std=2.0) if case["residual"] else None
        if case["op"] == "norm_train":
            s["dy"] = normal(n, w)
            s["dh"] = normal(n, w) if case["residual"] else None  # what arrives along the residual stream
        return s
    H, K, D = case["heads"], case["kv"], case["dim"]
    if case["op"] == "paged":
        cs = _contexts(case)
        n, page = sum(b for _, b in cs), case["page"]
        need = [-(-(a + b) // page) for a, b in cs]
        pool, wide = sum(need) + 3, max(need) + 2
        order = torch.randperm(pool, generator=g, device=dev).to(torch.int32).cpu()
        table = torch.zeros(len(cs), wide, dtype=torch.int32)
        at = 0
        for i, m in enumerate(need):
            table[i, :m] = order[at:at + m]
            at += m
        s.update(q=normal(n, H, D), k=normal(n, K, D), v=normal(n, K, D), k_cache=normal(pool, K, page, D),
                 v_cache=normal(pool, K, page, D), table=table.to(dev), longest=max(a + b for a, b in cs),
                 most=max(b for _, b in cs), cached=torch.tensor([a for a, _ in cs], dtype=torch.int32, device=dev))
        s["cu"] = _offsets([b for _, b in cs], dev)
        return s
    lens = _lengths(case)
    n = sum(lens)
    # one projection's output holds a token's queries, keys and values side by side
    qkv = normal(n, H + 2 * K, D)
    s.update(q=qkv[:, :H], k=qkv[:, H:H + K], v=qkv[:, H + K:], cu=_offsets(lens, dev), longest=max(lens))
    if case["op"] == "train":
        s["dout"] = normal(n, H, D)
    return s


def _offsets(lens, dev):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device=dev)


# ---------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state, op)
    if op in ("norm", "norm_train"):
        return _plain_norm(state, op)
    return _plain_paged(state) if op == "paged" else _plain_attention(state, op)


def _own(s, op):
    import chunk_weight_rnn_amd as e2
    c = s["case"]
    if op == "prompt":
        out, lse = e2.attention_forward(s["q"], s["k"], s["v"], s["cu"], window=c["window"])
        return {"out": out, "lse": lse}
    if op == "train":
        out, lse = e2.attention_forward(s["q"], s["k"], s["v"], s["cu"], window=c["window"])
        g = e2.attention_backward(s["q"], s["k"], s["v"], out, lse, s["dout"], s["cu"], window=c["window"])
        return {"out": out, "lse": lse, "dq": g["q"], "dk": g["k"], "dv": g["v"]}
    if op == "paged":
        out = e2.paged_attention(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["cu"], s["cached"],
                                 window=c["window"])
        return {"out": out, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    y, scale, h, rstd = e2.norm_forward(s["x"], s["weight"], residual=s["residual"], eps=_EPS, bits8=c["bits8"])
    if op == "norm":
        r = {"y": y, "scale": scale} if c["bits8"] else {"y": y}
        return dict(r, h=h) if c["residual"] else r
    dx, dweight = e2.norm_backward(s["dy"], h, s["weight"], rstd, dh=s["dh"])
    r = {"y": y, "dx": dx, "dweight": dweight}
    return dict(r, h=h) if c["residual"] else r


def _plain_norm(s, op):
    c, dt = s["case"], s["x"].dtype
    h = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(dt)
    x, w = h.float(), s["weight"]
    rstd = torch.rsqrt((x * x).mean(dim=1, keepdim=True) + _EPS)
    xhat = x * rstd
    y = xhat * w
    if c["bits8"]:
        top = y.abs().amax(dim=1, keepdim=True)
        scale = torch.where(top > 0, top / _F8_MAX, torch.ones_like(top))
        r = {"y": (y / scale).clamp(-_F8_MAX, _F8_MAX).to(_F8), "scale": scale[:, 0]}
    else:
        r = {"y": y.to(dt)}
    if c["residual"]:
        r["h"] = h
    if op == "norm_train":
        dy = s["dy"].float()
        dxhat = dy * w
        dx = rstd * (dxhat - xhat * (dxhat * xhat).mean(dim=1, keepdim=True))
        if s["dh"] is not None:
            dx = dx + s["dh"].float()
        r["dx"], r["dweight"] = dx.to(dt), (dy * xhat).sum(dim=0)
    return r


def _plain_attention(s, op):
    """Padded to [sequence, key head, query head of the group x position]."""
    c, dt = s["case"], s["q"].dtype
    H, K, D, W, L = c["heads"], c["kv"], c["dim"], c["window"], s["longest"]
    G, scale = H // K, D ** -0.5
    N, dev = s["q"].shape[0], s["q"].device
    cu = s["cu"].long()
    S, count = cu.numel() - 1, cu[1:] - cu[:-1]
    pos = torch.arange(L, device=dev)
    at = (cu[:-1, None] + pos).clamp(max=N - 1)
    seq = torch.searchsorted(cu, torch.arange(N, device=dev), right=True) - 1
    place = torch.arange(N, device=dev) - cu[seq]

    def rows(x):  # [N, H, D] -> [S, K, G L, D]
        return x.float()[at].reshape(S, L, K, G, D).permute(0, 2, 3, 1, 4).reshape(S, K, G * L, D)

    def cols(x):  # [N, K, D] -> [S, K, L, D]
        return x.float()[at].permute(0, 2, 1, 3).contiguous()

    def back_rows(x):
        return x.reshape(S, K, G, L, D).permute(0, 3, 1, 2, 4)[seq, place].reshape(N, H, D).to(dt)

    def back_cols(x):
        return x.permute(0, 2, 1, 3)[seq, place].to(dt)

    q, k, v = rows(s["q"]), cols(s["k"]), cols(s["v"])
    sees = (pos[None, :] <= pos[:, None]) & ((pos[None, :] > pos[:, None] - W) if W else True)
    sees = sees[None] & (pos < count[:, None])[:, None, :] & (pos < count[:, None])[:, :, None]  # [S, L, L]
    p = torch.matmul(q, k.transpose(2, 3)).mul_(scale).reshape(S, K, G, L, L)
    p.masked_fill_(~sees[:, None, None], float("-inf"))
    top = p.amax(dim=-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
    p.sub_(top).exp_()
    total = p.sum(dim=-1, keepdim=True)
    lse = (top + total.log()).reshape(S, K, G, L).permute(0, 3, 1, 2)[seq, place].reshape(N, H)
    p.div_(torch.where(total > 0, total, torch.ones_like(total)))
    p = p.reshape(S, K, G * L, L)
    out = torch.matmul(p, v)
    r = {"out": back_rows(out), "lse": lse}
    if op == "train":
        do = rows(s["dout"]) * (pos < count[:, None])[:, None, None, :, None].expand(S, 1, G, L, 1).reshape(S, 1, G * L, 1)
        r["dv"] = back_cols(torch.matmul(p.transpose(2, 3), do))
        ds = torch.matmul(do, v.transpose(2, 3)).sub_((do * out).sum(dim=-1, keepdim=True)).mul_(p).mul_(scale)
        r["dq"] = back_rows(torch.matmul(ds, k))
        r["dk"] = back_cols(torch.matmul(ds.transpose(2, 3), q))
    return r


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
    s["k_cache"][table[seq, where // page], :, where % page] = s["k"]
    s["v_cache"][table[seq, where // page], :, where % page] = s["v"]
    pos = torch.arange(L, device=dev)
    held = table[:, pos // page]  # [S, L]
    k = s["k_cache"][held, :, pos % page].float().permute(0, 2, 1, 3).contiguous()  # [S, K, L, D]
    v = s["v_cache"][held, :, pos % page].float().permute(0, 2, 1, 3).contiguous()
    new = torch.arange(M, device=dev)
    at = (cu[:-1, None] + new).clamp(max=N - 1)
    q = s["q"].float()[at].reshape(S, M, K, G, D).permute(0, 2, 3, 1, 4).reshape(S, K, G * M, D)
    mine = cached[:, None] + new  # [S, M]: the queries' positions
    real = new < (cu[1:] - cu[:-1])[:, None]
    sees = real[:, :, None] & (pos <= mine[:, :, None]) & ((pos > mine[:, :, None] - W) if W else True)
    p = torch.matmul(q, k.transpose(2, 3)).mul_(D ** -0.5).reshape(S, K, G, M, L)
    p.masked_fill_(~sees[:, None, None], float("-inf"))
    top = p.amax(dim=-1, keepdim=True)
    p.sub_(torch.where(torch.isfinite(top), top, torch.zeros_like(top))).exp_()
    total = p.sum(dim=-1, keepdim=True)
    p.div_(torch.where(total > 0, total, torch.ones_like(total)))
    # what no query sees may be anything that was left in the cache
    v = torch.where(sees.any(dim=1)[:, None, :, None], v, torch.zeros_like(v))
    out = torch.matmul(p.reshape(S, K, G * M, L), v)
    out = out.reshape(S, K, G, M, D).permute(0, 3, 1, 2, 4)[seq, place].reshape(N, H, D).to(dt)
    return {"out": out, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


# ------------------------------------------------- the definition, 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    f8 = torch.float64
    if case["op"] in ("norm", "norm_train"):
        h = s["x"]
        if s["residual"] is not None:  # the residual stream is held in its own type
            h = (s["x"].to(f8) + s["residual"].to(f8)).to(h.dtype)
        x = h.to(f8).requires_grad_(True)
        w = s["weight"].to(f8).requires_grad_(True)
        y = w * x / torch.sqrt(x.pow(2).sum(1, keepdim=True) / case["width"] + _EPS)
        r = {"y": y.detach()}
        if case["bits8"]:
            scale = y.detach().abs().amax(1) / _F8_MAX
            scale[scale == 0] = 1
            r = {"y": (y.detach() / scale[:, None]).float().to(_F8).to(f8), "scale": scale}
        if case["residual"]:
            r["h"] = h.to(f8)
        if case["op"] == "norm_train":
            gx, gw = torch.autograd.grad(y, (x, w), s["dy"].to(f8))
            r["dx"], r["dweight"] = gx if s["dh"] is None else gx + s["dh"].to(f8), gw
        return r
    H, K, D = case["heads"], case["kv"], case["dim"]
    G, cu = H // K, s["cu"].tolist()
    out = torch.zeros(cu[-1], H, D, dtype=f8, device="cuda")
    lse = torch.zeros(cu[-1], H, dtype=f8, device="cuda")
    d = {n: torch.zeros(cu[-1], h, D, dtype=f8, device="cuda") for n, h in (("dq", H), ("dk", K), ("dv", K))}
    for i, (a, b) in enumerate(zip(cu, cu[1:])):
        kept = int(s["cached"][i]) if case["op"] == "paged" else 0
        if case["op"] == "paged":
            slot = torch.arange(kept, device="cuda")
            held = s["table"][i].long()[slot // case["page"]]
        at = torch.arange(kept, kept + b - a, device="cuda")[:, None]
        key = torch.arange(kept + b - a, device="cuda")[None, :]
        hidden = key > at
        if case["window"]:
            hidden = hidden | (key <= at - case["window"])
        for h in range(H):
            q, k, v = s["q"][a:b, h].to(f8), s["k"][a:b, h // G].to(f8), s["v"][a:b, h // G].to(f8)
            if case["op"] == "paged":
                k = torch.cat([s["k_cache"][held, h // G, slot % case["page"]].to(f8), k])
                v = torch.cat([s["v_cache"][held, h // G, slot % case["page"]].to(f8), v])
            if case["op"] == "train":
                q, k, v = (t.requires_grad_(True) for t in (q, k, v))
            scores = (q @ k.T / D ** 0.5).masked_fill(hidden, float("-inf"))
            lse[a:b, h] = torch.logsumexp(scores, 1).detach()
            o = torch.softmax(scores, 1) @ v
            out[a:b, h] = o.detach()
            if case["op"] == "train":
                gq, gk, gv = torch.autograd.grad(o, (q, k, v), s["dout"][a:b, h].to(f8))
                d["dq"][a:b, h] = gq
                d["dk"][a:b, h // G] += gk
                d["dv"][a:b, h // G] += gv
    if case["op"] == "paged":
        return {"out": out, "k_cache": None, "v_cache": None}
    return dict(out=out, lse=lse, **d) if case["op"] == "train" else {"out": out, "lse": lse}
