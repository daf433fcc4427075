"""A small hybrid language model, trained and then served.

Each layer has one norm before two branches side by side, sliding window
attention and the E2-TTT chunk update, whose outputs are added to the residual
stream ("Rethinking Expressivity and Efficiency in Test-Time Training").
``recur`` adds a third one, that many channels of a gated linear recurrence.

Training runs whole sequences: ``embedding``, ``rms_norm``, ``attention``,
``chunk_update`` and ``gated_scan`` under autograd.  Serving keeps, per layer, a paged cache of keys and values,
the fast weights and momentum at the start of the open chunk, and that chunk's
tokens, and the recurrence's state: ``paged_attention`` extends the cache and attends, and ``chunk_forward``
gives the outputs of new tokens from the chunk-start weights and, when the
chunk is full, its end state.  A call takes one token per stream or up to the
end of the chunk.  ``bits8`` serves the branch projections in 8-bit floats,
from ``norm_forward``'s e4m3 rows and their scales; ``cache8`` keeps the keys and
values in 8 bits.  ``generate`` continues prompts with tokens drawn by ``sample``.

    python examples/hybrid_layer.py            # train on a random chain, then check and time serving
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch
import torch.nn.functional as F
from torch import nn

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import chunk_weight_rnn_amd as e2  # noqa: E402

D = 128      # head dimension of both branches (the chunk update's MFMA path)
HIDDEN = 64  # hidden units of the SwiGLU fast weight
CHUNK = 256
PAGE = 64
F8 = torch.float8_e4m3fn


class Layer(nn.Module):
    def __init__(self, width, heads, kv_heads, ttt_heads, window, recur=0):
        super().__init__()
        self.heads, self.kv, self.ttt, self.window, self.recur = heads, kv_heads, ttt_heads, window, recur
        # the gates' columns filled up to whole 16 bytes, so that q, k and v stay
        # views of the projection's output (the attention takes such strides)
        self.sizes = [heads * D, 2 * kv_heads * D, 3 * ttt_heads * D, -(-3 * ttt_heads // 8) * 8, recur, recur]
        std = width ** -0.5
        self.norm = nn.Parameter(torch.ones(width))
        self.q_norm, self.k_norm = nn.Parameter(torch.ones(D)), nn.Parameter(torch.ones(D))
        self.inp = nn.Parameter(std * torch.randn(sum(self.sizes), width))
        joined = (heads + ttt_heads) * D + recur
        self.out = nn.Parameter(0.5 * joined ** -0.5 * torch.randn(width, joined))
        self.W0 = nn.Parameter(0.5 * D ** -0.5 * torch.randn(1, ttt_heads, 3 * D * HIDDEN))

    def split(self, z):
        """A projection's rows [N, sum(sizes)] as attention q, k, v, the
        chunk update's tokens and gates, and the recurrence's inputs and gates."""
        n = z.shape[0]
        q, kv, t, gates, rx, ra = z.split(self.sizes, dim=1)
        k, v = kv.view(n, 2, self.kv, D).unbind(1)
        tq, tk, tv = t.view(n, 3, self.ttt, D).unbind(1)
        tq, tk = (e2.rms_norm(x.contiguous(), w)[0] * D ** -0.5 for x, w in ((tq, self.q_norm), (tk, self.k_norm)))
        a, b, c = gates[:, :3 * self.ttt].float().view(n, 3, self.ttt).unbind(1)
        ra = 0.999 * torch.sigmoid(3 + ra.float())  # a state lasts some 20 tokens to begin with
        recur = ((1 - ra * ra).sqrt() * rx).to(z.dtype), ra
        return ((q.view(n, self.heads, D), k, v), (tq, tk, tv),
                (0.1 * F.softplus(a), torch.sigmoid(4 + b), torch.sigmoid(2 + c)), recur)

    def join(self, attn, ttt, recur=None):
        branches = [attn.flatten(1), ttt.flatten(1)] + ([] if recur is None else [recur])
        return torch.cat(branches, dim=1) @ self.out.to(attn.dtype).t()

    def forward(self, x, h, cu, rows):
        """x: the last branch output, h: the residual stream (None: x starts it);
        rows sequences of equal length, [rows * T, width]."""
        y, h = e2.rms_norm(x, self.norm, h)
        (q, k, v), tok, gates, recur = self.split(y @ self.inp.to(y.dtype).t())
        attn = e2.attention(q, k, v, cu, window=self.window)
        heads_first = [t.view(rows, -1, self.ttt, *t.shape[2:]).transpose(1, 2).contiguous() for t in (*tok, *gates)]
        W0 = self.W0.expand(rows, -1, -1).contiguous()
        ttt, _, _ = e2.chunk_update(*heads_first, W0, torch.zeros_like(W0), chunk=CHUNK, Hd=HIDDEN)
        states = e2.gated_scan(*recur, cu)[0] if self.recur else None
        return self.join(attn, ttt.transpose(1, 2).reshape(-1, self.ttt, D), states), h


class Model(nn.Module):
    def __init__(self, vocab=256, width=512, layers=2, heads=4, kv_heads=2, ttt_heads=2, window=192, recur=0):
        super().__init__()
        self.embed = nn.Embedding(vocab, width)
        self.layers = nn.ModuleList(Layer(width, heads, kv_heads, ttt_heads, window, recur) for _ in range(layers))
        self.norm = nn.Parameter(torch.ones(width))
        self.head = nn.Parameter(0.1 * width ** -0.5 * torch.randn(vocab, width))

    def embedded(self, tokens):
        return e2.embedding(tokens.reshape(-1).contiguous(), self.embed.weight, dtype=torch.bfloat16)

    def logits(self, x, h):
        y, _ = e2.rms_norm(x, self.norm, h)
        return y @ self.head.to(y.dtype).t()

    def forward(self, tokens):
        """tokens: [rows, T] -> logits [rows, T, vocab]."""
        rows, T = tokens.shape
        cu = torch.arange(rows + 1, dtype=torch.int32, device=tokens.device) * T
        x, h = self.embedded(tokens), None
        for layer in self.layers:
            x, h = layer(x, h, cu, rows)
        return self.logits(x, h).view(rows, T, -1)


class Served:
    """One layer's serving state for `rows` streams of up to `limit` tokens."""

    def __init__(self, layer, rows, limit, bits8, cache8):
        dev = layer.inp.device
        self.layer, self.rows, self.bits8 = layer, rows, bits8
        per = -(-limit // PAGE)
        self.k_cache, self.v_cache = (torch.empty(rows * per, layer.kv, PAGE, D, dtype=F8 if cache8 else torch.bfloat16,
                                                  device=dev) for _ in range(2))
        self.scales = {n: torch.empty(rows * per, layer.kv, PAGE, dtype=torch.float8_e8m0fnu, device=dev)
                       for n in ("k_scale", "v_scale")} if cache8 else {}
        # pages are handed out in any order; here shuffled, as a busy pool's are
        self.table = torch.randperm(rows * per, device=dev).to(torch.int32).view(rows, per)
        self.W = layer.W0.detach().expand(rows, -1, -1).contiguous()
        self.M = torch.zeros_like(self.W)
        self.state = torch.zeros(rows, layer.recur, device=dev)
        self.open = [torch.zeros(rows, layer.ttt, CHUNK, D, dtype=torch.bfloat16, device=dev) for _ in range(3)]
        self.open += [torch.zeros(rows, layer.ttt, CHUNK, device=dev) for _ in range(3)]
        self.w_in = layer.inp.detach().bfloat16()
        if bits8:  # the projection's weight in 8 bits, a scale per output
            w = layer.inp.detach().float()
            self.w_scale = w.abs().amax(dim=1).clamp(min=1e-12) / 448
            self.w8 = (w / self.w_scale[:, None]).to(F8).bfloat16()

    def project(self, x, h):
        if not self.bits8:
            y, _, h, _ = e2.norm_forward(x, self.layer.norm, residual=h)
            return y @ self.w_in.t(), h
        # e4m3 values are exact in bf16: the product of the 8-bit operands, scaled after it
        y8, scale, h, _ = e2.norm_forward(x, self.layer.norm, residual=h, bits8=True)
        z = y8.bfloat16() @ self.w8.t()
        return (z.float() * scale[:, None] * self.w_scale).bfloat16(), h

    def step(self, x, h, cu, cached, at, n):
        """n new tokens per stream, packed, at places at .. at + n of the open chunk."""
        layer, rows = self.layer, self.rows
        z, h = self.project(x, h)
        (q, k, v), tok, gates, recur = layer.split(z)
        attn = e2.paged_attention(q, k, v, self.k_cache, self.v_cache, self.table, cu, cached, window=layer.window,
                                  **self.scales)
        states = e2.gated_scan_forward(*recur, cu, h0=self.state, state=self.state)[0] if layer.recur else None
        new = [t.view(rows, n, layer.ttt, *t.shape[2:]).transpose(1, 2) for t in (*tok, *gates)]
        for held, t in zip(self.open, new):
            held[:, :, at:at + n] = t
        kw = dict(chunk=CHUNK, kind="swiglu", loss="negdot", Hd=HIDDEN)
        if at + n == CHUNK:  # the whole chunk: its outputs and its end state
            out, self.W, self.M = e2.chunk_forward(*self.open, self.W, self.M, **kw)
            out = out[:, :, at:]
        else:  # outputs come from the chunk-start weights; the state waits for the chunk's end
            out, _, _ = e2.chunk_forward(*(t.contiguous() for t in new), self.W, self.M, **kw)
        return layer.join(attn, out.transpose(1, 2).reshape(-1, layer.ttt, D), states), h


class Server:
    def __init__(self, model, rows, limit, bits8=False, cache8=False):
        self.model, self.rows, self.length = model, rows, 0
        self.layers = [Served(layer, rows, limit, bits8, cache8) for layer in model.layers]

    @torch.no_grad()
    def feed(self, tokens):
        """tokens [rows, n] -> logits [rows, n, vocab], in calls that end with
        the open chunk at the latest."""
        out, dev = [], tokens.device
        while tokens.shape[1]:
            at = self.length % CHUNK
            n = min(CHUNK - at, tokens.shape[1])
            cu = torch.arange(self.rows + 1, dtype=torch.int32, device=dev) * n
            cached = torch.full((self.rows,), self.length, dtype=torch.int32, device=dev)
            x, h = self.model.embedded(tokens[:, :n]), None
            for layer in self.layers:
                x, h = layer.step(x, h, cu, cached, at, n)
            out.append(self.model.logits(x, h).view(self.rows, n, -1))
            self.length += n
            tokens = tokens[:, n:]
        return torch.cat(out, dim=1)


def batch(rows, T, vocab, gen):
    """Chains in which nine tokens of ten are the one before them times 5 plus 1."""
    tokens, free = (torch.randint(vocab, (rows, T), generator=gen) for _ in range(2))
    free = free < vocab // 10
    for i in range(1, T):
        tokens[:, i] = torch.where(free[:, i], tokens[:, i], (tokens[:, i - 1] * 5 + 1) % vocab)
    return tokens.cuda()


def train(model, steps, rows, T, lr=1e-3, seed=0):
    """Losses of the steps."""
    gen = torch.Generator().manual_seed(seed)
    opt = torch.optim.AdamW(model.parameters(), lr=lr)
    losses = []
    for _ in range(steps):
        tokens = batch(rows, T + 1, model.embed.num_embeddings, gen)
        loss = F.cross_entropy(model(tokens[:, :-1]).float().flatten(0, 1), tokens[:, 1:].flatten())
        opt.zero_grad(set_to_none=True)
        loss.backward()
        nn.utils.clip_grad_norm_(model.parameters(), 1.0)
        opt.step()
        losses.append(float(loss.detach()))
    return losses


def serve(model, tokens, prompt, bits8=False, cache8=False):
    """Logits of the tokens: a prompt in chunks, then one by one."""
    server = Server(model, tokens.shape[0], tokens.shape[1], bits8, cache8)
    out = [server.feed(tokens[:, :prompt])] if prompt else []
    for i in range(prompt, tokens.shape[1]):
        out.append(server.feed(tokens[:, i:i + 1]))
    return torch.cat(out, dim=1)


@torch.no_grad()
def generate(model, prompt, n, gen, cache8=False, **filters):
    """n tokens per row of prompt, [rows, n], and the logs of the probabilities that
    they were drawn with; ``filters`` as for ``sample``, gen a generator on the CPU."""
    rows = prompt.shape[0]
    server = Server(model, rows, prompt.shape[1] + n, cache8=cache8)
    u = torch.rand(n, rows, generator=gen).to(prompt.device)
    logits, tokens, logprobs = server.feed(prompt)[:, -1], [], []
    for i in range(n):
        token, logprob = e2.sample(logits, u[i], **filters)
        tokens.append(token)
        logprobs.append(logprob)
        if i + 1 < n:
            logits = server.feed(token[:, None])[:, -1]
    return torch.stack(tokens, dim=1), torch.stack(logprobs, dim=1)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=100)
    ap.add_argument("--rows", type=int, default=8)
    ap.add_argument("--tokens", type=int, default=768)
    ap.add_argument("--recur", type=int, default=0, help="channels of the gated linear recurrence, a multiple of 8")
    a = ap.parse_args()
    torch.manual_seed(0)
    model = Model(recur=a.recur).cuda()
    losses = train(model, a.steps, a.rows, a.tokens)
    for i in range(0, a.steps, max(1, a.steps // 10)):
        print(f"step {i:4d}  loss {losses[i]:.3f}")
    print(f"last       loss {losses[-1]:.3f}")

    tokens = batch(a.rows, 600, model.embed.num_embeddings, torch.Generator().manual_seed(1))
    with torch.no_grad():
        want = F.pad(tokens, (0, -tokens.shape[1] % CHUNK))  # causal: what follows does not reach the tokens
        want = model(want)[:, :tokens.shape[1]].float()
    for how, kw in (("in bf16", {}), ("with 8-bit projections", dict(bits8=True)), ("with an 8-bit cache", dict(cache8=True))):
        got = serve(model, tokens, 500, **kw).float()
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        serve(model, tokens, 500, **kw)
        torch.cuda.synchronize()
        t = time.perf_counter() - t0
        print(f"served {how}: logits differ from the training forward's by "
              f"{float((got - want).norm() / want.norm()):.4f} of their norm; {a.rows} streams of 500 + 100 tokens in "
              f"{t * 1e3:.0f} ms")

    drawn, logprobs = generate(model, tokens[:, :64], 100, torch.Generator().manual_seed(2), cache8=True,
                               temperature=0.8, top_k=50, top_p=0.95)
    chain = torch.cat([tokens[:, 63:64], drawn], dim=1)
    follows = (chain[:, 1:] == (chain[:, :-1] * 5 + 1) % model.embed.num_embeddings).float().mean()
    print(f"drawn: {float(follows):.2f} of the tokens continue the chain, mean log probability {float(logprobs.mean()):.3f}")


if __name__ == "__main__":
    main()
