"""Plain 64-bit implementations of the operators around a hybrid model's layers, on
the CPU, with a bound on how far a kernel's result may be from each value.

Bounds.  u is half the spacing of a type relative to the value: bf16 2^-8, fp32
2^-24; e = 2^-24 is that of the sums, which are held in fp32.

Recurrence.  A value h_t is a sum over s <= t of x_s times the gates between, and
(t = 0) h0 times all of them.  Each term passes a multiplication, rounded with
the addition after it, per step, and where stretches are folded a product of
gates that was itself rounded once per gate: at most two roundings per step, and
a few more where stretches meet (16 tokens, tiles, parts; 64 in all).  With
m_t = |a_t| m_{t-1} + |x_t| and d_t = |a_t| (d_{t-1} + m_{t-1}), the sum of
magnitudes and of magnitudes times steps, the error is at most
e (2 d_t + 64 m_t).  The gradient is the same recurrence run backwards, and
da_t = g_t h_{t-1} adds both relative errors and a rounding.

Lookup.  scale times a value, rounded to fp32 and to the type: u + e of it.  Its
gradient: a sum of n values, and the product with the scale: (n + 2) e of the
sum of magnitudes, and u of the result.
"""
from __future__ import annotations

import numpy as np

E = 2.0 ** -24
U = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
TINY = 1e-37  # below it fp32 itself is coarse


def recurrence(x, a, h0):
    """x, a [n, C], h0 [C], float64 -> (h [n, C], state [C]) and bounds of the same."""
    n, C = x.shape
    h, m, d = h0.copy(), np.abs(h0), np.zeros(C)
    out, bound = np.zeros((n, C)), np.zeros((n, C))
    for t in range(n):
        h = a[t] * h + x[t]
        d = np.abs(a[t]) * (d + m)
        m = np.abs(a[t]) * m + np.abs(x[t])
        out[t], bound[t] = h, E * (2 * d + 64 * m)
    return out, bound, h, (bound[-1] if n else np.zeros(C))


def scan(x, a, h0, lens, before, dtype, gate, dout=None, dstate=None):
    """Packed sequences from token `before` on; float64.  {name: (value, bound)}."""
    N, C = x.shape
    r = {k: (np.zeros((N, C)), np.zeros((N, C))) for k in ("out", "dx", "da")}
    r.update({k: (np.zeros((len(lens), C)), np.zeros((len(lens), C))) for k in ("state", "dh0")})
    at = before
    for i, n in enumerate(lens):
        s = slice(at, at + n)
        h, b, end, eb = recurrence(x[s], a[s], h0[i])
        r["out"][0][s], r["out"][1][s] = h, b + U[dtype] * np.abs(h)
        r["state"][0][i], r["state"][1][i] = end, eb
        at += n
        if dout is None:
            continue
        if n == 0:
            r["dh0"][0][i] = dstate[i]
            continue
        # g_t = dout_t + a_{t+1} g_{t+1}, the last with dstate
        after = np.concatenate([a[s][1:], np.ones((1, C))])[::-1]
        g, gb, _, _ = recurrence(dout[s][::-1], after, dstate[i])
        g, gb = g[::-1], gb[::-1]
        prev = np.concatenate([h0[i][None], h[:-1]])
        pb = np.concatenate([np.zeros((1, C)), b[:-1]])
        r["dx"][0][s], r["dx"][1][s] = g, gb + U[dtype] * np.abs(g)
        r["da"][0][s] = g * prev
        r["da"][1][s] = np.abs(prev) * gb + np.abs(g) * pb + gb * pb + (U[gate] + 2 * E) * np.abs(g * prev)
        r["dh0"][0][i], r["dh0"][1][i] = a[s][0] * g[0], np.abs(a[s][0]) * gb[0] + 2 * E * np.abs(a[s][0] * g[0])
    return {k: (v, b + TINY) for k, (v, b) in r.items()}


def lookup(tokens, table, scale, dtype):
    ok = (tokens >= 0) & (tokens < table.shape[0])
    v = np.where(ok[:, None], table[np.where(ok, tokens, 0)] * scale, 0.0)
    return v, (U[dtype] + E) * np.abs(v) + TINY


def lookup_gradient(tokens, dout, vocab, scale, dtype):
    v, m, n = np.zeros((vocab, dout.shape[1])), np.zeros((vocab, dout.shape[1])), np.zeros(vocab)
    ok = (tokens >= 0) & (tokens < vocab)
    np.add.at(v, tokens[ok], dout[ok])
    np.add.at(m, tokens[ok], np.abs(dout[ok]))
    np.add.at(n, tokens[ok], 1)
    v, m = v * scale, m * abs(scale)
    return v, (n[:, None] + 2) * E * m + U[dtype] * np.abs(v) + TINY


ONE = 1 << 44


def sample(logits, u, temperature, top_k, top_p, min_p):
    """One row, float64 logits and settings: (token, logprob, bound of logprob,
    distance of u from the nearest place where the token changes).  Sums of weights are
    whole numbers, exact."""
    from fractions import Fraction
    x = np.where(np.isnan(logits), -np.inf, logits)
    top = x.max()
    if top == -np.inf:
        return -1, np.nan, 0.0, 1.0
    if not temperature > 0:
        return int(np.argmax(x)), 0.0, 0.0, 1.0
    with np.errstate(invalid="ignore", over="ignore"):
        p = np.where(x == top, 1.0, np.where(x == -np.inf, 0.0, np.exp((x - top) / temperature)))
    w = [int(v) for v in np.rint(p * ONE)]
    order = sorted(range(len(x)), key=lambda i: (-x[i], i))
    if 0 < top_k < len(x):
        order = order[:top_k]
    if top_p < 1:
        whole, run, kept = sum(w[i] for i in order), 0, []
        for i in order:
            if kept and run >= Fraction(float(max(top_p, 0.0))) * whole:
                break
            kept.append(i)
            run += w[i]
        order = kept
    order = sorted(i for i in order if p[i] >= min(min_p, 1.0))
    total, run = sum(w[i] for i in order), 0
    at = Fraction(float(u)) * total
    for i in order:
        if run + w[i] > at:
            # a weight may be off by one unit, its log by that, and the result rounds to fp32
            lp = np.log(w[i] / total)
            # the first border and the last are exact, and all of them among equal weights of one
            far = min(at - run if run else total, run + w[i] - at if run + w[i] < total else total)
            far = total if all(w[k] == ONE for k in order) else far
            return i, lp, 2.0 ** -23 * abs(lp) + 2.0 / w[i] + 2.0 ** -40, float(far / total)
        run += w[i]
    raise AssertionError


def quantise(x):
    """Rows [..., D] float64 of bf16 values: (8-bit values times scale, biased exponent)."""
    import torch
    top = np.abs(x).max(axis=-1)
    b = np.full(top.shape, 127)
    for idx in np.ndindex(top.shape):
        if not np.isfinite(x[idx]).all():
            b[idx] = 255
        elif top[idx] > 0:
            b[idx] = next(e for e in range(255) if top[idx] <= 448 * 2.0 ** (e - 127))
    s = np.where(b < 255, 2.0 ** (b.astype(np.float64) - 127), np.nan)[..., None]
    y = torch.from_numpy((x / s).astype(np.float32)).to(torch.float8_e4m3fn).double().numpy()
    return y * s, b
