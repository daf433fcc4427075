"""Plain 64-bit implementations of the hybrid layer's operators, on the CPU,
one sequence and one query head at a time, with a bound on how far a kernel's
result may be from each value.

The bounds follow from the arithmetic, elementwise, with

  u     relative error of rounding a result to its type, half the spacing: bf16
        has 8 significant bits, 2^-8; fp32 24, 2^-24;
  w     relative error of rounding an operand (probabilities and score
        gradients, to bf16): 2^-8, or 0 in fp32, where they stay as they are;
  e_i   relative error of row i's probabilities in fp32.  A score is a sum of D
        products, off by at most (D + 2) 2^-24 scale sum |q_d k_d|; the
        exponential of it and of lse (off by as much again) doubles that; the
        exponent's own rounding adds 2 |s| 2^-24 and the base-2 exponential a
        few units, taken together as 2^-20;
  f     (terms + 8) 2^-24, the error of an fp32 sum of so many terms relative
        to the sum of their magnitudes.
"""
from __future__ import annotations

import numpy as np

BF16, F32 = "bf16", "f32"
TINY = 1e-30


def units(dtype):
    return (2.0 ** -8, 2.0 ** -8) if dtype == BF16 else (2.0 ** -24, 0.0)


def visible(first, n, keys, window):
    """[n, keys]: whether the query at position first + i sees key j."""
    p = first + np.arange(n)[:, None]
    j = np.arange(keys)[None, :]
    v = j <= p
    return v & (j > p - window) if window else v


def attention(q, k, v, first, window, scale, dtype, dout=None):
    """q [n, D] at positions first..., k, v [keys, D], all float64.  Returns a
    dict of (value, bound): out, lse and, with dout, dq, dk, dv."""
    u, w = units(dtype)
    n, D = q.shape
    keys = k.shape[0]
    see = visible(first, n, keys, window)
    with np.errstate(invalid="ignore", over="ignore"):
        s = np.where(see, scale * (q @ k.T), -np.inf)
        mag = np.where(see, scale * (np.abs(q) @ np.abs(k).T), 0.0)
    e = 4 * (D + 2) * 2.0 ** -24 * mag.max(axis=1) + 2.0 ** -20  # [n]
    f = (keys + 8) * 2.0 ** -24
    top = s.max(axis=1, initial=-np.inf)
    safe = np.where(np.isfinite(top), top, 0.0)
    p = np.exp(s - safe[:, None])
    total = p.sum(axis=1)
    lse = np.where(total > 0, safe + np.log(np.where(total > 0, total, 1.0)), -np.inf)
    p = p / np.where(total > 0, total, 1.0)[:, None]
    vz = np.where(see.any(axis=0)[:, None], v, 0.0)  # what nobody sees may be anything
    out = p @ vz
    vmag = p @ np.abs(vz)
    r = {"out": (out, u * np.abs(out) + (w + e[:, None] + f) * vmag * 1.01 + TINY),
         "lse": (lse, e + f + 2.0 ** -22 * np.abs(safe) + 2.0 ** -22)}
    if dout is None:
        return r
    kz = np.where(see.any(axis=0)[:, None], k, 0.0)
    r["dv"] = (p.T @ dout, None)
    dvmag = ((p * (1 + 0 * e[:, None])).T @ np.abs(dout))
    fr = (n + 8) * 2.0 ** -24
    r["dv"] = (p.T @ dout, u * np.abs(p.T @ dout) + 1.01 * ((w + fr) * dvmag + (p * e[:, None]).T @ np.abs(dout)) + TINY)
    dp = dout @ vz.T
    dpmag = np.abs(dout) @ np.abs(vz).T
    delta = (dout * out).sum(axis=1)
    # delta comes from the out that the forward returned
    ddelta = (np.abs(dout) * r["out"][1]).sum(axis=1) + (D + 2) * 2.0 ** -24 * (np.abs(dout) * np.abs(out)).sum(axis=1)
    ds = p * (dp - delta[:, None])
    err = w * np.abs(ds) + e[:, None] * np.abs(ds) + p * (ddelta[:, None] + (D + 4) * 2.0 ** -24 * (dpmag + np.abs(delta)[:, None]))
    dq = scale * ds @ kz
    dk = scale * ds.T @ q
    r["dq"] = (dq, u * np.abs(dq) + 1.01 * scale * ((err + f * np.abs(ds)) @ np.abs(kz)) + TINY)
    r["dk"] = (dk, u * np.abs(dk) + 1.01 * scale * ((err + fr * np.abs(ds)).T @ np.abs(q)) + TINY)
    return r


def packed(q, k, v, lens, window, scale, dtype, dout=None):
    """attention over packed sequences and all heads; float64 [N, H, D].  A key
    head's gradient is the sum over its group, and so is its bound."""
    N, H, D = q.shape
    K = k.shape[1]
    G = H // K
    names = ["out", "lse"] + (["dq", "dk", "dv"] if dout is not None else [])
    shape = {"out": (N, H, D), "lse": (N, H), "dq": (N, H, D), "dk": (N, K, D), "dv": (N, K, D)}
    val = {n: np.zeros(shape[n]) for n in names}
    bnd = {n: np.zeros(shape[n]) for n in names}
    a = 0
    for n in lens:
        sl = slice(a, a + n)
        for h in range(H):
            if n == 0:
                continue
            r = attention(q[sl, h], k[sl, h // G], v[sl, h // G], 0, window, scale, dtype,
                          None if dout is None else dout[sl, h])
            for name in names:
                at = h // G if name in ("dk", "dv") else h
                val[name][sl, at] += r[name][0]
                bnd[name][sl, at] += r[name][1]
        a += n
    if dout is not None and G > 1:  # the fp32 sum over the group
        for name in ("dk", "dv"):
            bnd[name] *= 1.0 + 1e-3
    return val, bnd


def norm(x, residual, weight, eps, dtype, round_to, dy=None, dh=None):
    """x, residual [rows, W] and weight [W], float64; round_to rounds float64
    values to the stream's type.  Returns a dict of (value, bound)."""
    u, _ = units(dtype)
    rows, W = x.shape
    h = x if residual is None else round_to(x + residual)
    f = (W + 8) * 2.0 ** -24
    rstd = 1.0 / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps)
    er = f + 2.0 ** -21  # of rstd, relative
    xhat = h * rstd
    y = xhat * weight
    r = {"h": (h, np.zeros_like(h)), "rstd": (rstd[:, 0], er * rstd[:, 0]),
         "y32": (y, (er + 2.0 ** -22) * np.abs(y)), "y": (y, (u + er + 2.0 ** -22) * 1.01 * np.abs(y) + TINY)}
    if dy is None:
        return r
    gg = dy * weight
    c = (gg * xhat).mean(axis=1, keepdims=True)
    cb = (f + 2 * er) * (np.abs(gg * xhat)).mean(axis=1, keepdims=True)
    dx = rstd * (gg - xhat * c)
    db = rstd * ((2 * er + 2.0 ** -21) * (np.abs(gg) + np.abs(xhat * c)) + np.abs(xhat) * cb)
    if dh is not None:
        dx = dx + dh
        db = db + 2.0 ** -23 * (np.abs(dx) + np.abs(dh))
    r["dx"] = (dx, u * np.abs(dx) * 1.01 + db + TINY)
    fr = (rows + 8) * 2.0 ** -24
    r["dweight"] = ((dy * xhat).sum(axis=0), (fr + er + 2.0 ** -22) * np.abs(dy * xhat).sum(axis=0) + TINY)
    return r
