"""The two ends of a hybrid model: Python binding of include/e2ttt_tokens.h.

Argument marshalling only, by the conventions of ``layer.py``.
"""
from __future__ import annotations

import ctypes
import math
from functools import lru_cache

import torch
from torch.autograd.function import once_differentiable

from ._lib import EmbeddingDesc, SampleDesc
from .layer import _IO, _call, _device, _full, _layout, _on, _one_stream_behind, _p, _size, _workspace

_TOKEN_BYTES = {torch.int32: 4, torch.int64: 8}


@lru_cache(maxsize=512)
def _embedding_plan(tokens, dtype, vocab, width, table_dtype, scale):
    shape, token_dtype = tokens
    if token_dtype not in _TOKEN_BYTES:
        raise TypeError(f"tokens must be int32 or int64, got {token_dtype}")
    for t in (dtype, table_dtype):
        if t not in _IO:
            raise TypeError(f"expected float32 or bfloat16, got {t}")
    n = math.prod(shape)
    d = EmbeddingDesc(_IO[table_dtype], _IO[dtype], _TOKEN_BYTES[token_dtype], scale, n, vocab, width)
    return n, ctypes.byref(d), _size("e2ttt_embedding_backward_workspace_size", d), d


def embedding_forward(tokens, weight, *, scale: float = 1.0, dtype=None, out=None, stream=None):
    """Rows of ``weight`` by token, times ``scale``; returns out.

    tokens: any shape, int32 or int64, contiguous; one outside [0, V) gives a row
    of zeros.  weight: [V, W] float32 or bfloat16, contiguous.  out: [..., W] in
    ``dtype`` (the weight's by default).
    """
    if stream is not None:
        with _on(stream, tokens):
            return embedding_forward(tokens, weight, scale=scale, dtype=dtype, out=out)
    dev = _device(tokens, weight=weight, out=out)
    if weight.dim() != 2 or not weight.is_contiguous() or not tokens.is_contiguous():
        raise ValueError("weight must be a contiguous (V, W) tensor, and tokens contiguous")
    dtype = weight.dtype if dtype is None else dtype
    n, desc, _, _ = _embedding_plan((tokens.shape, tokens.dtype), dtype, *weight.shape, weight.dtype, scale)
    shape = (*tokens.shape, weight.shape[1])
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=weight.device)
    else:
        _full("out", out, shape, dtype)
    if n:
        _call("e2ttt_embedding_forward", dev, desc, tokens.data_ptr(), weight.data_ptr(), out.data_ptr())
    return out


def embedding_backward(dout, tokens, vocab: int, *, scale: float = 1.0, dtype=None, out=None, workspace=None, stream=None):
    """Gradient of <dout, embedding_forward(tokens, weight)> with respect to a
    weight of ``vocab`` rows: [vocab, W] in ``dtype`` (dout's by default), zeros
    for tokens that do not occur.  dout: [..., W], contiguous."""
    if stream is not None:
        with _on(stream, tokens):
            return embedding_backward(dout, tokens, vocab, scale=scale, dtype=dtype, out=out, workspace=workspace)
    dev = _device(tokens, dout=dout, out=out)
    if dout.dim() < 1 or dout.shape[:-1] != tokens.shape:
        raise ValueError(f"dout must have shape {(*tokens.shape, 'W')}, got {tuple(dout.shape)}")
    if not dout.is_contiguous() or not tokens.is_contiguous():
        raise ValueError("dout and tokens must be contiguous")
    dtype = dout.dtype if dtype is None else dtype
    W = dout.shape[-1]
    _, desc, need, _ = _embedding_plan((tokens.shape, tokens.dtype), dout.dtype, vocab, W, dtype, scale)
    if out is None:
        out = torch.empty(vocab, W, dtype=dtype, device=dout.device)
    else:
        _full("out", out, (vocab, W), dtype)
    ws, n = _workspace(workspace, need, dout)
    _call("e2ttt_embedding_backward", dev, desc, dout.data_ptr(), tokens.data_ptr(), out.data_ptr(), ws, n)
    return out


class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, tokens, weight, scale, dtype):
        ctx.save_for_backward(tokens)
        ctx.opts = (weight.shape[0], scale, weight.dtype)
        return embedding_forward(tokens, weight, scale=scale, dtype=dtype)

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        vocab, scale, dtype = ctx.opts
        return None, embedding_backward(dout.contiguous(), ctx.saved_tensors[0], vocab, scale=scale, dtype=dtype), None, None


def embedding(tokens, weight, *, scale: float = 1.0, dtype=None):
    """``embedding_forward`` as a differentiable op, with the weight's gradient
    (dense, in the weight's type) from ``embedding_backward``.  Captured into a graph
    with its backward pass, no eager graph of the same leaves may be alive (RuntimeError, where
    one of the leaves was given to a call of this package directly)."""
    out = _Embedding.apply(tokens, weight, scale, dtype)
    _one_stream_behind(out, tokens.get_device())
    return out


@lru_cache(maxsize=512)
def _sample_plan(logits, temperature, top_k, top_p, min_p):
    shape, stride, dtype = logits
    if len(shape) != 2:
        raise ValueError(f"logits must have shape (rows, vocab), got {tuple(shape)}")
    if dtype not in _IO:
        raise TypeError(f"expected float32 or bfloat16, got {dtype}")
    if shape[1] > 1 and stride[1] != 1:
        raise ValueError("logits' last dimension must be contiguous")
    top_k = max(0, min(top_k, 0x7fffffff))  # ctypes would take a larger number's low 32 bits
    d = SampleDesc(_IO[dtype], top_k, temperature, top_p, min_p, 0, shape[0], shape[1], stride[0])
    return shape[0], ctypes.byref(d), _size("e2ttt_sample_workspace_size", d), d


def _setting(name, x, rows, dtype, off):
    """A number for all rows, or a tensor with one each: (number, tensor)."""
    if not torch.is_tensor(x):
        return x, None
    _full(name, x, (rows,), dtype)
    return off, x


def sample(logits, u, *, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, token=None, logprob=None, workspace=None,
           stream=None):
    """One token per row of logits from given random numbers; returns (token,
    logprob): [rows] int64, and [rows] float32, the log of the probability with
    which it was drawn.

    logits: [rows, V] float32 or bfloat16, last dimension contiguous; u: [rows]
    float32 in [0, 1).  The filters are numbers or tensors of one value per row
    (float32; top_k int32): ``temperature`` (0: the largest logit), then the
    ``top_k`` largest (0: all), then the fewest of those that have ``top_p`` of
    their weight (1: all), then those with at least ``min_p`` of the largest
    probability.  Equal logits are taken by index.  Of what is left, in order of
    index, the token is the one at which the running probability exceeds u.  A
    row without any logit above -infinity gives -1, logprob NaN.
    """
    if stream is not None:
        with _on(stream, logits):
            return sample(logits, u, temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p, token=token,
                          logprob=logprob, workspace=workspace)
    rows = logits.shape[0] if logits.dim() else 0
    temperature, t_row = _setting("temperature", temperature, rows, torch.float32, 1.0)
    top_k, k_row = _setting("top_k", top_k, rows, torch.int32, 0)
    top_p, p_row = _setting("top_p", top_p, rows, torch.float32, 1.0)
    min_p, m_row = _setting("min_p", min_p, rows, torch.float32, 0.0)
    dev = _device(logits, u=u, temperature=t_row, top_k=k_row, top_p=p_row, min_p=m_row, token=token, logprob=logprob)
    n, desc, need, _ = _sample_plan(_layout(logits), temperature, top_k, top_p, min_p)
    _full("u", u, (n,), torch.float32)
    if token is None:
        token = torch.empty(n, dtype=torch.int64, device=logits.device)
    else:
        _full("token", token, (n,), torch.int64)
    if logprob is None:
        logprob = torch.empty(n, dtype=torch.float32, device=logits.device)
    else:
        _full("logprob", logprob, (n,), torch.float32)
    ws, nb = _workspace(workspace, need, logits)
    _call("e2ttt_sample", dev, desc, logits.data_ptr(), u.data_ptr(), _p(t_row), _p(k_row), _p(p_row), _p(m_row),
          token.data_ptr(), logprob.data_ptr(), ws, nb)
    return token, logprob
