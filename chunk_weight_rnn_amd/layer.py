"""The operators of a hybrid layer beside the chunk update: Python binding of
include/e2ttt_layer.h.

Argument marshalling only, as in the package's ``__init__``: the work runs in
the HIP kernels behind the C ABI on the current stream (or ``stream``), with
tensors that the caller owns; outputs and workspaces that are not given are
allocated through torch.  CPU tensors raise.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from ._lib import AttentionDesc, E2TTTError, NormDesc, PagedDesc

_IO = {torch.float32: 0, torch.bfloat16: 1}
_BAD = ctypes.c_size_t(-1).value
F8 = torch.float8_e4m3fn


def _p(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    return (stream if stream is not None else torch.cuda.current_stream()).cuda_stream


def _gpu(**tensors):
    for name, t in tensors.items():
        if t is not None and not t.is_cuda:
            raise ValueError(f"{name} must be a GPU tensor (no CPU path exists)")


def _io(t: torch.Tensor) -> int:
    if t.dtype not in _IO:
        raise TypeError(f"expected float32 or bfloat16, got {t.dtype}")
    return _IO[t.dtype]


def _heads3(name, t, N, D, dtype):
    """Checks a [tokens, heads, D] tensor whose last dimension is contiguous."""
    if t.dim() != 3 or t.shape[0] != N or t.shape[2] != D:
        raise ValueError(f"{name} must have shape ({N}, heads, {D}), got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    if t.stride(2) != 1 and D > 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")


def _int32(name, t, shape):
    if t.dtype != torch.int32 or tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor of shape {shape}")


def _full(name, t, shape, dtype):
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _attention_desc(q, k, v, cu_seqlens, window, scale, kv_heads) -> AttentionDesc:
    if q.dim() != 3:
        raise ValueError(f"q must have shape (tokens, heads, D), got {tuple(q.shape)}")
    N, H, D = q.shape
    _heads3("q", q, N, D, q.dtype)
    io = _io(q)
    if k is not None:
        _heads3("k", k, N, D, q.dtype)
        _heads3("v", v, N, D, q.dtype)
        if k.shape[1] != kv_heads or v.shape[1] != kv_heads:
            raise ValueError("k and v must have the same heads")
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
        raise ValueError("cu_seqlens must have shape (sequences + 1,)")
    _int32("cu_seqlens", cu_seqlens, (cu_seqlens.shape[0],))
    if scale is None:
        scale = D ** -0.5 if D else 1.0
    s = (0, 0) if k is None else k.stride()
    t = (0, 0) if v is None else v.stride()
    return AttentionDesc(io, window, N, cu_seqlens.shape[0] - 1, H, kv_heads, D, scale, 0, q.stride(0), q.stride(1),
                         s[0], s[1], t[0], t[1])


def _workspace(fn, desc, workspace, device):
    n = getattr(_lib.load(), fn)(ctypes.byref(desc))
    if n == _BAD:
        return None, 0  # the call itself names the reason
    if workspace is None:
        workspace = torch.empty(n, dtype=torch.uint8, device=device) if n else None
    return workspace, (0 if workspace is None else workspace.numel())


def attention_forward(q, k, v, cu_seqlens, *, window: int = 0, scale: float | None = None, out=None, lse=None,
                      workspace=None, stream=None):
    """Causal attention over packed sequences; returns (out, lse).

    q: [N, H, D], k, v: [N, K, D], float32 or bfloat16, last dimension
    contiguous (views of one projection's output are fine); H a multiple of K,
    D a multiple of 8 up to 128.  cu_seqlens: [S + 1] int32 on the GPU, the
    sequences' offsets into the N tokens.  ``window`` > 0: a query sees that
    many positions, its own the last.  ``scale``: of the scores, D ** -0.5 by
    default.  out: [N, H, D]; lse: [N, H] float32, the log of each row's
    softmax sum, which the backward needs.
    """
    _gpu(q=q, k=k, v=v, cu_seqlens=cu_seqlens, out=out, lse=lse)
    desc = _attention_desc(q, k, v, cu_seqlens, window, scale, k.shape[1] if k.dim() == 3 else 0)
    N, H, D = q.shape
    if out is None:
        out = torch.empty(N, H, D, dtype=q.dtype, device=q.device)
    else:
        _full("out", out, (N, H, D), q.dtype)
    if lse is None:
        lse = torch.empty(N, H, dtype=torch.float32, device=q.device)
    else:
        _full("lse", lse, (N, H), torch.float32)
    ws, n = _workspace("e2ttt_attention_workspace_size", desc, workspace, q.device)
    st = _lib.load().e2ttt_attention_forward(ctypes.byref(desc), _p(q), _p(k), _p(v), _p(cu_seqlens), _p(out),
                                             _p(lse), _p(ws), n, _stream(stream))
    if st != 0:
        raise E2TTTError("e2ttt_attention_forward", st)
    return out, lse


def attention_backward(q, k, v, out, lse, dout, cu_seqlens, *, window: int = 0, scale: float | None = None,
                       workspace=None, stream=None):
    """Gradients of <dout, out> through ``attention_forward``, from its inputs
    and outputs; returns a dict with keys q, k, v (the I/O dtype, contiguous)."""
    _gpu(q=q, k=k, v=v, out=out, lse=lse, dout=dout, cu_seqlens=cu_seqlens)
    desc = _attention_desc(q, k, v, cu_seqlens, window, scale, k.shape[1] if k.dim() == 3 else 0)
    N, H, D = q.shape
    _full("out", out, (N, H, D), q.dtype)
    _full("dout", dout, (N, H, D), q.dtype)
    _full("lse", lse, (N, H), torch.float32)
    g = {n: torch.empty(t.shape, dtype=q.dtype, device=q.device) for n, t in (("q", q), ("k", k), ("v", v))}
    ws, n = _workspace("e2ttt_attention_backward_workspace_size", desc, workspace, q.device)
    st = _lib.load().e2ttt_attention_backward(ctypes.byref(desc), _p(q), _p(k), _p(v), _p(out), _p(lse), _p(dout),
                                              _p(cu_seqlens), _p(g["q"]), _p(g["k"]), _p(g["v"]), _p(ws), n,
                                              _stream(stream))
    if st != 0:
        raise E2TTTError("e2ttt_attention_backward", st)
    return g


class _Attention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, cu_seqlens, window, scale):
        out, lse = attention_forward(q, k, v, cu_seqlens, window=window, scale=scale)
        ctx.save_for_backward(q, k, v, out, lse, cu_seqlens)
        ctx.opts = (window, scale)
        return out

    @staticmethod
    def backward(ctx, dout):
        q, k, v, out, lse, cu_seqlens = ctx.saved_tensors
        window, scale = ctx.opts
        g = attention_backward(q, k, v, out, lse, dout.contiguous(), cu_seqlens, window=window, scale=scale)
        return g["q"], g["k"], g["v"], None, None, None


def attention(q, k, v, cu_seqlens, *, window: int = 0, scale: float | None = None):
    """``attention_forward`` as a differentiable op: returns out, with gradients
    for q, k and v from ``attention_backward``."""
    return _Attention.apply(q, k, v, cu_seqlens, window, scale)


def paged_attention(q, k, v, k_cache, v_cache, table, cu_seqlens, cached, *, window: int = 0,
                    scale: float | None = None, out=None, workspace=None, stream=None):
    """Attention of each sequence's new tokens over its cached ones and
    themselves; writes the new keys and values into the cache; returns out.

    q: [N, H, D], k, v: [N, K, D]: the new tokens of all sequences, packed by
    cu_seqlens [S + 1] int32 (one each: plain decoding; more: a chunk of a
    prompt).  k_cache, v_cache: [pages, K, page_size, D], page_size a power of
    two (any strides with a contiguous last dimension).  table: [S, W] int32,
    the pages of each sequence; cached: [S] int32, its tokens in the cache
    before the call.  New token i of sequence s is at position cached[s] + i.
    With k = v = None the cache holds the new tokens already.
    """
    if (k is None) != (v is None):
        raise ValueError("k and v must both be given, or neither")
    _gpu(q=q, k=k, v=v, k_cache=k_cache, v_cache=v_cache, table=table, cu_seqlens=cu_seqlens, cached=cached, out=out)
    if k_cache.dim() != 4 or k_cache.shape != v_cache.shape:
        raise ValueError("k_cache and v_cache must share one shape (pages, K, page_size, D)")
    P, K, ps, Dc = k_cache.shape
    if k_cache.dtype != q.dtype or v_cache.dtype != q.dtype:
        raise TypeError(f"k_cache and v_cache must be {q.dtype}")
    a = _attention_desc(q, k, v, cu_seqlens, window, scale, K)
    N, H, D = q.shape
    if Dc != D or (D > 1 and (k_cache.stride(3) != 1 or v_cache.stride(3) != 1)):
        raise ValueError(f"k_cache and v_cache must have a contiguous last dimension of {D}")
    S = cu_seqlens.shape[0] - 1
    if table.dim() != 2:
        raise ValueError("table must have shape (sequences, width)")
    _int32("table", table, (S, table.shape[1]))
    _int32("cached", cached, (S,))
    if out is None:
        out = torch.empty(N, H, D, dtype=q.dtype, device=q.device)
    else:
        _full("out", out, (N, H, D), q.dtype)
    s, t = k_cache.stride(), v_cache.stride()
    desc = PagedDesc(a, P, ps, table.shape[1], s[0], s[1], s[2], t[0], t[1], t[2])
    ws, n = _workspace("e2ttt_paged_workspace_size", desc, workspace, q.device)
    st = _lib.load().e2ttt_paged_attention(ctypes.byref(desc), _p(q), _p(k), _p(v), _p(k_cache), _p(v_cache),
                                           _p(table), _p(cu_seqlens), _p(cached), _p(out), _p(ws), n, _stream(stream))
    if st != 0:
        raise E2TTTError("e2ttt_paged_attention", st)
    return out


def _norm_desc(x, weight, eps, bits8) -> NormDesc:
    if x.dim() < 1 or not x.is_contiguous():
        raise ValueError("x must be contiguous, [..., width]")
    W = x.shape[-1]
    _full("weight", weight, (W,), torch.float32)
    return NormDesc(_io(x), int(bits8), x.numel() // W if W else 0, W, eps, 0)


def norm_forward(x, weight, *, residual=None, eps: float = 1e-6, bits8: bool = False, h=None, stream=None):
    """Root-mean-square norm with the residual's addition; returns
    (y, scale, h, rstd).

    x: [..., W] float32 or bfloat16, contiguous; weight: [W] float32.
    h = x + residual in x's type (x itself without ``residual``; ``h=residual``
    updates the stream in place); rstd: [...] float32, for the backward.
    y = h * rstd * weight in x's type, or with ``bits8`` in float8_e4m3fn, to be
    multiplied by scale [...] (float32, max|y| / 448 of its row; else None).
    """
    _gpu(x=x, weight=weight, residual=residual, h=h)
    desc = _norm_desc(x, weight, eps, bits8)
    if residual is not None:
        _full("residual", residual, x.shape, x.dtype)
        if h is None:
            h = torch.empty_like(x)
        else:
            _full("h", h, x.shape, x.dtype)
    elif h is not None:
        raise ValueError("h is an output of the residual's addition: give residual too")
    y = torch.empty(x.shape, dtype=F8 if bits8 else x.dtype, device=x.device)
    scale = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device) if bits8 else None
    rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    st = _lib.load().e2ttt_norm_forward(ctypes.byref(desc), _p(x), _p(residual), _p(weight), _p(y), _p(scale), _p(h),
                                        _p(rstd), _stream(stream))
    if st != 0:
        raise E2TTTError("e2ttt_norm_forward", st)
    return y, scale, (x if residual is None else h), rstd


def norm_backward(dy, h, weight, rstd, *, dh=None, workspace=None, stream=None):
    """Gradients through ``norm_forward`` (y in the stream's type): returns
    (dx, dweight).  dx is the gradient of both x and residual; ``dh`` is what
    arrives at h along the residual stream, added to it."""
    _gpu(dy=dy, h=h, weight=weight, rstd=rstd, dh=dh)
    desc = _norm_desc(h, weight, 0.0, False)
    _full("dy", dy, h.shape, h.dtype)
    _full("rstd", rstd, h.shape[:-1], torch.float32)
    if dh is not None:
        _full("dh", dh, h.shape, h.dtype)
    dx = torch.empty_like(h)
    dweight = torch.empty_like(weight)
    ws, n = _workspace("e2ttt_norm_backward_workspace_size", desc, workspace, h.device)
    st = _lib.load().e2ttt_norm_backward(ctypes.byref(desc), _p(dy), _p(h), _p(weight), _p(rstd), _p(dh), _p(dx),
                                         _p(dweight), _p(ws), n, _stream(stream))
    if st != 0:
        raise E2TTTError("e2ttt_norm_backward", st)
    return dx, dweight


class _Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, weight, eps):
        y, _, h, rstd = norm_forward(x, weight, residual=residual, eps=eps)
        ctx.save_for_backward(h, weight, rstd)
        ctx.has_residual = residual is not None
        ctx.set_materialize_grads(False)
        return (y, h) if ctx.has_residual else (y,)

    @staticmethod
    def backward(ctx, dy, dh=None):
        h, weight, rstd = ctx.saved_tensors
        dy = torch.zeros_like(h) if dy is None else dy
        dx, dweight = norm_backward(dy.contiguous(), h, weight, rstd, dh=None if dh is None else dh.contiguous())
        return dx, (dx if ctx.has_residual else None), dweight, None


def rms_norm(x, weight, residual=None, *, eps: float = 1e-6):
    """``norm_forward`` as a differentiable op: returns (y, h), h = x + residual
    (x itself without ``residual``), with gradients for x, weight and residual."""
    if residual is None:
        return _Norm.apply(x, None, weight, eps)[0], x
    return _Norm.apply(x, residual, weight, eps)
