"""The operators of a hybrid layer beside the chunk update: Python binding of
include/e2ttt_layer.h.

Argument marshalling only, as in the package's ``__init__``: the work runs in
the HIP kernels behind the C ABI on the current stream, with tensors that the
caller owns; outputs and workspaces that are not given are allocated through
torch.  With ``stream``, one of the tensors' device, the call runs as under
``torch.cuda.stream(stream)``: what it allocates belongs to that stream, so that
no other work reuses a workspace before the kernels are done with it.  CPU
tensors raise.
"""
from __future__ import annotations

import ctypes
from functools import lru_cache

import torch
from torch.autograd.function import once_differentiable

from . import _lib
from ._lib import SCAN_TILE, AttentionDesc, E2TTTError, NormDesc, PagedDesc, ScanDesc

_IO = {torch.float32: 0, torch.bfloat16: 1}
_BAD = ctypes.c_size_t(-1).value
F8 = torch.float8_e4m3fn
E8 = torch.float8_e8m0fnu
_functions: dict = {}


def _device(first, **others) -> int:
    """The one GPU that every tensor is on."""
    dev = first.get_device()
    if dev < 0:
        raise ValueError("tensors must be on a GPU (no CPU path exists)")
    for name, t in others.items():
        if t is not None and t.get_device() != dev:
            raise ValueError(f"{name} must be a GPU tensor on the same device as the others")
    return dev


def _on(stream, first):
    """The context of a stream of the tensors' device."""
    if stream.device.index != _device(first):
        raise ValueError(f"stream must be on the tensors' device {first.device}, not {stream.device}")
    return torch.cuda.stream(stream)


def _call(fn: str, dev: int, *args):
    """Calls the library on the current stream of the tensors' device, which is
    made current for the call if it is not."""
    if dev != torch._C._cuda_getDevice():
        with torch.cuda.device(dev):
            return _call(fn, dev, *args)
    f = _functions.get(fn)
    if f is None:
        f = _functions[fn] = getattr(_lib.load(), fn)
    st = f(*args, torch._C._cuda_getCurrentRawStream(dev))
    if st != 0:
        raise E2TTTError(fn, st)


def _leaves(nodes):
    """Those that stand for leaves: one node per leaf, as long as a graph holds it."""
    return [node for node in nodes if node is not None and node.name() == "torch::autograd::AccumulateGrad"]


def _before(node):
    return [n for n, _ in node.next_functions]


def _mark_leaves(out, dev: int):
    """Notes at each leaf that the call behind ``out`` was given the stream of the first such
    call in a graph that is still alive."""
    if out.grad_fn is not None:
        stream = torch._C._cuda_getCurrentRawStream(dev)
        for leaf in _leaves(_before(out.grad_fn)):
            leaf.metadata.setdefault("e2ttt_stream", stream)


def _refuse_other_streams(leaves, dev: int):
    stream = torch._C._cuda_getCurrentRawStream(dev)
    if any(leaf.metadata.get("e2ttt_stream", stream) != stream for leaf in leaves):
        raise RuntimeError("a leaf of this capture is in an autograd graph of another stream: "
                           "drop that graph's outputs first")


def _one_stream(out, dev: int):
    """Refuses a capture with gradients for leaves that an eager graph, still alive, used on
    another stream: the backward pass ends by making that stream wait, which a capture does
    not survive (the process ends in it).  The leaves that the call behind ``out`` was given."""
    _mark_leaves(out, dev)
    if out.grad_fn is not None and torch.cuda.is_current_stream_capturing():
        _refuse_other_streams(_leaves(_before(out.grad_fn)), dev)


def _one_stream_behind(out, dev: int):
    """``_one_stream`` for all leaves behind ``out``; the streams are known of those that a call
    of this package was given directly."""
    _one_stream(out, dev)
    if out.grad_fn is None or not torch.cuda.is_current_stream_capturing():
        return
    todo, seen = [out.grad_fn], {out.grad_fn}
    while todo:
        new = {node for node in _before(todo.pop()) if node is not None} - seen
        seen |= new
        todo += new
    _refuse_other_streams(_leaves(seen), dev)


def _p(t):
    return None if t is None else t.data_ptr()


def _heads3(name, shape, stride, dtype, N, D, want):
    """Checks a [tokens, heads, D] tensor whose last dimension is contiguous."""
    if len(shape) != 3 or shape[0] != N or shape[2] != D:
        raise ValueError(f"{name} must have shape ({N}, heads, {D}), got {tuple(shape)}")
    if dtype != want:
        raise TypeError(f"{name} must be {want}")
    if D > 1 and stride[2] != 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")


def _int32(name, t, shape):
    if t.dtype != torch.int32 or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor of shape {tuple(shape)}")


def _full(name, t, shape, dtype):
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _size(fn, desc):
    """Workspace bytes, 0 for a descriptor that the call itself will refuse."""
    n = getattr(_lib.load(), fn)(ctypes.byref(desc))
    return 0 if n == _BAD else n


def _layout(t):
    return None if t is None else (t.shape, t.stride(), t.dtype)


# Descriptors and workspace sizes by shapes, strides and types alone, so that a
# step of a serving loop builds and checks them once.
@lru_cache(maxsize=512)
def _attention_desc(q, k, v, cu, window, scale, kv_heads):
    shape, stride, dtype = q
    if len(shape) != 3:
        raise ValueError(f"q must have shape (tokens, heads, D), got {tuple(shape)}")
    N, H, D = shape
    if dtype not in _IO:
        raise TypeError(f"expected float32 or bfloat16, got {dtype}")
    _heads3("q", *q, N, D, dtype)
    ks = vs = (0, 0)
    if k is not None:
        _heads3("k", *k, N, D, dtype)
        _heads3("v", *v, N, D, dtype)
        if kv_heads is None:
            kv_heads = k[0][1]
        if k[0][1] != kv_heads or v[0][1] != kv_heads:
            raise ValueError(f"k and v must both have {kv_heads} heads")
        ks, vs = k[1], v[1]
    if len(cu[0]) != 1 or cu[0][0] < 1 or cu[2] != torch.int32 or (cu[0][0] > 1 and cu[1][0] != 1):
        raise ValueError("cu_seqlens must be a contiguous int32 tensor of shape (sequences + 1,)")
    if scale is None:
        scale = D ** -0.5 if D else 1.0
    # ctypes would take a larger number's low 32 bits; one as long as any sequence leaves none out
    window = max(-1, min(window, 0x7fffffff))
    return AttentionDesc(_IO[dtype], window, N, cu[0][0] - 1, H, kv_heads, D, scale, 0, stride[0], stride[1],
                         ks[0], ks[1], vs[0], vs[1])


@lru_cache(maxsize=512)
def _attention_plan(q, k, v, cu, window, scale):
    d = _attention_desc(q, k, v, cu, window, scale, None)
    return (tuple(q[0]), ctypes.byref(d), _size("e2ttt_attention_workspace_size", d),
            _size("e2ttt_attention_backward_workspace_size", d), d)


@lru_cache(maxsize=512)
def _paged_plan(q, k, v, kc, vc, table, cu, window, scale, bits8):
    if len(kc[0]) != 4 or kc[0] != vc[0]:
        raise ValueError("k_cache and v_cache must share one shape (pages, K, page_size, D)")
    P, K, ps, D = kc[0]
    want = F8 if bits8 else q[2]
    if kc[2] != want or vc[2] != want:
        raise TypeError(f"k_cache and v_cache must be {want}")
    a = _attention_desc(q, k, v, cu, window, scale, K)
    if a.D != D or (D > 1 and (kc[1][3] != 1 or vc[1][3] != 1)):
        raise ValueError(f"k_cache and v_cache must have a contiguous last dimension of {a.D}")
    if len(table[0]) != 2:
        raise ValueError("table must have shape (sequences, width)")
    s, t = kc[1], vc[1]
    d = PagedDesc(a, P, ps, table[0][1], s[0], s[1], s[2], t[0], t[1], t[2])
    return tuple(q[0]), ctypes.byref(d), _size("e2ttt_paged8_workspace_size" if bits8 else "e2ttt_paged_workspace_size", d), d


@lru_cache(maxsize=512)
def _norm_plan(shape, dtype, eps, bits8):
    if len(shape) < 1:
        raise ValueError("x must have shape (..., width)")
    if dtype not in _IO:
        raise TypeError(f"expected float32 or bfloat16, got {dtype}")
    rows = 1
    for n in shape[:-1]:
        rows *= n
    d = NormDesc(_IO[dtype], int(bits8), rows, shape[-1], eps, 0)
    return tuple(shape[:-1]), ctypes.byref(d), _size("e2ttt_norm_backward_workspace_size", d), d


@lru_cache(maxsize=512)
def _scan_plan(x, a, cu):
    shape, stride, dtype = x
    if len(shape) != 2:
        raise ValueError(f"x must have shape (tokens, width), got {tuple(shape)}")
    if dtype not in _IO:
        raise TypeError(f"expected float32 or bfloat16, got {dtype}")
    if a[0] != shape:
        raise ValueError(f"a must have shape {tuple(shape)}")
    if a[2] != torch.float32 and a[2] != dtype:
        raise TypeError(f"a must be float32 or {dtype}")
    if shape[1] > 1 and (stride[1] != 1 or a[1][1] != 1):
        raise ValueError("x's and a's last dimension must be contiguous")
    if len(cu[0]) != 1 or cu[0][0] < 1 or cu[2] != torch.int32 or (cu[0][0] > 1 and cu[1][0] != 1):
        raise ValueError("cu_seqlens must be a contiguous int32 tensor of shape (sequences + 1,)")
    N, C = shape
    d = ScanDesc(_IO[dtype], _IO[a[2]], N, cu[0][0] - 1, C, stride[0], a[1][0])
    return (N, C, cu[0][0] - 1, ctypes.byref(d), _size("e2ttt_scan_workspace_size", d),
            _size("e2ttt_scan_backward_workspace_size", d), d)


def _row_values(lead, x):
    if len(lead) == 1:  # sizes as numbers of their own are quicker than a tuple
        return torch.empty(lead[0], dtype=torch.float32, device=x.device)
    return torch.empty(lead, dtype=torch.float32, device=x.device)


def _workspace(workspace, n, like):
    if workspace is None:
        if n == 0:
            return None, 0
        workspace = torch.empty(n, dtype=torch.uint8, device=like.device)
    elif workspace.get_device() != like.get_device():
        raise ValueError("workspace must be a GPU tensor on the same device as the others")
    elif not workspace.is_contiguous():  # an expanded one has fewer bytes than elements
        raise ValueError("workspace must be contiguous")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def attention_forward(q, k, v, cu_seqlens, *, window: int = 0, scale: float | None = None, out=None, lse=None,
                      workspace=None, stream=None):
    """Causal attention over packed sequences; returns (out, lse).

    q: [N, H, D], k, v: [N, K, D], float32 or bfloat16, last dimension
    contiguous (views of one projection's output are fine); H a multiple of K,
    D a multiple of 8 up to 128.  cu_seqlens: [S + 1] int32 on the GPU, the
    sequences' offsets into the N tokens; tokens before the first or from the
    last on belong to no sequence: out and their gradients are 0, lse
    -infinity.  ``window`` > 0: a query sees that
    many positions, its own the last.  ``scale``: of the scores, D ** -0.5 by
    default.  out: [N, H, D]; lse: [N, H] float32, the log of each row's
    softmax sum, which the backward needs.
    """
    if stream is not None:
        with _on(stream, q):
            return attention_forward(q, k, v, cu_seqlens, window=window, scale=scale, out=out, lse=lse, workspace=workspace)
    dev = _device(q, k=k, v=v, cu_seqlens=cu_seqlens, out=out, lse=lse)
    (N, H, D), desc, need, _, _ = _attention_plan(_layout(q), _layout(k), _layout(v), _layout(cu_seqlens), window, scale)
    if out is None:
        out = torch.empty(N, H, D, dtype=q.dtype, device=q.device)
    else:
        _full("out", out, (N, H, D), q.dtype)
    if lse is None:
        lse = torch.empty(N, H, dtype=torch.float32, device=q.device)
    else:
        _full("lse", lse, (N, H), torch.float32)
    if cu_seqlens.shape[0] == 1:  # no sequences, no launch
        return out.zero_(), lse.fill_(float("-inf"))
    ws, n = _workspace(workspace, need, q)
    _call("e2ttt_attention_forward", dev, desc, q.data_ptr(), k.data_ptr(), v.data_ptr(),
          cu_seqlens.data_ptr(), out.data_ptr(), lse.data_ptr(), ws, n)
    return out, lse


def attention_backward(q, k, v, out, lse, dout, cu_seqlens, *, window: int = 0, scale: float | None = None,
                       workspace=None, stream=None):
    """Gradients of <dout, out> through ``attention_forward``, from its inputs
    and outputs; returns a dict with keys q, k, v (the I/O dtype, contiguous)."""
    if stream is not None:
        with _on(stream, q):
            return attention_backward(q, k, v, out, lse, dout, cu_seqlens, window=window, scale=scale,
                                      workspace=workspace)
    dev = _device(q, k=k, v=v, out=out, lse=lse, dout=dout, cu_seqlens=cu_seqlens)
    (N, H, D), desc, _, need, _ = _attention_plan(_layout(q), _layout(k), _layout(v), _layout(cu_seqlens), window, scale)
    _full("out", out, (N, H, D), q.dtype)
    _full("dout", dout, (N, H, D), q.dtype)
    _full("lse", lse, (N, H), torch.float32)
    g = {n: torch.empty(t.shape, dtype=q.dtype, device=q.device) for n, t in (("q", q), ("k", k), ("v", v))}
    if cu_seqlens.shape[0] == 1:  # as in the forward
        return {n: t.zero_() for n, t in g.items()}
    ws, n = _workspace(workspace, need, q)
    _call("e2ttt_attention_backward", dev, desc, q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
          lse.data_ptr(), dout.data_ptr(), cu_seqlens.data_ptr(), g["q"].data_ptr(), g["k"].data_ptr(),
          g["v"].data_ptr(), ws, n)
    return g


class _Attention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, cu_seqlens, window, scale):
        out, lse = attention_forward(q, k, v, cu_seqlens, window=window, scale=scale)
        ctx.save_for_backward(q, k, v, out, lse, cu_seqlens)
        ctx.opts = (window, scale)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        q, k, v, out, lse, cu_seqlens = ctx.saved_tensors
        window, scale = ctx.opts
        g = attention_backward(q, k, v, out, lse, dout.contiguous(), cu_seqlens, window=window, scale=scale)
        return g["q"], g["k"], g["v"], None, None, None


def attention(q, k, v, cu_seqlens, *, window: int = 0, scale: float | None = None):
    """``attention_forward`` as a differentiable op: returns out, with gradients
    for q, k and v from ``attention_backward``."""
    out = _Attention.apply(q, k, v, cu_seqlens, window, scale)
    _mark_leaves(out, q.get_device())
    return out


def paged_attention(q, k, v, k_cache, v_cache, table, cu_seqlens, cached, *, window: int = 0,
                    scale: float | None = None, k_scale=None, v_scale=None, out=None, workspace=None, stream=None):
    """Attention of each sequence's new tokens over its cached ones and
    themselves; writes the new keys and values into the cache; returns out.

    q: [N, H, D], k, v: [N, K, D]: the new tokens of all sequences, packed by
    cu_seqlens [S + 1] int32 (one each: plain decoding; more: a chunk of a
    prompt).  k_cache, v_cache: [pages, K, page_size, D], page_size a power of
    two (any strides with a contiguous last dimension).  table: [S, W] int32,
    the pages of each sequence; cached: [S] int32, its tokens in the cache
    before the call.  New token i of sequence s is at position cached[s] + i.
    Tokens before the first offset or from the last on belong to no sequence:
    their out is 0, their k and v go nowhere.
    With k = v = None the cache holds the new tokens already.

    With k_scale and v_scale, [pages, K, page_size] float8_e8m0fnu, contiguous, the
    cache is in 8 bits (float8_e4m3fn, D a multiple of 16; q, k, v bfloat16): a key
    or value is its row of the cache times its scale, a power of two.  New ones are
    rounded into it, with the smallest scale that brings their largest magnitude to
    448, and queries see them as the cache holds them; one with a NaN or an Inf in
    it becomes NaN as a whole.
    """
    if stream is not None:
        with _on(stream, q):
            return paged_attention(q, k, v, k_cache, v_cache, table, cu_seqlens, cached, window=window, scale=scale,
                                   k_scale=k_scale, v_scale=v_scale, out=out, workspace=workspace)
    if (k is None) != (v is None):
        raise ValueError("k and v must both be given, or neither")
    bits8 = k_scale is not None
    if bits8 != (v_scale is not None):
        raise ValueError("k_scale and v_scale must both be given, or neither")
    dev = _device(q, k=k, v=v, k_cache=k_cache, v_cache=v_cache, table=table, cu_seqlens=cu_seqlens, cached=cached,
                  out=out, k_scale=k_scale, v_scale=v_scale)
    (N, H, D), desc, need, _ = _paged_plan(_layout(q), _layout(k), _layout(v), _layout(k_cache), _layout(v_cache),
                                           _layout(table), _layout(cu_seqlens), window, scale, bits8)
    if bits8:
        _full("k_scale", k_scale, k_cache.shape[:3], E8)
        _full("v_scale", v_scale, k_cache.shape[:3], E8)
    S = cu_seqlens.shape[0] - 1
    _int32("table", table, (S, table.shape[1]))
    _int32("cached", cached, (S,))
    if out is None:
        out = torch.empty(N, H, D, dtype=q.dtype, device=q.device)
    else:
        _full("out", out, (N, H, D), q.dtype)
    if S == 0:  # no sequences, no launch
        return out.zero_()
    ws, n = _workspace(workspace, need, q)
    if bits8:
        _call("e2ttt_paged8_attention", dev, desc, q.data_ptr(), _p(k), _p(v), k_cache.data_ptr(), v_cache.data_ptr(),
              k_scale.data_ptr(), v_scale.data_ptr(), table.data_ptr(), cu_seqlens.data_ptr(), cached.data_ptr(),
              out.data_ptr(), ws, n)
        return out
    _call("e2ttt_paged_attention", dev, desc, q.data_ptr(), _p(k), _p(v), k_cache.data_ptr(),
          v_cache.data_ptr(), table.data_ptr(), cu_seqlens.data_ptr(), cached.data_ptr(), out.data_ptr(), ws, n)
    return out


def gated_scan_forward(x, a, cu_seqlens, *, h0=None, out=None, state=None, save: bool = False, workspace=None, stream=None):
    """Gated linear recurrence h_t = a_t h_{t-1} + x_t of every channel over
    packed sequences; returns (out, state, starts).

    x: [N, C] float32 or bfloat16, a: [N, C] in x's type or float32, gates of
    magnitude up to 1; last dimension contiguous (views of a projection's output
    are fine).  cu_seqlens: [S + 1] int32, as for ``attention_forward``; tokens of
    no sequence give 0.  h0: [S, C] float32, the state before each sequence (None:
    0).  out: [N, C], every h_t in x's type; state: [S, C] float32, the last one of
    each sequence (h0 for an empty one; ``state=h0`` updates it in place).  With
    sequences of one token each this is the step of a serving loop.  ``save``
    also gives starts, the states that ``gated_scan_backward`` begins from
    (else None).
    """
    if stream is not None:
        with _on(stream, x):
            return gated_scan_forward(x, a, cu_seqlens, h0=h0, out=out, state=state, save=save, workspace=workspace)
    dev = _device(x, a=a, cu_seqlens=cu_seqlens, h0=h0, out=out, state=state)
    N, C, S, desc, need, _, _ = _scan_plan(_layout(x), _layout(a), _layout(cu_seqlens))
    if h0 is not None:
        _full("h0", h0, (S, C), torch.float32)
    if out is None:
        out = torch.empty(N, C, dtype=x.dtype, device=x.device)
    else:
        _full("out", out, (N, C), x.dtype)
    if state is None:
        state = torch.empty(S, C, dtype=torch.float32, device=x.device)
    else:
        _full("state", state, (S, C), torch.float32)
    starts = torch.empty(N // SCAN_TILE + S, C, dtype=torch.float32, device=x.device) if save else None
    if S == 0:  # no sequences, no launch
        return out.zero_(), state, starts
    ws, n = _workspace(workspace, need, x)
    _call("e2ttt_scan_forward", dev, desc, x.data_ptr(), a.data_ptr(), _p(h0), cu_seqlens.data_ptr(), out.data_ptr(),
          state.data_ptr(), _p(starts), ws, n)
    return out, state, starts


def gated_scan_backward(dout, x, a, starts, cu_seqlens, *, dstate=None, workspace=None, stream=None):
    """Gradients of <dout, out> + <dstate, state> through ``gated_scan_forward``,
    from its inputs and starts; returns a dict with keys x and a (contiguous, in
    their types) and h0 ([S, C] float32)."""
    if stream is not None:
        with _on(stream, x):
            return gated_scan_backward(dout, x, a, starts, cu_seqlens, dstate=dstate, workspace=workspace)
    dev = _device(x, a=a, dout=dout, starts=starts, cu_seqlens=cu_seqlens, dstate=dstate)
    N, C, S, desc, _, need, _ = _scan_plan(_layout(x), _layout(a), _layout(cu_seqlens))
    _full("dout", dout, (N, C), x.dtype)
    _full("starts", starts, (N // SCAN_TILE + S, C), torch.float32)
    if dstate is not None:
        _full("dstate", dstate, (S, C), torch.float32)
    g = {"x": torch.empty(N, C, dtype=x.dtype, device=x.device), "a": torch.empty(N, C, dtype=a.dtype, device=x.device),
         "h0": torch.empty(S, C, dtype=torch.float32, device=x.device)}
    if S == 0:  # as in the forward
        return {n: t.zero_() for n, t in g.items()}
    ws, n = _workspace(workspace, need, x)
    _call("e2ttt_scan_backward", dev, desc, dout.data_ptr(), x.data_ptr(), a.data_ptr(), starts.data_ptr(), _p(dstate),
          cu_seqlens.data_ptr(), g["x"].data_ptr(), g["a"].data_ptr(), g["h0"].data_ptr(), ws, n)
    return g


class _GatedScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, a, h0, cu_seqlens):
        out, state, starts = gated_scan_forward(x, a, cu_seqlens, h0=h0, save=True)
        ctx.save_for_backward(x, a, starts, cu_seqlens)
        ctx.set_materialize_grads(False)
        return out, state

    @staticmethod
    @once_differentiable
    def backward(ctx, dout, dstate):
        x, a, starts, cu_seqlens = ctx.saved_tensors
        dout = torch.zeros(x.shape, dtype=x.dtype, device=x.device) if dout is None else dout.contiguous()
        g = gated_scan_backward(dout, x, a, starts, cu_seqlens, dstate=None if dstate is None else dstate.contiguous())
        return g["x"], g["a"], (g["h0"] if ctx.needs_input_grad[2] else None), None


def gated_scan(x, a, cu_seqlens, h0=None):
    """``gated_scan_forward`` as a differentiable op: returns (out, state), with
    gradients for x, a and h0 from ``gated_scan_backward``.  Captured into a graph with its
    backward pass, no eager graph of the same leaves may be alive (RuntimeError, where one of
    the leaves was given to a call of this package directly)."""
    out, state = _GatedScan.apply(x, a, h0, cu_seqlens)
    _one_stream_behind(out, x.get_device())
    return out, state


def norm_forward(x, weight, *, residual=None, eps: float = 1e-6, bits8: bool = False, h=None, stream=None):
    """Root-mean-square norm with the residual's addition; returns
    (y, scale, h, rstd).

    x: [..., W] float32 or bfloat16, contiguous; weight: [W] float32.
    h = x + residual in x's type (x itself without ``residual``; ``h=residual``
    updates the stream in place); rstd: [...] float32, for the backward (None
    with ``bits8``, which has none).  y = h * rstd * weight in x's type, or with
    ``bits8`` in float8_e4m3fn, to be multiplied by scale [...] (float32,
    max|y| / 448 of its row; else None).
    """
    if stream is not None:
        with _on(stream, x):
            return norm_forward(x, weight, residual=residual, eps=eps, bits8=bits8, h=h)
    dev = _device(x, weight=weight, residual=residual, h=h)
    lead, desc, _, _ = _norm_plan(x.shape, x.dtype, eps, bits8)
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    _full("weight", weight, x.shape[-1:], torch.float32)
    if residual is not None:
        _full("residual", residual, x.shape, x.dtype)
        if h is None:
            h = torch.empty_like(x)
        else:
            _full("h", h, x.shape, x.dtype)
    elif h is not None:
        raise ValueError("h is an output of the residual's addition: give residual too")
    scale = rstd = None
    if bits8:
        y = torch.empty_like(x, dtype=F8)
        scale = _row_values(lead, x)
    else:
        y = torch.empty_like(x)
        rstd = _row_values(lead, x)
    _call("e2ttt_norm_forward", dev, desc, x.data_ptr(), _p(residual), weight.data_ptr(), y.data_ptr(),
          _p(scale), _p(h), _p(rstd))
    return y, scale, (x if residual is None else h), rstd


def norm_backward(dy, h, weight, rstd, *, dh=None, workspace=None, stream=None):
    """Gradients through ``norm_forward`` (y in the stream's type): returns
    (dx, dweight).  dx is the gradient of both x and residual; ``dh`` is what
    arrives at h along the residual stream, added to it."""
    if stream is not None:
        with _on(stream, dy):
            return norm_backward(dy, h, weight, rstd, dh=dh, workspace=workspace)
    dev = _device(h, dy=dy, weight=weight, rstd=rstd, dh=dh)
    lead, desc, need, _ = _norm_plan(h.shape, h.dtype, 0.0, False)
    _full("h", h, h.shape, h.dtype)
    _full("weight", weight, h.shape[-1:], torch.float32)
    _full("dy", dy, h.shape, h.dtype)
    _full("rstd", rstd, lead, torch.float32)
    if dh is not None:
        _full("dh", dh, h.shape, h.dtype)
    dx = torch.empty_like(h)
    dweight = torch.empty_like(weight)
    ws, n = _workspace(workspace, need, h)
    _call("e2ttt_norm_backward", dev, desc, dy.data_ptr(), h.data_ptr(), weight.data_ptr(), rstd.data_ptr(),
          _p(dh), dx.data_ptr(), dweight.data_ptr(), ws, n)
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
    @once_differentiable
    def backward(ctx, dy, dh=None):
        h, weight, rstd = ctx.saved_tensors
        dy = torch.zeros_like(h) if dy is None else dy
        dx, dweight = norm_backward(dy.contiguous(), h, weight, rstd, dh=None if dh is None else dh.contiguous())
        return dx, (dx if ctx.has_residual else None), dweight, None


def rms_norm(x, weight, residual=None, *, eps: float = 1e-6):
    """``norm_forward`` as a differentiable op: returns (y, h), h = x + residual
    (x itself without ``residual``), with gradients for x, weight and residual."""
    y, h = (_Norm.apply(x, None, weight, eps)[0], x) if residual is None else _Norm.apply(x, residual, weight, eps)
    _mark_leaves(y, x.get_device())
    return y, h
