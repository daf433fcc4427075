"""Host-side checks of include/e2ttt_layer.h: the library exports what the
header declares, and every refusal happens before any device call (no GPU
needed; the pointers here are never read)."""
import ctypes
import os
import re

import pytest
import torch

from chunk_weight_rnn_amd import _lib as L

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BASE = 1 << 40
GAP = 1 << 36
BAD = ctypes.c_size_t(-1).value
OK, INVALID, UNSUPPORTED, ALIAS, WORKSPACE = 0, 1, 2, 3, 4


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(L.LIB_PATH):
        from chunk_weight_rnn_amd import build
        build.build()
    return L.load()


def attn(N=1000, S=2, H=8, K=2, D=128, dtype=1, window=0, scale=0.1, **kw):
    d = L.AttentionDesc(dtype, window, N, S, H, K, D, scale, 0, H * D, D, K * D, D, K * D, D)
    for n, v in kw.items():
        setattr(d, n, v)
    return d


def ptrs(n):
    return [BASE + i * GAP for i in range(n)]


def fwd(lib, d, p=None, ws=None, n=1 << 40):
    """Statuses before the launch only: a call that would launch is not made here."""
    p = ptrs(6) if p is None else p
    return lib.e2ttt_attention_forward(ctypes.byref(d), *p, ws, n, None)


def test_exports(lib):
    text = open(os.path.join(ROOT, "include", "e2ttt_layer.h")).read()
    names = set(re.findall(r"E2TTT_API[^;(]*?\b(e2ttt_\w+)\s*\(", text))
    assert names == set(L.LAYER_EXPORTS)
    assert not names & set(L.EXPORTS)
    for n in names:
        assert hasattr(lib, n), n


def test_desc_sizes_match_the_header(tmp_path):
    """The ctypes structs are laid out as the C compiler lays out the header's."""
    import shutil
    import subprocess
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "e2ttt_layer.h"\nint main(void){printf("%zu %zu %zu %zu %zu %zu\\n",'
                   'sizeof(e2ttt_attention_desc),sizeof(e2ttt_paged_desc),sizeof(e2ttt_norm_desc),'
                   'offsetof(e2ttt_attention_desc,q_tok),offsetof(e2ttt_paged_desc,kc_page),offsetof(e2ttt_norm_desc,eps));return 0;}')
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(tmp_path / "s")], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "s")], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(L.AttentionDesc), ctypes.sizeof(L.PagedDesc), ctypes.sizeof(L.NormDesc),
                   L.AttentionDesc.q_tok.offset, L.PagedDesc.kc_page.offset, L.NormDesc.eps.offset]


@pytest.mark.parametrize("field,value", [("io_dtype", 2), ("window", -1), ("tokens", -1), ("seqs", -1), ("heads", 0),
                                         ("kv_heads", 0), ("kv_heads", 3), ("D", 0), ("scale", 0.0), ("scale", -1.0),
                                         ("scale", float("inf")), ("scale", float("nan")), ("reserved", 1),
                                         ("q_tok", 4), ("k_head", 12), ("v_tok", -8), ("k_tok", 64)])
def test_attention_bad_desc(lib, field, value):
    d = attn(**{field: value})
    assert fwd(lib, d) == INVALID
    assert lib.e2ttt_attention_workspace_size(ctypes.byref(d)) == BAD
    assert lib.e2ttt_attention_backward_workspace_size(ctypes.byref(d)) == BAD


@pytest.mark.parametrize("kw", [dict(D=4), dict(D=136), dict(D=100), dict(N=1 << 31), dict(N=(1 << 28)),
                                dict(N=1 << 24, H=64, K=1), dict(S=1 << 28), dict(k_tok=(1 << 23) + 8)])
def test_attention_unsupported(lib, kw):
    d = attn(**kw)
    assert fwd(lib, d) == UNSUPPORTED
    assert lib.e2ttt_attention_workspace_size(ctypes.byref(d)) == BAD


def test_attention_pointers(lib):
    for i in range(5):  # lse may be null
        p = ptrs(6)
        p[i] = 0
        assert fwd(lib, attn(), p) == INVALID, i
        p[i] = BASE + i * GAP + 2
        assert fwd(lib, attn(), p) == INVALID, i
    assert fwd(lib, attn(), [0] * 6) == INVALID
    assert fwd(lib, attn(N=0), [0] * 6) == OK  # nothing to do
    assert fwd(lib, attn(S=0), [0] * 6) == OK


def test_attention_workspace(lib):
    d = attn(N=300, S=1, H=2, K=1)  # few row tiles: keys are split, partial results need room
    need = lib.e2ttt_attention_workspace_size(ctypes.byref(d))
    assert 0 < need < 1 << 24
    assert fwd(lib, d, ws=None) == WORKSPACE
    assert fwd(lib, d, ws=BASE + 7 * GAP, n=need - 1) == WORKSPACE
    assert fwd(lib, d, ws=BASE + 7 * GAP + 16, n=need) == WORKSPACE
    assert lib.e2ttt_attention_workspace_size(ctypes.byref(attn(N=1 << 16))) == 0
    b = lambda ws, n: lib.e2ttt_attention_backward(ctypes.byref(d), *ptrs(10), ws, n, None)
    need = lib.e2ttt_attention_backward_workspace_size(ctypes.byref(d))
    assert need >= 300 * 2 * 4
    assert b(None, 0) == WORKSPACE and b(BASE + 12 * GAP, need - 1) == WORKSPACE


def test_attention_aliasing(lib):
    d = attn(N=1 << 16)
    for i in range(4):
        p = ptrs(6)
        p[4] = p[i] + (0 if i < 3 else -64)  # out over q, k, v or the offsets
        assert fwd(lib, d, p) == ALIAS, i
    p = ptrs(6)
    p[5] = p[4] + 64  # lse inside out
    assert fwd(lib, d, p) == ALIAS
    need = lib.e2ttt_attention_backward_workspace_size(ctypes.byref(d))
    names = ptrs(10)
    for o in (7, 8, 9):
        for i in range(10):
            if i == o:
                continue
            p = list(names)
            p[o] = p[i]
            assert lib.e2ttt_attention_backward(ctypes.byref(d), *p, BASE + 12 * GAP, need, None) == ALIAS, (o, i)


def paged(P=100, ps=16, W=32, **kw):
    a = attn(N=4, S=4, **kw)
    K, D = a.kv_heads, a.D
    return L.PagedDesc(a, P, ps, W, K * ps * D, ps * D, D, K * ps * D, ps * D, D)


def page_call(lib, d, p=None, ws=BASE + 20 * GAP, n=1 << 40):
    return lib.e2ttt_paged_attention(ctypes.byref(d), *(ptrs(9) if p is None else p), ws, n, None)


@pytest.mark.parametrize("field,value", [("page_size", 0), ("page_size", 24), ("pages", -1), ("table_width", -1),
                                         ("kc_slot", 4), ("vc_head", 64), ("kc_page", -8), ("vc_slot", 0)])
def test_paged_bad_desc(lib, field, value):
    d = paged()
    setattr(d, field, value)
    assert page_call(lib, d) == INVALID
    assert lib.e2ttt_paged_workspace_size(ctypes.byref(d)) == BAD


def test_paged_refusals(lib):
    assert page_call(lib, paged(D=20)) == UNSUPPORTED
    assert page_call(lib, paged(W=1 << 28)) == UNSUPPORTED
    d = paged()
    for i in range(9):  # q, k, v, k_cache, v_cache, table, cu, cached, out
        p = ptrs(9)
        p[i] = 0
        assert page_call(lib, d, p) == INVALID, i  # k without v among them
    p = ptrs(9)
    p[8] = p[3] + 4096
    assert page_call(lib, d, p) == ALIAS  # out inside the cache
    p = ptrs(9)
    p[1] = p[4] + 4096
    assert page_call(lib, d, p) == ALIAS  # the new keys inside the cache
    d = paged(W=4096)
    assert lib.e2ttt_paged_workspace_size(ctypes.byref(d)) > 0
    assert page_call(lib, d, ws=None) == WORKSPACE
    d = paged()
    d.a.tokens = 0
    assert page_call(lib, d, [0] * 9) == OK


def norm(rows=10, W=64, dtype=1, bits8=0, eps=1e-6, **kw):
    d = L.NormDesc(dtype, bits8, rows, W, eps, 0)
    for n, v in kw.items():
        setattr(d, n, v)
    return d


def norm_call(lib, d, p=None):
    p = ptrs(7) if p is None else p  # x, residual, weight, y, scale, h, rstd
    if not d.bits8 and p[4] == BASE + 4 * GAP:
        p = p[:4] + [0] + p[5:]
    return lib.e2ttt_norm_forward(ctypes.byref(d), *p, None)


@pytest.mark.parametrize("field,value", [("io_dtype", -1), ("bits8", 2), ("rows", -1), ("width", 0), ("eps", -1.0),
                                         ("eps", float("nan")), ("reserved", 3)])
def test_norm_bad_desc(lib, field, value):
    d = norm(**{field: value})
    assert norm_call(lib, d) == INVALID
    assert lib.e2ttt_norm_backward_workspace_size(ctypes.byref(d)) == BAD


def test_norm_refusals(lib):
    assert norm_call(lib, norm(W=65537)) == UNSUPPORTED
    assert norm_call(lib, norm(rows=0), [0] * 7) == OK
    for i in (0, 1, 2, 3, 5):
        p = ptrs(7)
        p[i] = 0
        assert norm_call(lib, norm(), p) == INVALID, i  # a residual without h, and h without one, among them
    p = ptrs(7)
    p[4] = 0
    assert norm_call(lib, norm(bits8=1), p) == INVALID
    assert lib.e2ttt_norm_forward(ctypes.byref(norm()), *ptrs(7), None) == INVALID  # scale without bits8
    for o, i in ((3, 0), (3, 1), (3, 2), (6, 0), (5, 3)):
        p = ptrs(7)
        p[o] = p[i]
        assert norm_call(lib, norm(), p) == ALIAS, (o, i)
    p = ptrs(7)
    p[5] = p[0] + 64  # h partly over x
    assert norm_call(lib, norm(), p) == ALIAS
    b = lambda p, ws=BASE + 20 * GAP, n=1 << 40, d=norm(): lib.e2ttt_norm_backward(ctypes.byref(d), *p, ws, n, None)
    names = ptrs(7)  # dy, h, weight, rstd, dh, dx, dweight
    assert b(names, ws=None) == WORKSPACE
    assert b(names, d=norm(bits8=1)) == INVALID
    for o in (5, 6):
        for i in range(4):
            p = list(names)
            p[o] = p[i]
            assert b(p) == ALIAS, (o, i)
    p = list(names)
    p[5] = p[4] + 32
    assert b(p) == ALIAS


def test_python_refuses_what_is_not_on_a_gpu_or_does_not_fit():
    import chunk_weight_rnn_amd as e2
    q = torch.zeros(4, 4, 64)
    k = torch.zeros(4, 2, 64)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        e2.attention_forward(q, k, k, cu)
    with pytest.raises(ValueError, match="GPU"):
        e2.norm_forward(q, torch.ones(64))
    with pytest.raises(ValueError, match="both"):
        e2.paged_attention(q, k, None, k, k, cu, cu, cu)
