"""Host-side checks of the operators around a hybrid model's layers
(include/e2ttt_tokens.h, and the recurrence and the 8-bit cache of
include/e2ttt_layer.h): every refusal happens before any device call (no GPU
needed; the pointers here are never read)."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest

from chunk_weight_rnn_amd import _lib as L
from tests.test_layer_abi import ALIAS, BAD, BASE, GAP, INVALID, OK, ROOT, UNSUPPORTED, WORKSPACE, lib, paged, ptrs  # noqa: F401

NAN, INF = float("nan"), float("inf")
WS = BASE + 30 * GAP


def make(cls, base, kw):
    d = cls(*base)
    for n, v in kw.items():
        assert hasattr(d, n)
        setattr(d, n, v)
    return d


def scan(N=1000, S=3, C=64, io=1, gate=0, **kw):
    return make(L.ScanDesc, (io, gate, N, S, C, C, C), kw)


def embed(N=100, V=50, W=64, table=0, io=1, nbytes=8, scale=1.0, **kw):
    return make(L.EmbeddingDesc, (table, io, nbytes, scale, N, V, W), kw)


def sampling(rows=4, V=100, io=1, **kw):
    return make(L.SampleDesc, (io, 0, 1.0, 1.0, 0.0, 0, rows, V, V), kw)


def scan_fwd(lib, d, p=None, ws=WS, n=1 << 40):  # x, a, h0, cu, out, state, starts
    return lib.e2ttt_scan_forward(ctypes.byref(d), *(ptrs(7) if p is None else p), ws, n, None)


def scan_bwd(lib, d, p=None, ws=WS, n=1 << 40):  # dout, x, a, starts, dstate, cu, dx, da, dh0
    return lib.e2ttt_scan_backward(ctypes.byref(d), *(ptrs(9) if p is None else p), ws, n, None)


def look(lib, d, p=None):  # tokens, table, out
    return lib.e2ttt_embedding_forward(ctypes.byref(d), *(ptrs(3) if p is None else p), None)


def look_bwd(lib, d, p=None, ws=WS, n=1 << 40):  # dout, tokens, dtable
    return lib.e2ttt_embedding_backward(ctypes.byref(d), *(ptrs(3) if p is None else p), ws, n, None)


def draw(lib, d, p=None):  # logits, u, temperature, top_k, top_p, min_p, token, logprob
    return lib.e2ttt_sample(ctypes.byref(d), *(ptrs(8) if p is None else p), None, 0, None)


def test_exports(lib):  # noqa: F811
    text = open(os.path.join(ROOT, "include", "e2ttt_tokens.h")).read()
    names = set(re.findall(r"E2TTT_API[^;(]*?\b(e2ttt_\w+)\s*\(", text))
    assert names == set(L.TOKENS_EXPORTS)
    assert not names & (set(L.EXPORTS) | set(L.LAYER_EXPORTS))
    for n in names:
        assert hasattr(lib, n), n


def test_desc_sizes_and_constants_match_the_headers(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "e2ttt_layer.h"\n#include "e2ttt_tokens.h"\n'
                   'int main(void){printf("%zu %zu %zu %zu %zu %zu %d\\n",sizeof(e2ttt_scan_desc),sizeof(e2ttt_embedding_desc),'
                   'sizeof(e2ttt_sample_desc),offsetof(e2ttt_scan_desc,x_tok),offsetof(e2ttt_embedding_desc,tokens),'
                   'offsetof(e2ttt_sample_desc,rows),E2TTT_SCAN_TILE);return 0;}')
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(tmp_path / "s")], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "s")], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(L.ScanDesc), ctypes.sizeof(L.EmbeddingDesc), ctypes.sizeof(L.SampleDesc), L.ScanDesc.x_tok.offset,
                   L.EmbeddingDesc.tokens.offset, L.SampleDesc.rows.offset, L.SCAN_TILE]


@pytest.mark.parametrize("field,value", [("io_dtype", 2), ("io_dtype", -1), ("gate_dtype", 2), ("tokens", -1), ("seqs", -1),
                                         ("width", 0), ("x_tok", 63), ("a_tok", 0)])
def test_scan_bad_desc(lib, field, value):  # noqa: F811
    d = scan(**{field: value})
    assert scan_fwd(lib, d) == INVALID and scan_bwd(lib, d) == INVALID
    assert lib.e2ttt_scan_workspace_size(ctypes.byref(d)) == BAD
    assert lib.e2ttt_scan_backward_workspace_size(ctypes.byref(d)) == BAD


def test_scan_refusals(lib):  # noqa: F811
    assert scan_fwd(lib, scan(io=0, gate=1)) == INVALID  # gates of fewer bits than the values
    for kw in (dict(N=1 << 31), dict(S=1 << 28), dict(C=(1 << 24) + 1), dict(x_tok=(1 << 31) + 1), dict(S=1 << 23, N=1 << 30)):
        assert scan_fwd(lib, scan(**kw)) == UNSUPPORTED, kw
        assert scan_bwd(lib, scan(**kw)) == UNSUPPORTED, kw
    for i in (0, 1, 3, 4):  # h0, state and starts may be null
        p = ptrs(7)
        p[i] = 0
        assert scan_fwd(lib, scan(), p) == INVALID, i
    for i in range(7):
        p = ptrs(7)
        p[i] += 1
        assert scan_fwd(lib, scan(), p) == INVALID, i
    for i in (0, 1, 2, 3, 5, 6, 7):  # dstate and dh0 may be null
        p = ptrs(9)
        p[i] = 0
        assert scan_bwd(lib, scan(), p) == INVALID, i
    assert scan_fwd(lib, scan(S=0), [0] * 7) == OK and scan_bwd(lib, scan(S=0), [0] * 9) == OK
    assert lib.e2ttt_scan_forward(None, *ptrs(7), WS, 1 << 40, None) == INVALID


def test_scan_aliasing(lib):  # noqa: F811
    for o in (4, 5, 6):
        for i in range(7):
            if i == o or (o, i) == (5, 2):  # state in place of h0
                continue
            p = ptrs(7)
            p[o] = p[i]
            assert scan_fwd(lib, scan(N=1 << 16), p) == ALIAS, (o, i)
    p = ptrs(7)
    p[5] = p[2] + 4  # state partly over h0
    assert scan_fwd(lib, scan(), p) == ALIAS
    for o in (6, 7, 8):
        for i in range(9):
            if i != o:
                p = ptrs(9)
                p[o] = p[i]
                assert scan_bwd(lib, scan(N=1 << 16), p) == ALIAS, (o, i)


def test_scan_workspace(lib):  # noqa: F811
    """Tiles of a sequence tell each other their states; alignment of the tensors changes the
    plan but not the size that was asked for."""
    d = scan(N=4000, S=1, C=62)
    need, back = lib.e2ttt_scan_workspace_size(ctypes.byref(d)), lib.e2ttt_scan_backward_workspace_size(ctypes.byref(d))
    assert 0 < back == need < 1 << 20
    for ws, n in ((None, need), (WS, need - 1), (WS + 16, need)):
        assert scan_fwd(lib, d, ws=ws, n=n) == WORKSPACE
        p = ptrs(7)
        p[0] += 2  # bf16 values at an odd place
        assert scan_fwd(lib, d, p, ws=ws, n=n) == WORKSPACE
    assert scan_bwd(lib, d, ws=WS, n=back - 1) == WORKSPACE
    assert lib.e2ttt_scan_workspace_size(ctypes.byref(scan(N=64, S=64, C=2048))) == 0
    assert lib.e2ttt_scan_backward_workspace_size(ctypes.byref(scan(N=300, S=64, C=2048))) > 0
    assert lib.e2ttt_scan_workspace_size(ctypes.byref(scan(N=128, S=1))) == 0


@pytest.mark.parametrize("field,value", [("table_dtype", 2), ("io_dtype", -1), ("token_bytes", 2), ("scale", NAN), ("scale", INF),
                                         ("tokens", -1), ("vocab", 0), ("width", 0)])
def test_embedding_bad_desc(lib, field, value):  # noqa: F811
    d = embed(**{field: value})
    assert look(lib, d) == INVALID and look_bwd(lib, d) == INVALID
    assert lib.e2ttt_embedding_backward_workspace_size(ctypes.byref(d)) == BAD


def test_embedding_refusals(lib):  # noqa: F811
    for kw in (dict(N=(1 << 31) - 1), dict(V=(1 << 24) + 1), dict(W=(1 << 20) + 1)):
        assert look(lib, embed(**kw)) == UNSUPPORTED and look_bwd(lib, embed(**kw)) == UNSUPPORTED
    for i in range(3):
        for bad in (0, BASE + i * GAP + 1):
            p = ptrs(3)
            p[i] = bad
            assert look(lib, embed(), p) == INVALID, i
            assert look_bwd(lib, embed(), p) == INVALID, i
    for i in (0, 1):
        p = ptrs(3)
        p[2] = p[i] + 16
        assert look(lib, embed(N=1000), p) == ALIAS and look_bwd(lib, embed(N=1000), p) == ALIAS
    assert look(lib, embed(N=0), [0] * 3) == OK
    need = lib.e2ttt_embedding_backward_workspace_size(ctypes.byref(embed()))
    assert need >= 4 * 51 + 4 * 100
    assert look_bwd(lib, embed(), ws=None) == WORKSPACE and look_bwd(lib, embed(), n=need - 1) == WORKSPACE
    assert look_bwd(lib, embed(), [ptrs(3)[0], ptrs(3)[1], WS + 64]) == ALIAS


@pytest.mark.parametrize("field,value", [("io_dtype", 2), ("temperature", -1.0), ("temperature", NAN), ("temperature", INF),
                                         ("top_p", -0.1), ("top_p", NAN), ("min_p", -0.1), ("min_p", 1.1), ("min_p", NAN),
                                         ("rows", -1), ("vocab", 0), ("row_stride", 99), ("reserved", 1)])
def test_sample_bad_desc(lib, field, value):  # noqa: F811
    d = sampling(**{field: value})
    assert draw(lib, d) == INVALID
    assert lib.e2ttt_sample_workspace_size(ctypes.byref(d)) == BAD


def test_sample_refusals(lib):  # noqa: F811
    for kw in (dict(V=(1 << 18) - 7), dict(rows=1 << 22), dict(row_stride=(1 << 40) + 1)):
        assert draw(lib, sampling(**kw)) == UNSUPPORTED, kw
    for i in (0, 1, 6):
        p = ptrs(8)
        p[i] = 0
        assert draw(lib, sampling(), p) == INVALID, i
    for i in range(8):
        p = ptrs(8)
        p[i] += 1
        assert draw(lib, sampling(), p) == INVALID, i
    for o in (6, 7):
        for i in range(8):
            if i != o:
                p = ptrs(8)
                p[o] = p[i]
                assert draw(lib, sampling(), p) == ALIAS, (o, i)
    assert draw(lib, sampling(rows=0), [0] * 8) == OK


def page8(lib, d, p=None, ws=WS, n=1 << 40):  # q, k, v, k_cache, v_cache, k_scale, v_scale, table, cu, cached, out
    return lib.e2ttt_paged8_attention(ctypes.byref(d), *(ptrs(11) if p is None else p), ws, n, None)


def test_paged8_refusals(lib):  # noqa: F811
    assert page8(lib, paged(dtype=0)) == UNSUPPORTED  # fp32 beside 8 bits
    for D, want in ((24, INVALID), (8, INVALID), (20, UNSUPPORTED), (136, UNSUPPORTED)):  # strides of whole 16 bytes
        assert page8(lib, paged(D=D)) == want, D
    d = paged(D=24)
    d.kc_slot = d.vc_slot = 32
    d.kc_head = d.vc_head = 16 * 32
    d.kc_page = d.vc_page = 2 * 16 * 32
    assert page8(lib, d) == UNSUPPORTED
    for field, value in (("page_size", 24), ("pages", -1), ("kc_slot", 8), ("vc_head", 64), ("kc_page", -16), ("vc_slot", 0)):
        d = paged()
        setattr(d, field, value)
        assert page8(lib, d) == INVALID, field
        assert lib.e2ttt_paged8_workspace_size(ctypes.byref(d)) == BAD
    for i in range(11):
        p = ptrs(11)
        p[i] = 0
        assert page8(lib, paged(), p) == INVALID, i  # k without v among them
    for i in (0, 1, 2, 3, 4, 7, 8, 9, 10):  # scales are bytes
        p = ptrs(11)
        p[i] += 2
        assert page8(lib, paged(), p) == INVALID, i
    for o in (3, 4, 5, 6, 10):
        for i in range(11):
            if o == i or {o, i} == {3, 4}:  # one tensor may hold both caches
                continue
            p = ptrs(11)
            p[o] = p[i]
            assert page8(lib, paged(), p) == ALIAS, (o, i)
    d = paged(W=4096)
    need = lib.e2ttt_paged8_workspace_size(ctypes.byref(d))
    assert need == 2 * lib.e2ttt_paged_workspace_size(ctypes.byref(d)) > 0  # twice the workgroups share the keys
    assert page8(lib, d, ws=None) == WORKSPACE and page8(lib, d, n=need - 1) == WORKSPACE
    d = paged()
    d.a.tokens = 0
    assert page8(lib, d, [0] * 11) == OK


def test_paged8_grids_are_checked_before_the_cache_is_written(lib):  # noqa: F811
    """A call of too many workgroups is refused before its first launch."""
    at = [1 << 46 | i << 40 for i in range(16)]
    for N, S, kw in ((1 << 24, 1 << 24, dict(H=1, K=1)), (1 << 22, 1, dict(H=64, K=64))):
        d = paged(P=10, W=1, ps=16, **kw)
        d.a.tokens, d.a.seqs = N, S
        assert page8(lib, d, at[:11], at[15], 1 << 39) == UNSUPPORTED, (N, S, kw)
