"""What the layer's host code plans, seen through the workspace sizes (no GPU)."""
import ctypes

import pytest

from tests.test_layer_abi import attn, lib, paged  # noqa: F401  (lib is a fixture)

BAD = ctypes.c_size_t(-1).value
WIDEST = 2 ** 31 - 1


def packed_size(lib, **kw):
    return lib.e2ttt_attention_workspace_size(ctypes.byref(attn(**kw)))


def paged_size(lib, N, S, window, pages, dtype):
    d = paged(P=1000, ps=64, W=pages, H=16, K=4, window=window, dtype=dtype)
    d.a.tokens, d.a.seqs = N, S
    return lib.e2ttt_paged_workspace_size(ctypes.byref(d))


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("window", [WIDEST, WIDEST - 1, WIDEST - 70, 1 << 30])
def test_a_window_wider_than_every_context_plans_as_none(lib, window, dtype):  # noqa: F811
    n = (512, 2048)[dtype]  # row tiles that leave compute units idle (16 rows each in fp32, 128 in bf16)
    whole = packed_size(lib, N=n, S=1, H=4, K=1, dtype=dtype)
    assert whole not in (0, BAD)
    assert packed_size(lib, N=n, S=1, H=4, K=1, dtype=dtype, window=window) == whole
    for N, S, pages in ((n // 8, 1, 260), (8, 8, 64)):  # a chunk, single tokens
        want = paged_size(lib, N, S, 0, pages, dtype)
        assert want not in (0, BAD)
        assert paged_size(lib, N, S, window, pages, dtype) == want
