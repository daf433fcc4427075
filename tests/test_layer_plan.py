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


def test_grids_that_would_wrap_around_are_refused(lib):  # noqa: F811
    """2^24 workgroups of 256 threads are 2^32 threads, more than HIP counts; before any launch."""
    from tests.test_layer_abi import UNSUPPORTED, page_call
    at = [1 << 46 | i << 40 for i in range(16)]  # never read, a TiB apart
    ws, room = at[15], 1 << 39

    def forward(**kw):
        return lib.e2ttt_attention_forward(ctypes.byref(attn(**kw)), *at[:6], ws, room, None)

    def backward(**kw):
        return lib.e2ttt_attention_backward(ctypes.byref(attn(**kw)), *at[:10], ws, room, None)

    for kw in (dict(N=1000, S=1 << 24, H=1, K=1), dict(N=1000, S=(1 << 24) // 64, H=64, K=64),
               dict(N=1 << 22, S=1, H=64, K=64, dtype=0), dict(N=1 << 22, S=(1 << 24) - 4, H=4, K=1)):
        assert forward(**kw) == UNSUPPORTED, kw
        assert backward(**kw) == UNSUPPORTED, kw
    # more key blocks than row tiles
    assert backward(N=1 << 24, S=(1 << 24) - (1 << 17) - 1000, H=1, K=1) == UNSUPPORTED
    # single tokens by items, new keys by their bytes
    for N, S, kw in ((1 << 24, 1 << 24, dict(H=1, K=1)), (1 << 20, 1 << 20, dict(H=16, K=16)),
                     (1 << 24, 1, dict(H=32, K=32)), (1 << 22, 1, dict(H=64, K=64, dtype=0))):
        d = paged(P=10, W=1, ps=16, **kw)
        d.a.tokens, d.a.seqs = N, S
        assert page_call(lib, d, at[:9], ws, room) == UNSUPPORTED, (N, S, kw)
