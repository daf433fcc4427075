"""Windows that the attention's bindings pass on (CPU only)."""
import pytest
import torch

from chunk_weight_rnn_amd import layer

BF, F8 = torch.bfloat16, torch.float8_e4m3fn
CASES = [(0, 0), (5, 5), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31, 2 ** 31 - 1), (2 ** 32 + 5, 2 ** 31 - 1), (2 ** 32, 2 ** 31 - 1),
         (-3, -1), (5 - 2 ** 32, -1)]  # a negative one is refused by the call


def tensor(*shape, dtype=BF):
    t = torch.empty(shape, dtype=dtype, device="meta")
    return tuple(t.shape), t.stride(), dtype


@pytest.mark.parametrize("window,want", CASES)
def test_windows_of_more_than_32_bits(window, want):
    q, kv, cu = tensor(8, 4, 64), tensor(8, 2, 64), tensor(3, dtype=torch.int32)
    assert layer._attention_plan(q, kv, kv, cu, window, None)[-1].window == want
    table = tensor(2, 3, dtype=torch.int32)
    for dtype, bits8 in ((BF, False), (F8, True)):
        cache = tensor(5, 2, 16, 64, dtype=dtype)
        assert layer._paged_plan(q, kv, kv, cache, cache, table, cu, window, None, bits8)[-1].a.window == want
