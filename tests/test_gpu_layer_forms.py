"""Forms of the layer's kernels that only larger calls take, each with a check on
the host that the call is planned in the form that is meant: the decoding
kernel's shared-out line of keys (stretches of several units and of several
items, items over many stretches), and the fp32 backward where items are not
shared out over workgroups."""
import ctypes

import pytest

from chunk_weight_rnn_amd import _lib as L
from tests.test_gpu_attention import check as check_packed
from tests.test_gpu_paged import check as check_paged

pytestmark = pytest.mark.gpu

GROUPS, UNIT, ROWS = 256, 128, 32  # workgroups of the line, keys of a unit, rows of an item


def up(x, n):
    return -(-x // n)


def line_of(ctx, new, H, K, page, D, window):
    """[(units, items) per sequence] of the decoding kernel's line, after a check
    that the call takes the kernel in its two-launch form."""
    width = max(up(a + b, page) for a, b in zip(ctx, new)) + 1  # of the table that check() makes
    N, S = sum(new), len(ctx)
    a = L.AttentionDesc(1, window, N, S, H, K, D, D ** -0.5, 0, H * D, D, K * D, D, K * D, D)
    d = L.PagedDesc(a, sum(up(x + y, page) for x, y in zip(ctx, new)) + 3, page, width,
                    K * page * D, page * D, D, K * page * D, page * D, D)
    rows = 2 * GROUPS * ROWS
    assert L.load().e2ttt_paged_workspace_size(ctypes.byref(d)) == rows * D * 4 + rows * 4
    units = []
    for c, n in zip(ctx, new):
        lo = max(0, c - window + 1) // 32 * 32 if window else 0
        units += [up(c + n - lo, UNIT)] * (up(n * H // K, ROWS) * K)
    return units


def spread(count, top):
    return [(i * i * 37 + i * 611) % (top + 1) for i in range(count)]


@pytest.mark.parametrize("D,page", [(128, 64), (128, 16), (64, 32), (96, 64)])
@pytest.mark.parametrize("window", [0, 1500])
@pytest.mark.parametrize("n", [1, 2])
def test_stretches_of_several_units(D, page, window, n):
    """Uneven contexts: stretches hold whole items between parts of two others,
    and longer items are cut several times."""
    ctx, new = spread(40, 4000) + [0, 3, 4000], [n] * 43
    units = line_of(ctx, new, 16, 4, page, D, window)
    per = up(sum(units), GROUPS)
    assert per > 2 and sum(units) > 2 * GROUPS
    assert min(units) * 3 <= per and max(units) > per  # several items in a stretch, and items over several
    check_paged(ctx, new, 16, 4, D, page, "bf16", window, seed=D + n)


@pytest.mark.parametrize("context,D,per", [(12000, 128, 1), (40000, 128, 2), (12000, 64, 1)])
def test_an_item_over_many_stretches(context, D, per):
    """More stretches than a wave has lanes join into one row."""
    units = line_of([context], [1], 8, 1, 64, D, 0)
    assert up(sum(units), GROUPS) == per and units[0] / per > 64
    check_paged([context], [1], 8, 1, D, 64, "bf16")


def test_more_sequences_than_lanes_share_the_line():
    ctx, new = spread(150, 1500), [1] * 150
    assert up(sum(line_of(ctx, new, 4, 2, 16, 128, 0)), GROUPS) > 2
    check_paged(ctx, new, 4, 2, 128, 16, "bf16")


def parts_of(lens, H, K, D):
    """(dq, dk and dv) workgroups per item of the fp32 backward, from its workspace."""
    N = sum(lens)
    d = L.AttentionDesc(0, 0, N, len(lens), H, K, D, D ** -0.5, 0, H * D, D, K * D, D, K * D, D)
    room = L.load().e2ttt_attention_backward_workspace_size(ctypes.byref(d)) - up(N * H * 8, 256) * 256
    block = 32 if D <= 64 else 16
    want = [min(8, up(512, up(n, block) * K)) for n in (N * H // K, N)]
    assert room == 4 * N * D * ((want[0] * H if want[0] > 1 else 0) + (2 * want[1] * K if want[1] > 1 else 0))
    return tuple(want)


@pytest.mark.parametrize("window", [0, 100])
@pytest.mark.parametrize("H,K,D,tokens,parts", [(4, 2, 64, 4100, (1, 2)), (4, 4, 64, 4100, (1, 1)),
                                                (12, 4, 64, 4100, (1, 1)), (4, 1, 128, 2100, (1, 4)),
                                                (4, 4, 128, 2100, (1, 1)), (6, 2, 32, 4100, (1, 2))])
def test_fp32_backward_of_larger_calls(H, K, D, tokens, parts, window):
    lens = [333, 1, 0, 64, 450]
    while sum(lens) < tokens:
        lens.append(min(257 + 13 * len(lens), tokens - sum(lens)))
    assert parts_of(lens, H, K, D) == parts
    check_packed(lens, H, K, D, "f32", window)
