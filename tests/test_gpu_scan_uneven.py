"""The gated linear recurrence over batches of many short sequences and a few long ones
(next tokens beside chunks of prompts), against model_ref: the form for short sequences
meets lengths of every kind, gradients from the states it saves, and a long sequence is
not left to one wave."""
import numpy as np
import pytest
import torch

from tests import model_ref as ref
from tests.gpu_util import note
from tests.test_gpu_attention import f64, within
from tests.test_gpu_scan import TYPES, check, make

pytestmark = pytest.mark.gpu

LENS = {
    "a chunk after single tokens": [1] * 64 + [512],
    "a chunk before": [300] + [1] * 40,
    "a chunk among them": [1] * 21 + [1000] + [1] * 60,
    "short ones of more than a step": [16, 17, 33, 20, 32, 48, 49, 63, 64, 5] + [1] * 40,
    "where waves join": [63, 64, 65, 127, 128, 129, 255, 256, 257] + [2] * 90,
    "several in one workgroup": [0] * 60 + [70, 300, 0, 129, 1, 65, 128, 100],
    "many tiles": [1] * 300 + [4000],
    "one tile in all": [70] + [0] * 20,
    "none past a tile": [0, 128, 0] + [0] * 40,
    "seventeen": [17] * 3 + [1] * 60,
}


def test_the_short_form_takes_them():
    """Sums of at most 16 tokens a sequence, or 4 where no sequence can have two tiles: these need no workspace."""
    for name, lens in LENS.items():
        n, s = sum(lens), len(lens)
        assert n <= (16 if n > 128 else 4) * s, name


@pytest.mark.parametrize("dtype,gate", TYPES)
@pytest.mark.parametrize("name", list(LENS))
def test_lengths(name, dtype, gate):
    check(LENS[name], 70, dtype, gate, low=0.5)


@pytest.mark.parametrize("C", [1, 64, 65, 200])
def test_widths(C):
    check([1] * 30 + [150, 3, 200] + [1] * 30, C, "bf16", "f32")


@pytest.mark.parametrize("C,lens", [(16400, [1] * 66 + [100] + [2] * 5 + [80] + [1] * 70), (2000, [1] * 1200 + [300, 0, 70] + [1] * 200 + [150])])
def test_more_sequences_than_one_look(C, lens):
    """The workgroups for long ones look at 64 sequences each at a time: one of them per 64
    channels of many, sixteen of 2000."""
    check(lens, C, "bf16", "bf16", low=0.5)


@pytest.mark.parametrize("before,after", [(0, 40), (17, 0), (130, 300)])
def test_tokens_outside_every_sequence(before, after, monkeypatch):
    real = torch.empty

    def empty(*a, **k):
        t = real(*a, **k)
        return t.fill_(float("nan") if t.is_floating_point() else 255)
    monkeypatch.setattr(torch, "empty", empty)
    check([1] * 60 + [200, 0, 70], 66, "bf16", "f32", before=before, after=after)


@pytest.mark.parametrize("dtype,gate", TYPES)
def test_state_in_place_and_repeats(dtype, gate):
    import chunk_weight_rnn_amd as e2
    lens = [1] * 50 + [400, 90] + [3] * 20
    m = make(lens, 130, dtype, gate, seed=4)
    want = e2.gated_scan_forward(m["x"], m["a"], m["cu"], h0=m["h0"], save=True)
    for _ in range(3):
        h = m["h0"].clone()
        out, state, _ = e2.gated_scan_forward(m["x"], m["a"], m["cu"], h0=h, state=h)
        assert state is h and torch.equal(h, want[1]) and torch.equal(out, want[0])


@pytest.mark.parametrize("dtype,gate", TYPES)
def test_views_of_wider_tensors(dtype, gate):
    import chunk_weight_rnn_amd as e2
    lens = [1] * 40 + [333, 70]
    m = make(lens, 62, dtype, gate)
    want = e2.gated_scan_forward(m["x"], m["a"], m["cu"], h0=m["h0"])
    for off, wide in ((0, 200), (1, 63), (3, 71)):
        x, a = (torch.full((sum(lens), wide), 7.0, device="cuda").to(m[k].dtype) for k in ("x", "a"))
        x[:, off:off + 62], a[:, off:off + 62] = m["x"], m["a"]
        got = e2.gated_scan_forward(x[:, off:off + 62], a[:, off:off + 62], m["cu"], h0=m["h0"])
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_a_gate_of_zero_and_values_that_are_not_finite():
    import chunk_weight_rnn_amd as e2
    lens = [1] * 60 + [400] + [1] * 10
    m = make(lens, 66, "f32", "f32", seed=6)
    want, ws, _ = e2.gated_scan_forward(m["x"], m["a"], m["cu"], h0=m["h0"])
    m["x"][200, 7] = float("nan")
    out, state, _ = e2.gated_scan_forward(m["x"], m["a"], m["cu"], h0=m["h0"])
    assert torch.isnan(out[200:460, 7]).all() and torch.isnan(state[60, 7])
    keep = torch.ones_like(out, dtype=torch.bool)
    keep[200:460, 7] = False
    assert torch.equal(out[keep], want[keep])
    m["x"][200, 7], m["a"][260] = 1.0, 0.0
    out, _, _ = e2.gated_scan_forward(m["x"], m["a"], m["cu"], h0=m["h0"])
    r = ref.scan(f64(m["x"][260:460]), f64(m["a"][260:460]), np.zeros((1, 66)), [200], 0, "f32", "f32")
    within("out", out[260:460], *r["out"], "after the gate of 0")


def test_wrong_offsets_stay_inside():
    """Clamped: no access outside, no result promised."""
    import chunk_weight_rnn_amd as e2
    lens = [1] * 60 + [400, 70] + [1] * 10
    m = make(lens, 64, "bf16", "f32")
    n = sum(lens)
    for cu in (m["cu"].flip(0).contiguous(), m["cu"] + 10 ** 6, m["cu"] - 10 ** 6, m["cu"] * 0 + n,
               torch.tensor([0] + [n] * len(lens), dtype=torch.int32, device="cuda"),
               torch.tensor([0, n] * (len(lens) // 2) + [0], dtype=torch.int32, device="cuda")[:len(lens) + 1].contiguous()):
        assert cu.numel() == len(lens) + 1
        _, _, starts = e2.gated_scan_forward(m["x"], m["a"], cu, h0=m["h0"], save=True)
        e2.gated_scan_backward(m["dout"], m["x"], m["a"], starts, cu, dstate=m["dstate"])
    torch.cuda.synchronize()


def test_a_long_sequence_is_not_one_waves():
    """A chunk of 3800 tokens beside 256 single ones against the chunk alone, which the whole
    chip shares (21 us): read by the eight waves of a workgroup per 64 channels it takes 30 tiles
    one after the other, at 3 us each less than five times as long; one wave's 238 steps of 16
    tokens take 28 times as long."""
    import chunk_weight_rnn_amd as e2
    note("recurrence, time of an uneven batch")

    def best(lens):
        m = make(lens, 2048, "bf16", "f32")
        times = []
        for _ in range(12):
            s, e = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            s.record()
            for _ in range(10):
                e2.gated_scan_forward(m["x"], m["a"], m["cu"], h0=m["h0"], state=m["h0"])
            e.record()
            torch.cuda.synchronize()
            times.append(s.elapsed_time(e))
        return min(times)
    assert best([1] * 256 + [3800]) < 10 * best([3800])
