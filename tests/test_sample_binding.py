"""Numbers that the binding of sampling passes on (CPU only)."""
import pytest
import torch

from chunk_weight_rnn_amd import tokens


def plan(top_k):
    return tokens._sample_plan(((4, 50), (50, 1), torch.bfloat16), 1.0, top_k, 1.0, 0.0)[3]


@pytest.mark.parametrize("top_k,want", [(0, 0), (7, 7), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31, 2 ** 31 - 1), (2 ** 32 + 5, 2 ** 31 - 1),
                                        (2 ** 63, 2 ** 31 - 1), (-1, 0), (5 - 2 ** 32, 0)])
def test_a_top_k_of_more_than_32_bits_keeps_all(top_k, want):
    """More than there are logits, or none and less, is all of them, and not its low 32 bits."""
    assert plan(top_k).top_k == want


def test_a_top_k_that_is_no_whole_number_is_refused():
    with pytest.raises(TypeError):
        plan(5.0)
