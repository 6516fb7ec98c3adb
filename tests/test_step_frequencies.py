"""Rotary frequencies in parts where the trained positions are few or many turns."""

import math

import pytest

from sparse_attention_indexer_pmqa_gb300 import pmqa


@pytest.mark.parametrize("dim,base", [(2, 10000.0), (16, 10.0), (64, 10000.0), (128, 1e6)])
@pytest.mark.parametrize("trained", [1.0, 4.0, 6.0, 6.4, 40.0, 300.0, 4096.0, 1e6, 1e12])
@pytest.mark.parametrize("slow,fast", [(1.0, 32.0), (0.1, 0.2), (3.0, 3.1)])
def test_pairs_of_few_turns_are_divided_and_of_many_kept(dim, base, trained, slow, fast):
    """By the definition, pair by pair: divided where a pair turns fewer than `slow` times over the
    trained positions, kept where more than `fast` times and a pair within a step of either end
    anything between."""
    f, _ = pmqa.rope_frequencies(dim, base, kind=pmqa.PMQA_ROPE_PARTS, factor=8.0, trained=trained,
                                 slow_turns=slow, fast_turns=fast, device="cpu")
    step = base ** (2 / dim)  # of the turns from one pair to the next
    last = 0.0
    for i, x in enumerate(f.tolist()):
        plain = base ** (-2 * i / dim)
        turns = trained * plain / (2 * math.pi)
        share = (plain - x) / (plain - plain / 8.0)
        assert -1e-9 <= share <= 1 + 1e-9 and share >= last - 1e-9
        last = share
        if turns <= slow / step * (1 - 1e-9) or i == 0 and turns <= slow * (1 - 1e-9):
            assert abs(share - 1) <= 1e-9, (i, turns)
        if turns >= fast * step * (1 + 1e-9):
            assert abs(share) <= 1e-9, (i, turns)
