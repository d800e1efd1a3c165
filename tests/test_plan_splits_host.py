"""A plan's split lists have an entry for each rank: others are refused by the binding, which would else hand
the library a list filled up with zeros."""
import pytest

from ulysses_sequence_all_gb300 import binding as B


@pytest.mark.parametrize("W, seq, heads, what", [
    (4, [16, 0], [1] * 4, "seq_splits"), (4, [16, 0, 0, 0], [2, 2], "head_splits"), (2, [], [1, 1], "seq_splits"),
    (1, [16, 0], [1], "seq_splits"), (1, [16], [1, 0], "head_splits")])
def test_lists_of_another_length_are_refused(W, seq, heads, what):
    with pytest.raises(ValueError, match=what):
        B.ulysses_plan(W, 1, seq, heads, 128, "bfloat16")


@pytest.mark.parametrize("W", [1, 2, 4])
def test_the_readme_cache(W):
    plan = B.ulysses_plan(W, 40, [16] + [0] * (W - 1), [2] * W, 128, "bfloat16")
    assert plan.seq_splits == [16] + [0] * (W - 1) and plan.head_splits == [2] * W


def test_splits_of_any_iterable():
    plan = B.ulysses_plan(2, 1, (n for n in (5, 7)), iter([1, 2]), 128, "bfloat16")
    assert plan.seq_splits == [5, 7] and plan.head_splits == [1, 2]
