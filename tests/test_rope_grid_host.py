"""Refusals of ulysses_plan_set_rope_grid (host only)."""
import pytest

from ulysses_sequence_all_gb300 import binding as B
from ulysses_sequence_all_gb300 import build as build_mod


@pytest.fixture(scope="module", autouse=True)
def built():
    import os
    if not os.path.exists(B.LIBRARY):
        build_mod.build_library()


def plan():
    return B.ulysses_plan(2, 1, [20, 16], [2, 2], 64, "bfloat16")


@pytest.mark.parametrize("extents,pairs,first", [
    ((), (), 0),
    ((36,), (32,), 0),
    ((2, 3, 6), (12, 10, 10), 0),
    ((5, 7), (0, 32), 1),
    ((1, 1, 1, 1), (8, 8, 8, 8), 35),
])
def test_accepted(extents, pairs, first):
    B.ulysses_plan_set_rope_grid(plan(), extents, pairs, first)


@pytest.mark.parametrize("extents,pairs,first", [
    ((37,), (32,), 0),                    # longer than the sequence
    ((6, 6), (16, 16), 1),                # passes its end
    ((6, 6), (16, 17), 0),                # more pairs than d/2
    ((6, 6), (33, 0), 0),
    ((6, 6), (-1, 16), 0),
    ((0, 6), (16, 16), 0),
    ((-6, -6), (16, 16), 0),
    ((6, 6), (16, 16), -1),
    ((2,) * 5, (4,) * 5, 0),              # five axes
    ((2 ** 62, 4), (16, 16), 0),          # a product past 64 bits
    ((6,), (32,), 2 ** 62),
])
def test_refused(extents, pairs, first):
    with pytest.raises(B.UlyssesError) as e:
        B.ulysses_plan_set_rope_grid(plan(), extents, pairs, first)
    assert e.value.status == B.ULY_EINVAL


def test_refused_arguments():
    with pytest.raises(ValueError):
        B.ulysses_plan_set_rope_grid(plan(), (6, 6), (16,))
    lib = B.library()
    one = (B._i64 * 1)(4)
    assert lib.ulysses_plan_set_rope_grid(None, 1, one, one, 0) == B.ULY_EINVAL
    assert lib.ulysses_plan_set_rope_grid(plan(), -1, one, one, 0) == B.ULY_EINVAL
    assert lib.ulysses_plan_set_rope_grid(plan(), 1, None, one, 0) == B.ULY_EINVAL
    assert lib.ulysses_plan_set_rope_grid(plan(), 1, one, None, 0) == B.ULY_EINVAL
