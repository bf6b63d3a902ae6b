"""The hand-over of work between the roles of the paged attention's tcgen05 kernels, under many schedules of barrier_model."""
import random

import pytest

import barrier_model as M

PARTS = [[1] * 6, [1, 1], [1, 1, 1], [2] * 4, [3, 3], [1, 2, 1, 1, 2, 1], [2, 1, 1, 1, 3], [1, 1, 5, 1, 1], [9], [4, 1, 1, 1, 1, 1, 1, 2]]


def faults(make, parts, seeds=15):
    out = set()
    for seed in range(seeds):
        out |= make(list(parts)).run(seed)
    return out


@pytest.mark.parametrize("parts", PARTS, ids=str)
@pytest.mark.parametrize("make", [M.rows128, M.rows256, M.causal])
def test_no_wait_is_two_phases_behind(make, parts):
    assert not faults(make, parts)


@pytest.mark.parametrize("make", [M.rows128, M.rows256, M.causal])
def test_any_parts(make):
    rng = random.Random(5)
    for seed in range(25):
        parts = [rng.choice((1, 1, 1, 2, 3, 6)) for _ in range(rng.randint(1, 12))]
        assert not make(parts).run(seed), parts


def test_a_wait_for_the_queries_misses_phases():
    """Were the second issuer to wait for a part's queries, which nothing holds back for it, it could find the next part's
    there too and wait for those of the one after, which may never come."""
    wrong = lambda parts: M.rows128(parts, pv_waits_for_queries=True)
    assert {"phase", "stuck"} <= faults(wrong, [1] * 6, 40)


def test_a_part_s_end_by_its_last_product_s_phase():
    """Were a part's end to wait for its last product by that product's phase, a group a unit ahead of the issuer could
    take the product before the last for it."""
    wrong = lambda parts: M.causal(parts, end_by_product=True)
    assert "phase" in faults(wrong, [2] * 4, 60) or "phase" in faults(wrong, [3, 3, 3], 60)


def test_places_for_the_factors():
    """Three parts' factors are alive in the 128-row kernel where parts have one unit, two in the other."""
    assert "factors" in faults(lambda parts: M.rows128(parts, factors=2), [1] * 6, 40)
    assert not faults(lambda parts: M.rows128(parts, factors=3), [1] * 8, 40)
    assert not faults(lambda parts: M.rows128(parts, factors=2), [2] * 4, 40)
    assert "factors" in faults(lambda parts: M.rows256(parts, factors=1), [1] * 6, 40)
