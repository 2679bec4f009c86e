"""The waits of the wide cache attention kernel, on a model of its warps (CPU): every
role reads what it waits for and none waits for ever, whatever the schedule."""
import random

import pytest

from tests.cache_split import RAGGED, Stale, ragged_lens, schedules, segments


def runs_ahead(segs):
    """Whether half 1 passes three or more segments of one tile before one that it shares."""
    run = 0
    for n, by_rows in segs:
        if n == 1 and not by_rows:
            run += 1
        elif run >= 3 and not by_rows:
            return True
        else:
            run = 0
    return False


def ctas(B, longest, Sq, H, G, seed):
    return segments(ragged_lens(B, longest, seed), Sq * G, H, Sq, G)


@pytest.mark.parametrize("shape", RAGGED)
def test_the_ragged_shapes_have_a_half_that_runs_ahead(shape):
    assert any(runs_ahead(s) for s in ctas(*shape))


@pytest.mark.parametrize("segs", [[(1, False)] * 4 + [(2, False)], [(1, False)] * 3 + [(4, False)], [(3, False)] + [(1, False)] * 4 + [(3, False)]])
def test_the_scores_have_to_wait_for_the_scales(segs):
    """A softmax that waits for a tile's scales first, without the scores' thread having
    seen them, may meet the parity of an older phase: the model finds it."""
    with pytest.raises(Stale):
        for seed in range(200):
            schedules(segs, False, 1, seed)
    for seed in range(200):
        schedules(segs, True, 1, seed)


@pytest.mark.parametrize("shape", RAGGED)
def test_every_cta_of_the_ragged_shapes(shape):
    for segs in sorted(set(map(tuple, ctas(*shape)))):
        schedules(list(segs), True, 2, len(segs))


@pytest.mark.parametrize("seed", range(4))
def test_segments_in_any_order(seed):
    r = random.Random(seed)
    for _ in range(150):
        segs = []
        for _ in range(r.randint(1, 9)):
            segs += [(r.choice([1, 1, 1, 2, 2, 3, 4, 7]), r.random() < r.choice([0, 0, 0.3, 0.8]))] * r.choice([1, 1, 2, 4])
        schedules(segs, True, 2, r.random())
