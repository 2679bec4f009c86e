"""The waits of the wide cache attention's softmax as the kernel has them (CPU): a tile's
second score buffer does not wait for the scales that its first has waited for."""
import random

import pytest

from tests.cache_split import RAGGED, ROLES, SLOTS, Stale, Wide, ragged_lens, segments


class Once(Wide):
    """The model's softmax without the wait for the scales at the buffers that `waits`
    does not name (0: a tile's first, 1: its second)."""
    waits = (0,)

    def softmax(self, t):
        buffers = 0
        for at in super().softmax(t):
            if at is not None and any(at[0] is s for s in self.scales):
                buffers += 1                     # one wait a buffer, two buffers a tile
                if (buffers - 1) % 2 not in self.waits:
                    continue
            yield at


class Never(Once):
    waits = ()


def run(kind, segs, count, seed):
    rng = random.Random(seed)
    for _ in range(count):
        kind(segs, True).run(rng, rng.sample(ROLES, rng.randint(0, 2)))


@pytest.mark.parametrize("shape", RAGGED)
def test_every_cta_of_the_ragged_shapes(shape):
    B, longest, Sq, H, G, seed = shape
    for segs in sorted(set(map(tuple, segments(ragged_lens(B, longest, seed), Sq * G, H, Sq, G)))):
        run(Once, list(segs), 2, len(segs))


@pytest.mark.parametrize("seed", range(4))
def test_segments_in_any_order(seed):
    r = random.Random(seed)
    for _ in range(150):
        segs = []
        for _ in range(r.randint(1, 9)):
            segs += [(r.choice([1, 1, 1, 2, 2, 3, 4, 7]), r.random() < r.choice([0, 0, 0.3, 0.8]))] * r.choice([1, 1, 2, 4])
        run(Once, segs, 2, r.random())


@pytest.mark.parametrize("slow", ["softmax 0", "softmax 1", "convert k", "convert v", "sums 0", "sums 1"])
def test_one_role_far_behind(slow):
    """More tiles than there are slots while one role hardly moves."""
    for segs in ([(3 * SLOTS, False)], [(3 * SLOTS, True)], [(1, False)] * 5 + [(2 * SLOTS, True)] + [(1, True)] * 5):
        for seed in range(20):
            Once(segs, True).run(random.Random(seed), (slow,))


def test_the_first_buffer_has_to_wait():
    """The model finds a softmax that waits at neither buffer."""
    with pytest.raises(Stale):
        for seed in range(200):
            run(Never, [(6, False), (1, False), (5, True)], 1, seed)
