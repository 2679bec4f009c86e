"""What kv_pages_reserve and kv_pages_release do with what is wrong on the device: tokens
without a row, errors that are pending, table entries that are no pages."""
import random

import pytest
import torch

from tests.cache_common import ints
from tests.gpu_common import ensure_library

pytestmark = pytest.mark.gpu
PAGE = 16


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    return ensure_library()


@pytest.fixture(autouse=True)
def no_device_error():
    import quantized_attention_diffusion_gb300 as qad
    yield
    assert qad.sync_status() == 0


def pages_of(n):
    return -(-n // PAGE)


# One kernel; two; two of which the first finds the pages.
@pytest.mark.parametrize("B,new,rows", [(5, 9, 0.6), (300, 40, 0.5), (300, 90, 0.7), (1024, 20, 0.99), (1500, 30, 0.5), (2500, 3, 0.0)])
def test_packed_tokens_without_a_row_are_not_served(B, new, rows):
    """Sequences are served while their tokens have rows; one whose count alone is above
    `tokens` takes none, as one with a negative count."""
    import quantized_attention_diffusion_gb300 as qad
    r = random.Random(B + new)
    lens = [r.randint(0, 50) for _ in range(B)]
    counts = [r.randint(0, new) for _ in range(B)]
    tokens = max(new, int(rows * sum(counts)))
    for b in (2, B // 3):
        counts[b] = r.choice([-1, tokens + 1, tokens + 500])
    counts[B // 4] = 0
    width = pages_of(max(50 + max(counts), 1))
    need = sum(pages_of(n + max(c, 0)) for n, c in zip(lens, counts))
    pool = list(range(need + 3))
    r.shuffle(pool)
    table, at = [], 0
    for n in lens:
        table.append(pool[at:at + pages_of(n)] + [-1] * (width - pages_of(n)))
        at += pages_of(n)
    free, stack = len(pool) - at, pool[at:] + [-7] * at

    want_table, taken, first, slots, positions = [list(x) for x in table], [], [], [-1] * tokens, [0] * tokens
    row, gone = 0, 0
    for b, (n, c) in enumerate(zip(lens, counts)):
        takes = c if 0 <= c <= tokens else 0
        ok = 0 <= c <= tokens and (c == 0 or row + c <= tokens)
        first.append(row)
        taken.append(c if ok else 0)
        if ok:
            for j in range(pages_of(n), pages_of(n + c)):
                want_table[b][j] = stack[free - 1 - gone]
                gone += 1
            for i in range(c):
                slots[row + i] = want_table[b][(n + i) // PAGE] * PAGE + (n + i) % PAGE
                positions[row + i] = n + i
        row += takes
    assert row > tokens and sum(taken) <= tokens

    t = torch.tensor(table, dtype=torch.int32, device="cuda")
    got = qad.kv_pages_reserve(ints(stack), ints([free]), ints(lens), ints(counts), t, PAGE, tokens)
    assert qad.sync_status() == 8
    assert got.taken.tolist() == taken and got.first.tolist() == first
    assert got.lens.tolist() == [n + c for n, c in zip(lens, taken)]
    assert got.free_count.tolist() == [free - gone]
    assert t.tolist() == want_table
    assert got.slots.tolist() == slots and got.positions.tolist() == positions


def test_a_batch_whose_rows_are_just_enough_or_one_too_few():
    import quantized_attention_diffusion_gb300 as qad
    for tokens, taken, left in ((6, [3, 0, 3], 2), (5, [3, 0, 0], 3), (3, [3, 0, 0], 3), (2, [0, 0, 0], 4)):
        table = torch.full((3, 2), -1, dtype=torch.int32, device="cuda")
        got = qad.kv_pages_reserve(ints([0, 1, 2, 3]), ints([4]), ints([0] * 3), ints([3, 0, 3]), table, PAGE, tokens)
        assert qad.sync_status() == (0 if tokens == 6 else 8)
        assert got.taken.tolist() == taken and got.lens.tolist() == taken and got.free_count.tolist() == [left]
        assert [x[0] for x in table.tolist()] == [3 if taken[0] else -1, -1, 2 if taken[2] else -1]
        assert got.slots.tolist() == ([48, 49, 50] if taken[0] else [-1] * min(3, tokens)) + ([32, 33, 34] if taken[2] else [-1] * max(0, tokens - 3))


def short_reserve():
    """One page of the two that are wanted."""
    import quantized_attention_diffusion_gb300 as qad
    table = torch.full((2, 1), -1, dtype=torch.int32, device="cuda")
    got = qad.kv_pages_reserve(ints([0, 1]), ints([1]), ints([0, 0]), ints([1, 1]), table, PAGE, 2)
    assert got.taken.tolist() == [1, 0]


def test_too_few_pages_do_not_hide_an_error_that_is_pending():
    import quantized_attention_diffusion_gb300 as qad
    cache = qad.kv_cache_alloc(2, 1, PAGE)
    x = torch.ones((1, 1, 1, 128), dtype=torch.bfloat16, device="cuda")
    short_reserve()
    assert qad.sync_status() == 9 and qad.sync_status() == 0
    qad.kv_cache_append(None, x, x, cache, ints([2 * PAGE]))             # a slot behind the cache
    short_reserve()
    assert qad.sync_status() == 8 and qad.sync_status() == 0
    short_reserve()
    qad.kv_cache_append(None, x, x, cache, ints([2 * PAGE]))             # the graver one is kept, whichever is first
    assert qad.sync_status() == 8 and qad.sync_status() == 0


@pytest.mark.parametrize("free", [5, -1, 2 ** 31 - 1, -2 ** 31])
def test_a_free_count_out_of_range_is_a_bad_page(free):
    import quantized_attention_diffusion_gb300 as qad
    table = torch.full((3, 1), -1, dtype=torch.int32, device="cuda")
    got = qad.kv_pages_reserve(ints([0, 1, 2, 3]), ints([free]), ints([0] * 3), ints([1] * 3), table, PAGE, 3)
    assert qad.sync_status() == 8
    assert got.taken.tolist() == ([1] * 3 if free > 0 else [0] * 3) and got.free_count.tolist() == [1 if free > 0 else 0]


@pytest.mark.parametrize("B,longest,free,bad", [(3, 60, 0, 1), (9, 500, 4, 3), (40, 3000, 17, 40), (1400, 90, 100, 50), (2100, 40, 0, 1), (64, 900, 5, 10 ** 9)])
def test_entries_that_are_no_pages_stay_out_of_the_free_list(B, longest, free, bad):
    import quantized_attention_diffusion_gb300 as qad
    r = random.Random(B)
    lens = [r.randint(1, longest) for _ in range(B)]
    keep = [r.choice([0, 0, r.randint(0, n), n, n + 5, -2]) for n in lens]
    total = sum(pages_of(n) for n in lens)
    pages = list(range(total + free))
    r.shuffle(pages)
    table, at = [], free
    for n in lens:
        table.append(pages[at:at + pages_of(n)] + [-1] * (pages_of(longest) - pages_of(n)))
        at += pages_of(n)
    held = [(b, j) for b, n in enumerate(lens) for j in range(pages_of(n))]
    for b, j in (held if bad >= len(held) else r.sample(held, bad)):
        table[b][j] = r.choice([-1, len(pages), 2 ** 31 - 1, -2 ** 31])
    stack = pages[:free] + [-9] * total

    back, want = [], [list(x) for x in table]
    for b, (n, c) in enumerate(zip(lens, keep)):
        if c < n:
            for j in range(pages_of(max(0, c)), pages_of(n)):
                back.append(table[b][j])
                want[b][j] = -1
    valid = [p for p in back if 0 <= p < len(pages)]
    t = torch.tensor(table, dtype=torch.int32, device="cuda")
    s, f, n = ints(stack), ints([free]), ints(lens)
    qad.kv_pages_release(s, f, n, ints(keep), t, PAGE)
    assert qad.sync_status() == (0 if len(valid) == len(back) else 8)
    assert f.tolist() == [free + len(valid)]
    assert s.tolist()[:free + len(valid)] == pages[:free] + valid[::-1]
    assert s.tolist()[free + len(back):] == stack[free + len(back):]
    assert t.tolist() == want and n.tolist() == [min(a, max(0, b)) for a, b in zip(lens, keep)]

    # and what is reserved next are pages
    room = torch.full((1, max(1, free + len(valid))), -1, dtype=torch.int32, device="cuda")
    count = PAGE * (free + len(valid))
    if count:
        got = qad.kv_pages_reserve(s, f, ints([0]), ints([count]), room, PAGE, count)
        assert qad.sync_status() == 0 and got.taken.tolist() == [count] and got.free_count.tolist() == [0]
        assert sorted(room[0].tolist()) == sorted(pages[:free] + valid)


@pytest.mark.parametrize("table,free,left", [
    ([[1, 9, -1]], 3, [0, 2, 3, 1]),                        # room for one, and one is a page
    ([[9, 1, 7]], 3, [0, 2, 3, 1]),
    ([[-1, -1, -1]], 4, [0, 2, 3, 5]),                      # a full list and a row that has no pages
])
def test_a_list_without_room_for_what_is_no_page(table, free, left):
    import quantized_attention_diffusion_gb300 as qad
    guard = ints([0, 2, 3, 5 if free == 4 else 77, 88])
    pool = guard[:4]
    t, f, n = torch.tensor(table, dtype=torch.int32, device="cuda"), ints([free]), ints([48])
    qad.kv_pages_release(pool, f, n, ints([0]), t, PAGE)
    assert qad.sync_status() == 8
    assert pool.tolist() == left and f.tolist() == [4] and guard[4] == 88 and n.tolist() == [0] and (t == -1).all()


def test_more_pages_than_the_list_has_room_for():
    """A page given back twice: the list is full and holds pages alone."""
    import quantized_attention_diffusion_gb300 as qad
    guard = ints([0, 1, 2, 77, 88, 99])
    t, f, n = ints([3, 2, 1, 0]).view(2, 2), ints([3]), ints([32, 32])
    qad.kv_pages_release(guard[:5], f, n, ints([0, 0]), t, PAGE)
    assert qad.sync_status() == 8
    assert f.tolist() == [5] and guard.tolist()[:3] == [0, 1, 2] and guard[5] == 99
    assert set(guard.tolist()[3:5]) <= {0, 1, 2, 3} and (t == -1).all() and not n.any()
