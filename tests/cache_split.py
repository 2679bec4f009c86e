"""How the cache attention's wide kernel cuts its work up, and a model of its warps
and barriers (no test functions here).

A segment is (tiles, by_rows): the key tiles of one unit that a CTA has, and whether
the unit has more than 128 query rows.
"""
import random

WIDE_ROWS, WIDE_TOK, WIDE_COST, SMS = 256, 128, 3, 152

# Ragged batches over roomy tables, many heads, 17 to 128 query rows to a key/value
# head: some CTA gets three or more segments of one tile and then a longer one.
# B, longest, Sq, H, G, seed
RAGGED = [(48, 700, 16, 16, 4, 1), (40, 700, 31, 16, 1, 7), (48, 500, 12, 16, 2, 7), (24, 2000, 17, 8, 1, 3), (24, 1000, 24, 16, 1, 1), (32, 400, 20, 16, 1, 0)]


def ragged_lens(B, longest, seed):
    r = random.Random(seed)
    return [r.randint(0, longest) for _ in range(B)]


def segments(lens, rows, H, Sq, G, causal=True, ctas=SMS):
    """For each CTA of a launch over full tables its segments, in order."""
    row_tiles = -(-rows // WIDE_ROWS)
    steps, at = [], 0                  # (first step, tiles, by_rows) of each unit
    for n in lens:
        for rt in range(row_tiles):
            last = min(rows, (rt + 1) * WIDE_ROWS) - 1
            keys = max(0, min(n, n - Sq + last // G + 1)) if causal else n
            tiles = max(1, -(-keys // WIDE_TOK))
            for _ in range(H):
                steps.append((at, tiles, rows - rt * WIDE_ROWS > 128))
                at += WIDE_COST + tiles
    per = -(-at // ctas)
    out = [[] for _ in range(ctas)]
    for first, tiles, by_rows in steps:
        t0 = first + WIDE_COST
        for c in range(t0 // per, (t0 + tiles - 1) // per + 1):
            n = min(t0 + tiles, (c + 1) * per) - max(t0, c * per)
            out[c].append((n, by_rows))
    return out


class Stale(AssertionError):
    """A role has read what was not there yet, or not any more."""


class Stuck(AssertionError):
    """No role can go on."""


class Barrier:
    def __init__(self, count):
        self.count, self.left, self.phase = count, count, 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left, self.phase = self.count, self.phase + 1

    def over(self, parity):            # as try_wait.parity: the phase of this parity has ended
        return (self.phase & 1) != (parity & 1)


SLOTS = 4


class Wide:
    """The roles of one CTA: converters of K and V, the issuing threads of both products
    of both halves, the tensor core behind each, the softmax of both halves.  A role is
    a generator that yields the barriers it waits for."""

    def __init__(self, segs, scores_wait):
        self.segs, self.scores_wait = segs, scores_wait
        self.tiles = [(i, j, n, by_rows) for i, (n, by_rows) in enumerate(segs) for j in range(n)]
        B = Barrier
        self.full = {o: [B(1), B(1)] for o in "kv"}
        self.empty = {o: [B(2), B(2)] for o in "kv"}
        self.scales = [B(2) for _ in range(SLOTS)]
        self.q_full = [B(1) for _ in range(3)]
        self.half_full, self.half_read = B(1), B(1)
        self.s_full, self.p_full, self.pv_done = ([[B(1), B(1)] for _ in range(2)] for _ in range(3))
        self.stage = {o: [None, None] for o in "kv"}           # the tile in a stage
        self.scale = {o: [None] * SLOTS for o in "kv"}         # the tile whose scales a slot has
        self.q_of = [None, None]                               # the segment whose queries a Q tile has
        self.scores = [[None, None], [None, None]]             # [half][buffer]: (tile, weights?)
        self.queue = [[] for _ in range(4)]                    # products and commits of each issuing thread

    def convert(self, o):
        for it in range(len(self.tiles)):
            if o == "v":
                self.scale[o][it % SLOTS] = it
                self.scales[it % SLOTS].arrive()
                yield None
            if it >= 2:
                yield self.empty[o][it & 1], it // 2 - 1
            if o == "k":
                self.scale[o][it % SLOTS] = it
                self.scales[it % SLOTS].arrive()
                yield None
            self.stage[o][it & 1] = it
            self.full[o][it & 1].arrive()
            yield None

    def issue(self, t, is_pv):
        o, q = ("v", 2 + t) if is_pv else ("k", t)
        done = seen = seen_odd = 0
        for g, (seg, j, n, by_rows) in enumerate(self.tiles):
            s = g & 1
            yield self.full[o][s], g // 2
            if not is_pv and self.scores_wait and g >= 2:
                yield self.scales[(g - 2) % SLOTS], (g - 2) // SLOTS
            if not is_pv and j == 0:
                if t == 0 or by_rows:
                    yield self.q_full[t], seen
                    seen += 1
                elif n > 1:
                    yield self.q_full[2], seen_odd
                    seen_odd += 1
            if not by_rows and j & 1 != t:
                if not is_pv and n == 1 and done > 0:
                    yield self.pv_done[t][(done - 1) & 1], (done - 1) // 2
                self.empty[o][s].arrive()
                yield None
                continue
            for sub in range(2):
                if is_pv:
                    yield self.p_full[t][sub], done // 2
                elif done >= 2:
                    yield self.pv_done[t][sub], (done - 2) // 2
                self.queue[q].append(("mul", is_pv, t, sub, g, seg, by_rows))
                self.queue[q].append(("commit", self.pv_done[t][sub] if is_pv else self.s_full[t][sub]))
                done += 1
                yield None
            self.queue[q].append(("commit", self.empty[o][s]))

    def core(self, q):                 # the products of one thread, in order
        while True:
            while not self.queue[q]:
                yield "idle"
            what = self.queue[q].pop(0)
            if what[0] == "commit":
                what[1].arrive()
            else:
                _, is_pv, t, sub, g, seg, by_rows = what
                if self.stage["v" if is_pv else "k"][g & 1] != g:
                    raise Stale(f"product of tile {g}: its stage has another tile")
                if is_pv:
                    if self.scores[t][sub] != (g, True):
                        raise Stale(f"product of tile {g}: no weights")
                else:
                    if self.q_of[t if by_rows else 0] != seg:
                        raise Stale(f"scores of tile {g}: another segment's queries")
                    self.scores[t][sub] = (g, False)
            yield None

    def softmax(self, t):
        it = done = joined = 0
        for seg, (n, by_rows) in enumerate(self.segs):
            if by_rows or t < n:
                if by_rows or t == 0:
                    self.q_of[t] = seg
                    self.q_full[t].arrive()
                    yield None
                    if not by_rows and n > 1:
                        self.q_full[2].arrive()
                        yield None
                nv = 2 * (n if by_rows else (n - t + 1) // 2)
                for v in range(nv):
                    j = v // 2 if by_rows else (v & ~1) + t
                    tile, slot = it + j, (it + j) % SLOTS
                    waits = [(self.scales[slot], tile // SLOTS), (self.s_full[t][v & 1], (done + v) // 2)]
                    for w in reversed(waits) if self.scores_wait else waits:
                        yield w
                    for _ in range(2):                          # the buffer's two halves
                        if self.scores[t][v & 1] != (tile, False):
                            raise Stale(f"half {t}, tile {tile}: another tile's scores")
                        if self.scale["k"][slot] != tile or self.scale["v"][slot] != tile:
                            raise Stale(f"half {t}, tile {tile}: scales of {self.scale['k'][slot]} and {self.scale['v'][slot]}")
                        yield None
                    if v > 0 and tile % 3 == 0:                 # the row's references move
                        yield self.pv_done[t][(v - 1) & 1], (done + v - 1) // 2
                    self.scores[t][v & 1] = (tile, True)
                    self.p_full[t][v & 1].arrive()
                    yield None
                yield self.pv_done[t][(nv - 1) & 1], (done + nv - 1) // 2
                done += nv
                if not by_rows and n > 1:
                    for _ in range(2):
                        if t == 1:
                            self.q_of[1] = None                 # the exchange stands in the second Q tile
                            self.half_full.arrive()
                            yield self.half_read, joined
                        else:
                            yield self.half_full, joined
                            self.half_read.arrive()
                            yield None
                        joined += 1
            it += n

    def run(self, rng, slow=()):
        """One schedule: a random role at a time, those named in `slow` seldom."""
        roles = {"convert k": self.convert("k"), "convert v": self.convert("v")}
        for t in range(2):
            roles[f"scores {t}"] = self.issue(t, False)
            roles[f"sums {t}"] = self.issue(t, True)
            roles[f"softmax {t}"] = self.softmax(t)
        cores = {f"core {q}": self.core(q) for q in range(4)}
        at = dict.fromkeys(roles)
        while roles:
            ready = [k for k in roles if at[k] is None or at[k][0].over(at[k][1])]
            ready += [k for k in cores if self.queue[int(k[-1])]]
            if not ready:
                raise Stuck(", ".join(roles))
            quick = [k for k in ready if k not in slow]
            k = rng.choice(quick if quick and rng.random() < 0.99 else ready)
            if k in cores:
                next(cores[k])
                continue
            try:
                at[k] = next(roles[k])
            except StopIteration:
                del roles[k]


ROLES = ("convert k", "convert v", "scores 0", "scores 1", "sums 0", "sums 1", "softmax 0", "softmax 1",
         "core 0", "core 1", "core 2", "core 3")


def schedules(segs, scores_wait, count, seed):
    """`count` schedules of one CTA, none, one or two roles slow in each."""
    rng = random.Random(seed)
    for _ in range(count):
        Wide(segs, scores_wait).run(rng, rng.sample(ROLES, rng.randint(0, 2)))
