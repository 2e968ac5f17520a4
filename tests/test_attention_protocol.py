"""The barriers of the attention kernel, on the CPU.

attention_kernel's warps meet only at mbarriers, and a wait knows no more of a
barrier than the parity of its phase: one that is a phase behind, or two ahead,
of what the waiting warp thinks lets it pass at once.  This model runs the
kernel's roles (the warp that finds segments and copies K, the one that copies Q
and V, two issuing warps, the warps of two softmax groups) with the same
barriers, counts, parities and ring arithmetic under random schedules, with
copies that land out of order and products that run late.  What a role reads has
to be what its segment and tile call for, nothing in use is overwritten, and
every run ends.
"""
import collections
import os
import random
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = os.path.join(ROOT, "smc_speculative_decoding_gb300", "csrc", "tree_attention.cu")
PAIR, ALTERNATE, TWO = "pair", "alternate", "two"
WARPS = 2  # of a softmax group: enough for them to be at different tiles


class Wrong(AssertionError):
    pass


def check(truth, *what):
    if not truth:
        raise Wrong(*what)


class Barrier:
    arrivals = 0  # of all barriers: what shows that a run gets on

    def __init__(self, count):
        self.count = self.left = count
        self.phase = 0

    def arrive(self):
        Barrier.arrivals += 1
        self.left -= 1
        if self.left == 0:
            self.left = self.count
            self.phase += 1

    def passed(self, parity):
        return self.phase & 1 != parity


class Ring:
    """Ring in the kernel: the half of the slots for even tiles, and for odd ones."""

    def __init__(self, slots):
        self.half, self.used = slots // 2, [0, 0]

    def at(self, odd):
        return 2 * (self.used[odd] % self.half) + odd

    def parity(self, odd):
        return self.used[odd] // self.half & 1

    def step(self, odd, n=1):
        self.used[odd] += n


class Cta:
    """One CTA's run over `segments`: (kind, tiles, the other's tiles, cut, edges, bad).  edges: the tiles past the
    committed tokens; bad: those of them with a value that is not finite, by the part that a warp scans.
    without: a wait to leave out."""

    def __init__(self, seed, slots_k, slots_v, segments, bulk=True, without=None):
        self.random = random.Random(seed)
        self.segments, self.bulk, self.without = segments, bulk, without
        slots = (slots_k, slots_v)
        self.slots = slots
        self.full = [[Barrier(1) for _ in range(n)] for n in slots]
        self.empty = [[Barrier(2) for _ in range(n)] for n in slots]
        self.data = [[None] * n for n in slots]
        self.bad = [set() for _ in range(slots_v)]
        self.users = [[set() for _ in range(n)] for n in slots]
        self.seg_full = [Barrier(1) for _ in range(4)]
        self.seg_empty = [Barrier(2 * WARPS + 3) for _ in range(4)]
        self.seg = [None] * 4
        self.q_full, self.q_free = [Barrier(1), Barrier(1)], [Barrier(2), Barrier(2)]
        self.q, self.q_users = [None, None], [set(), set()]
        self.scores = [Barrier(1), Barrier(1)]
        self.s_free = [Barrier(WARPS), Barrier(WARPS)]
        self.weights = [[Barrier(WARPS) for _ in range(2)] for _ in range(2)]
        self.o_full = [Barrier(1), Barrier(1)]
        self.o_free, self.stats, self.stored = (Barrier(2 * WARPS) for _ in range(3))
        self.counted = Barrier(1)
        self.s = [None, None]                                # a group's scores: (segment, tile)
        self.p = [[[None] * WARPS for _ in range(2)] for _ in range(2)]  # its weights, by warp
        self.products = [0, 0]                               # done, of either group
        self.o = [None, None]                                # segment of either accumulator
        self.stat = [[None] * WARPS for _ in range(2)]
        self.nonfinite = [None, None]
        self.queue = [collections.deque(), collections.deque()]  # what the tensor core has yet to do
        self.landing = []
        self.clock = 0

    # -- segments
    def halves(self, x):
        """Tiles of segment x in either half of the rings."""
        kind, n, m = self.segments[x][:3]
        return (n, m) if kind == TWO else ((n + 1) // 2, n // 2)

    def own(self, x, g):
        """The tiles of group g."""
        kind, n, m = self.segments[x][:3]
        if kind == PAIR:
            return range(n)
        return range(g, 2 * (m if g else n), 2) if kind == TWO else range(g, n, 2)

    def wait(self, barrier, parity):
        while not barrier.passed(parity):
            yield

    def pause(self):
        """A warp is not issued for a while."""
        for _ in range(self.random.choice([1, 1, 1, 1, 2, 5, 40])):
            yield

    def take(self, x):
        yield from self.wait(self.seg_full[x % 4], x // 4 & 1)
        check(self.seg[x % 4] == x, "segment", self.seg[x % 4], x)

    # -- copies
    def land(self, *what):
        late = self.random.randint(0, 30) if self.random.random() < 0.9 else self.random.randint(0, 600)
        self.landing.append((self.clock + late, *what))

    def copy_tiles(self, kind_of, ring, x):
        kind, n, m = self.segments[x][:3]
        unseen = None
        for turn in range(2 * max(n, m) if kind == TWO else n):
            odd = turn & 1
            if kind == TWO and turn >> 1 >= (m if odd else n):
                continue
            at = ring.at(odd)
            yield from self.wait(self.empty[kind_of][at], ring.parity(odd) ^ 1)
            check(not self.users[kind_of][at], "overwritten in use")
            if kind != PAIR:
                self.empty[kind_of][at].arrive()
            ring.step(odd)
            self.users[kind_of][at] = {0, 1} if kind == PAIR else {odd}
            self.data[kind_of][at] = None
            self.land(kind_of, at, (x, turn))
            yield
            if not self.bulk:  # a tile is announced behind the next one's copies
                if unseen is not None:
                    yield from self.announce(kind_of, *unseen)
                unseen = at, (x, turn)
        if unseen is not None:
            yield from self.announce(kind_of, *unseen)

    def announce(self, kind_of, at, tile):
        while self.data[kind_of][at] != tile:
            yield
        self.full[kind_of][at].arrive()

    def k_warp(self):
        ring = Ring(self.slots[0])
        for x in range(len(self.segments) + 1):
            if x >= 4:
                yield from self.wait(self.seg_empty[x % 4], x // 4 - 1 & 1)
            self.seg[x % 4] = x
            yield
            self.seg_full[x % 4].arrive()
            if x < len(self.segments):
                yield from self.copy_tiles(0, ring, x)

    def v_warp(self):
        ring, q_turn = Ring(self.slots[1]), 0
        for x in range(len(self.segments)):
            yield from self.take(x)
            apart = self.segments[x][0] != ALTERNATE
            for j in range(2 if apart else 1):
                at = q_turn & 1
                if q_turn >= 2:
                    yield from self.wait(self.q_free[at], (q_turn >> 1) - 1 & 1)
                check(not self.q_users[at], "Q overwritten in use")
                self.q_users[at] = {g for g in range(2) if self.own(x, g) and (not apart or g == j)}
                self.q[at] = None
                self.land(2, at, (x, j))
                q_turn += 1
                yield
            yield from self.copy_tiles(1, ring, x)
            self.seg_empty[x % 4].arrive()

    # -- products
    def issuer(self, g):
        ring_k, ring_v = Ring(self.slots[0]), Ring(self.slots[1])
        q_turn = asked = given = 0
        for x in range(len(self.segments)):
            yield from self.take(x)
            self.seg_empty[x % 4].arrive()
            apart = self.segments[x][0] != ALTERNATE
            q_at, q_other = q_turn + (g if apart else 0), q_turn + 1 - g
            q_turn += 2 if apart else 1
            tiles = list(self.own(x, g))
            k0, v0 = list(ring_k.used), list(ring_v.used)

            def ask(i):
                nonlocal asked
                yield from self.wait(self.s_free[g], ~asked & 1)
                at = ring_k.at(i & 1)
                yield from self.wait(self.full[0][at], ring_k.parity(i & 1))
                asked += 1
                ring_k.step(i & 1)
                self.queue[g].append(("scores", x, i, at, q_at & 1))

            def free_q():
                self.queue[g].append(("free", q_at & 1))
                if apart:
                    self.queue[g].append(("free", q_other & 1))

            yield from self.wait(self.q_full[q_at & 1], q_at >> 1 & 1)
            if apart:
                yield from self.wait(self.q_full[q_other & 1], q_other >> 1 & 1)
            if [s[0] for s in self.segments[max(x - 1, 0):x + 1]] == [TWO, PAIR] and self.without != "o_free":
                yield from self.wait(self.o_free, x - 1 & 1)
            if tiles:
                yield from ask(tiles[0])
            if len(tiles) <= 1:
                free_q()
            for j, i in enumerate(tiles):
                if j + 1 < len(tiles):
                    yield from ask(tiles[j + 1])
                    if j + 2 == len(tiles):
                        free_q()
                if j == 0 and x > 0:
                    yield from self.wait(self.o_free, x - 1 & 1)
                at = ring_v.at(i & 1)
                yield from self.wait(self.full[1][at], ring_v.parity(i & 1))
                yield from self.wait(self.weights[g][given & 1], given >> 1 & 1)
                self.queue[g].append(("product", x, i, at, given & 1))
                given += 1
                ring_v.step(i & 1)
                yield
            if not tiles and x > 0:
                yield from self.wait(self.o_free, x - 1 & 1)
            self.queue[g].append(("end",))
            for ring, before in ((ring_k, k0), (ring_v, v0)):
                ring.used = [a + b for a, b in zip(before, self.halves(x))]
            yield

    def tensor_core(self, g):
        do = self.queue[g].popleft()
        if do[0] == "scores":
            _, x, i, at, q_at = do
            check(self.data[0][at] == (x, i), "K", self.data[0][at], x, i)
            check(self.q[q_at] == (x, g if self.segments[x][0] != ALTERNATE else 0), "Q")
            check(self.s[g] is None, "scores overwritten")
            self.s[g] = (x, i)
            self.users[0][at].discard(g)
            self.scores[g].arrive()
            self.empty[0][at].arrive()
        elif do[0] == "product":
            _, x, i, at, buf = do
            check(self.data[1][at] == (x, i), "V", self.data[1][at], x, i)
            check(self.p[g][buf] == [(x, i)] * WARPS, "weights")
            check(self.o[g] in (None, x), "accumulator overwritten")
            self.p[g][buf] = [None] * WARPS
            self.users[1][at].discard(g)
            self.products[g] += 1
            self.o[g] = x
            self.empty[1][at].arrive()
        elif do[0] == "free":
            self.q_users[do[1]].discard(g)
            self.q_free[do[1]].arrive()
        else:
            self.o_full[g].arrive()

    # -- softmax
    def softmax(self, g, w):
        ring = Ring(self.slots[1])
        turn = cuts = 0
        for x in range(len(self.segments)):
            yield from self.take(x)
            kind, n, m, cut, edges, bad = self.segments[x]
            self.seg_empty[x % 4].arrive()
            seg = x + 1
            v0 = list(ring.used)
            last = before = None
            for i in self.own(x, g):
                buf = turn & 1
                yield from self.wait(self.scores[g], buf)
                turn += 1
                check(self.s[g] == (x, i), "scores", self.s[g], x, i)
                if before:
                    yield from self.wait(*before)
                    check(self.products[g] >= turn - 2, "weights' columns in use")
                if self.s_free[g].left == 1:
                    self.s[g] = None  # every warp of the group has its scores
                self.s_free[g].arrive()
                yield from self.pause()
                if last and self.random.random() < 0.5:  # the maximum rises
                    yield from self.wait(*last)
                    check(self.products[g] == turn - 1, "accumulator rescaled ahead of its product")
                check(self.p[g][buf][w] is None, "weights overwritten")
                self.p[g][buf][w] = (x, i)
                yield
                at = ring.at(i & 1)
                if i in edges:
                    yield from self.wait(self.full[1][at], ring.parity(i & 1))
                    check(self.data[1][at] == (x, i), "V before its time", self.data[1][at], x, i)
                    found = w in self.bad[at]
                    self.bad[at].discard(w)
                    yield from self.pause()
                    if found:
                        self.nonfinite[seg & 1] = seg
                self.weights[g][buf].arrive()
                before, last = last, (self.empty[1][at], ring.parity(i & 1))
                ring.step(i & 1)
                yield
            ring.used = [a + b for a, b in zip(v0, self.halves(x))]
            yield from self.wait(self.o_full[g], x & 1)
            if kind == ALTERNATE:
                yield from self.wait(self.o_full[1 - g], x & 1)
            self.stat[g][w] = x
            self.stats.arrive()
            yield
            if kind == ALTERNATE or (kind == PAIR and self.without != "stats"):
                yield from self.wait(self.stats, x & 1)
                check(self.stat == [[x] * WARPS] * 2, "maximum and sum")
            mine = set(self.own(x, g)) if kind != ALTERNATE else set(range(n))
            check(not any(i in mine for i, _ in bad) or self.nonfinite[seg & 1] == seg, "not finite, and unseen")
            for other in range(2) if kind == ALTERNATE else (g,):
                check(not self.own(x, other) or self.o[other] == x, "accumulator")
            if self.o_free.left == 1:
                self.o = [None, None]
            self.o_free.arrive()
            yield
            if cut:
                self.stored.arrive()
                if (g, w) == (0, 0):
                    yield from self.wait(self.stored, cuts & 1)
                    self.counted.arrive()
                yield from self.wait(self.counted, cuts & 1)
                cuts += 1
            yield from self.pause()

    # -- one run
    def step_memory(self):
        when, kind_of, at, tile = self.landing.pop(self.random.randrange(len(self.landing)))
        if when > self.clock:
            self.landing.append((when, kind_of, at, tile))
        elif kind_of == 2:
            self.q[at] = tile
            self.q_full[at].arrive()
        else:
            self.data[kind_of][at] = tile
            if kind_of == 1:
                x, i = tile
                self.bad[at] = {w for j, w in self.segments[x][5] if j == i}
            if self.bulk:
                self.full[kind_of][at].arrive()

    def run(self):
        roles = [self.k_warp(), self.v_warp(), self.issuer(0), self.issuer(1)]
        roles += [self.softmax(g, w) for g in range(2) for w in range(WARPS)]
        pace = [self.random.random() ** 2 + 0.05 for _ in roles]
        live, seen, still = list(range(len(roles))), 0, 0
        while live or self.landing or any(self.queue):
            self.clock += 1
            u = self.random.random()
            if u < 0.25 and self.landing:
                self.step_memory()
            elif u < 0.45:
                g = self.random.randrange(2)
                if self.queue[g]:
                    self.tensor_core(g)
            elif live:
                a = self.random.choices(live, [pace[i] for i in live])[0]
                if next(roles[a], self) is self:  # (a role yields nothing but None)
                    live.remove(a)
            still = still + 1 if seen == Barrier.arrivals else 0
            seen = Barrier.arrivals
            check(still < 40000, "no progress")


def random_segments(r):
    segments = []
    for _ in range(r.randint(1, 10)):
        n = r.choice([1, 1, 2, 3, 4, 5, 7, r.randint(1, 24)])
        kind = r.choice([PAIR, ALTERNATE, TWO, TWO])
        m = max(1, n + r.randint(-3, 3)) if kind == TWO else 0
        count = 2 * max(n, m) if kind == TWO else n
        edges = {i for i in range(count) if r.random() < 0.4}
        bad = {(i, r.randrange(WARPS)) for i in edges if r.random() < 0.3}
        if kind == TWO:  # tiles past a segment's own
            bad = {(i, w) for i, w in bad if i >> 1 < (m if i & 1 else n)}
        segments.append((kind, n, m, kind != TWO and r.random() < 0.5, edges, bad))
    return segments


def ring_sizes():
    """(K, V) slots of heads past 64 wide, and of the others, as the source has them."""
    k, v = map(int, re.search(r"kSlotsK = (\d+) \* \(2 / kHalves\), kSlotsV = (\d+) \* \(2 / kHalves\)",
                              open(SOURCE).read()).groups())
    return [(k, v), (2 * k, 2 * v)]


def failures(seeds, slots, bulk=True, without=None):
    for seed in seeds:
        try:
            Cta(seed, *slots, random_segments(random.Random(seed)), bulk, without).run()
        except Wrong as e:
            yield seed, e.args


@pytest.mark.parametrize("bulk", [True, False])
@pytest.mark.parametrize("wide", [True, False])
def test_every_schedule_reads_what_it_should_and_ends(wide, bulk):
    assert list(failures(range(150), ring_sizes()[0 if wide else 1], bulk)) == []


@pytest.mark.parametrize("without", ["o_free", "stats"])
def test_the_model_sees_a_missing_wait(without):
    assert any(failures(range(1000), ring_sizes()[0], without=without))
