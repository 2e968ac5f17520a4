"""The barriers of the 8-bit cache's attention kernel, on the CPU.

attention8_kernel's warps meet at mbarriers, and a wait knows no more of one
than the parity of its phase.  This model runs the kernel's roles (the warp that
finds segments, copies K and V and prepares a tile's scales; the issuing warp;
eight softmax warps with their vote, a tile's second pass and the maxima raised
between the two) with the barriers, counts, parities and rotating vote words of
the source under random schedules, with copies that land out of order and
products that run late.  What a role reads has to be what its segment and tile
call for, nothing in use is overwritten, all warps learn the same of a vote, and
every run ends.
"""
import collections
import os
import random
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = os.path.join(ROOT, "smc_speculative_decoding_gb300", "csrc", "tree_attention8.cu")
TEXT = open(SOURCE).read()
WARPS, SEGS = 8, 4


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


def counts():
    """Arrivals of a phase of each barrier, as the source sets them up."""
    found = dict(re.findall(r"mbar_init\(&s->(\w+)(?:\[i\])?, (\d+)\)", TEXT))
    return {name: int(n) for name, n in found.items()}


Segment = collections.namedtuple("Segment", "tiles chunks edges bad cut rises")
# edges: tiles past the committed tokens; bad: those with a value that is not finite; rises: {tile: {warp: chunks}} in
# which a warp finds a weight that is too large


class Cta:
    """One CTA's run over `segments`.  without: a wait, or a step, to leave out."""

    def __init__(self, seed, segments, without=None):
        self.random = random.Random(seed)
        self.segments, self.without = segments, without
        n = counts()
        two = lambda name: [Barrier(n[name]), Barrier(n[name])]  # noqa: E731
        self.full, self.empty = [two("k_full"), two("v_full")], [two("k_empty"), two("v_empty")]
        self.s_full = two("s_full")
        self.p_full, self.pv_done, self.q_full, self.o_full, self.o_free, self.group = (
            Barrier(n[name]) for name in ("p_full", "pv_done", "q_full", "o_full", "o_free", "group"))
        self.seg_full = [Barrier(n["seg_full"]) for _ in range(SEGS)]
        self.seg_empty = [Barrier(n["seg_empty"]) for _ in range(SEGS)]
        self.seg = [None] * SEGS
        self.readers = [set() for _ in range(SEGS)]  # of a segment's record
        self.data = [[None, None], [None, None]]     # tiles of K and V in shared memory
        self.users = [[False, False], [False, False]]
        self.scales = [None, None]                   # and their tokens' scales
        self.scale_users = [set(), set()]
        self.q, self.q_reads = [None] * WARPS, 0     # pieces of q; products that are to read them
        self.s, self.s_users = [None, None], [set(), set()]
        self.p = {}                                  # weights by (warp, chunk), and sums in the same place
        self.p_reads = 0
        self.o = None                                # segment and tiles in the accumulator
        self.products = 0                            # done
        self.rise = [0, 0, 0]
        self.votes = []                              # what each vote should come to, and its voters
        self.top = [None] * 2                        # by the warp that resets and reads it
        self.top_readers = set()
        self.maxima = [0, 0]                         # versions, by the warp that writes them
        self.nonfinite = 0
        self.queue, self.landing, self.clock = collections.deque(), [], 0

    def wait(self, barrier, parity):
        while not barrier.passed(parity):
            yield

    def pause(self):
        for _ in range(self.random.choice([1, 1, 1, 1, 2, 5, 40])):
            yield

    # -- segments, copies and scales
    def producer(self):
        tile = 0
        for x in range(len(self.segments) + 1):
            if x >= SEGS:
                yield from self.wait(self.seg_empty[x % SEGS], x // SEGS - 1 & 1)
            check(not self.readers[x % SEGS], "a segment's record overwritten in use")
            self.seg[x % SEGS] = x
            if x < len(self.segments):
                self.readers[x % SEGS] = set(range(WARPS + 1))
            yield
            self.seg_full[x % SEGS].arrive()
            if x == len(self.segments):
                return
            for i in range(self.segments[x].tiles):
                slot, turn = tile & 1, tile >> 1 & 1
                for which in range(2):
                    yield from self.wait(self.empty[which][slot], turn ^ 1)
                    check(not self.users[which][slot], "a tile overwritten in use", which)
                    self.users[which][slot] = True
                    self.data[which][slot] = None
                    late = self.random.randint(0, 30) if self.random.random() < 0.9 else self.random.randint(0, 600)
                    self.landing.append((self.clock + late, which, slot, (x, i)))
                    yield
                check(not self.scale_users[slot], "scales overwritten in use")
                self.scales[slot] = (x, i)
                self.scale_users[slot] = set(range(WARPS))
                yield
                self.s_full[slot].arrive()
                tile += 1
                yield

    # -- products
    def issuer(self):
        tile = 0
        for x, seg in enumerate(self.segments):
            yield from self.wait(self.seg_full[x % SEGS], x // SEGS & 1)
            check(self.seg[x % SEGS] == x, "segment")
            self.readers[x % SEGS].discard(WARPS)
            self.seg_empty[x % SEGS].arrive()
            yield from self.wait(self.q_full, x & 1)
            for i in range(seg.tiles + 1):
                if i < seg.tiles:
                    at = tile + i & 1
                    yield from self.wait(self.full[0][at], tile + i >> 1 & 1)
                    self.q_reads += 1
                    self.queue.append(("scores", x, i, at))
                    yield
                if i == 0:
                    continue
                last = tile + i - 1
                at = last & 1
                if i == 1 and x > 0:
                    yield from self.wait(self.o_free, x - 1 & 1)
                yield from self.wait(self.full[1][at], last >> 1 & 1)
                if self.without != "p_full":
                    yield from self.wait(self.p_full, last & 1)
                self.p_reads += 1
                self.queue.append(("product", x, i - 1, at))
                yield
            self.queue.append(("end", x))
            tile += seg.tiles

    def tensor_core(self):
        what, x, *rest = self.queue.popleft()
        if what == "scores":
            i, at = rest
            check(self.data[0][at] == (x, i), "K", self.data[0][at], x, i)
            check(self.q == [x] * WARPS, "pieces of q", self.q, x)
            check(not self.s_users[at], "scores overwritten in use")
            self.s[at], self.s_users[at] = (x, i), set(range(WARPS))
            self.q_reads -= 1
            self.users[0][at] = False
            self.s_full[at].arrive()
            self.empty[0][at].arrive()
        elif what == "product":
            i, at = rest
            check(self.data[1][at] == (x, i), "V", self.data[1][at], x, i)
            for w in range(WARPS):
                for cb in range(w >> 2, self.segments[x].chunks, 2):
                    check(self.p.get((w, cb)) == (x, i, self.passes(x, i, cb)), "weights", self.p.get((w, cb)), x, i)
            check(self.o == ((x, i - 1) if i else None), "accumulator", self.o, x, i)
            self.o = (x, i)
            self.p_reads -= 1
            self.products += 1
            self.users[1][at] = False
            self.empty[1][at].arrive()
            self.pv_done.arrive()
        else:
            self.o_full.arrive()

    def passes(self, x, i, cb):
        """How often a chunk's weights of a tile are written."""
        over = set().union(*self.segments[x].rises.get(i, {}).values()) if i else set()
        return 2 if cb in over else 1

    # -- softmax
    def softmax(self, w):
        half = w >> 2
        turns = votes = voted = tile = 0

        def meet():
            nonlocal turns
            self.group.arrive()
            turns += 1
            if self.without != "group":
                yield from self.wait(self.group, turns - 1 & 1)

        def vote(mine):
            """group_or: the union, as this warp reads it."""
            nonlocal turns, votes, voted
            if voted == len(self.votes):
                self.votes.append([0, 0])
            self.votes[voted][0] |= mine
            self.votes[voted][1] += 1
            self.rise[votes] |= mine
            yield
            self.group.arrive()
            turns += 1
            yield from self.wait(self.group, turns - 1 & 1)
            yield
            union = self.rise[votes]
            check(self.votes[voted] == [union, WARPS], "vote", union, self.votes[voted])
            voted += 1
            votes = 0 if votes == 2 else votes + 1
            if w == 0:
                self.rise[0 if votes == 2 else votes + 1] = 0
            return union

        for x, seg in enumerate(self.segments):
            yield from self.wait(self.seg_full[x % SEGS], x // SEGS & 1)
            check(self.seg[x % SEGS] == x, "segment")
            mine = list(range(half, seg.chunks, 2))
            check(self.q_reads == 0, "pieces of q overwritten in use")
            self.q[w] = x
            yield
            self.q_full.arrive()
            yield from meet()
            for i in range(seg.tiles):
                buf = tile & 1
                yield from self.wait(self.s_full[buf], tile >> 1 & 1)
                check(self.s[buf] == (x, i) and self.scales[buf] == (x, i), "scores", self.s[buf], self.scales[buf], x, i)
                todo, known, again = set(range(4)), i > 0, False
                while True:
                    if known:
                        waited = False
                        for cb in mine:
                            if cb not in todo:
                                continue
                            check(self.s[buf] == (x, i), "scores gone")
                            if cb == half and tile > 0 and not waited and self.without != "pv_done":
                                yield from self.wait(self.pv_done, tile - 1 & 1)
                                waited = True
                            check(self.products >= tile and self.p_reads == 0, "weights overwritten in use")
                            passes = self.p[w, cb][2] + 1 if self.p.get((w, cb), (0,))[:2] == (x, i) else 1
                            self.p[w, cb] = (x, i, passes)
                            yield from self.pause()
                        if i in seg.edges:
                            yield from self.wait(self.full[1][buf], tile >> 1 & 1)
                            check(self.data[1][buf] == (x, i), "V before its time", self.data[1][buf], x, i)
                            if i in seg.bad and w == (x + i) % WARPS:
                                self.nonfinite = x + 1
                        over = seg.rises.get(i, {}).get(w, set()) if i and not again else set()
                        bits = sum(1 << cb for cb in over)
                        union = yield from vote(bits)
                        todo = {cb for cb in range(4) if union >> cb & 1}
                        if not todo:
                            break
                        again = True
                    if w < 2:
                        check(not self.top_readers, "factors overwritten in use")
                        self.top[w] = ("reset", x, i)
                    yield from meet()
                    check(self.top == [("reset", x, i)] * 2, "maxima", self.top)
                    check(self.s[buf] == (x, i), "scores gone")
                    before = list(self.maxima)
                    yield from self.pause()
                    check(self.maxima == before, "maxima change as they are read")
                    yield from meet()
                    if w < 2:
                        self.maxima[w] += 1
                        self.top[w] = ("factor", x, i)
                        if i > 0:
                            self.top_readers |= set(range(WARPS))
                    yield from meet()
                    if i > 0:
                        check(self.top == [("factor", x, i)] * 2, "factors", self.top)
                        check(self.products == tile and self.p_reads == 0, "accumulator rescaled beside a product")
                        yield from self.pause()
                        self.top_readers.discard(w)
                    known = True
                # by the vote all have read the tile's scores and scales: one arrival stands for all of them
                if self.s[buf] == (x, i):
                    self.s_users[buf].clear()
                if self.scales[buf] == (x, i):
                    self.scale_users[buf].clear()
                if w == 0:
                    self.p_full.arrive()
                tile += 1
                yield
            yield from self.wait(self.o_full, x & 1)
            check(self.products == tile and self.p_reads == 0, "the weights' place is in use")
            for cb in mine:
                self.p[w, cb] = ("sums", x)
            yield from meet()
            for v in range(WARPS):
                for cb in range(v >> 2, seg.chunks, 2):
                    check(self.p[v, cb] == ("sums", x), "sums", self.p[v, cb], x)
            yield from meet()
            bad = self.nonfinite == x + 1
            check(bad == any(i in seg.edges for i in seg.bad), "not finite", self.nonfinite, x)
            check(self.o == (x, seg.tiles - 1), "accumulator", self.o, x)
            yield from self.pause()
            check(self.o == (x, seg.tiles - 1), "accumulator gone", self.o, x)
            if self.o_free.left == 1:
                self.o = None
            self.o_free.arrive()
            yield
            if bad:
                yield from meet()
            if seg.cut:
                yield from meet()
                yield from meet()
            for cb in mine:
                check(self.p[w, cb] == ("sums", x), "addresses overwritten in use")
            self.readers[x % SEGS].discard(w)
            self.seg_empty[x % SEGS].arrive()
            yield from self.pause()

    # -- one run
    def land(self):
        item = self.landing.pop(self.random.randrange(len(self.landing)))
        if item[0] > self.clock:
            self.landing.append(item)
            return
        _, which, slot, tile = item
        self.data[which][slot] = tile
        self.full[which][slot].arrive()

    def run(self):
        roles = [self.producer(), self.issuer(), *(self.softmax(w) for w in range(WARPS))]
        pace = [self.random.random() ** 2 + 0.05 for _ in roles]
        live, seen, still = list(range(len(roles))), 0, 0
        while live or self.landing or self.queue:
            self.clock += 1
            u = self.random.random()
            if u < 0.2 and self.landing:
                self.land()
            elif u < 0.35 and self.queue:
                self.tensor_core()
            elif live:
                a = self.random.choices(live, [pace[i] for i in live])[0]
                if next(roles[a], self) is self:  # (a role yields nothing but None)
                    live.remove(a)
            still = still + 1 if seen == Barrier.arrivals else 0
            seen = Barrier.arrivals
            check(still < 40000, "no progress")


def random_segments(r):
    segments = []
    for _ in range(r.randint(1, 9)):
        tiles, chunks = r.choice([1, 1, 2, 3, 4, r.randint(1, 9)]), r.randint(1, 4)
        edges = {i for i in range(tiles) if r.random() < 0.4}
        bad = {i for i in edges if r.random() < 0.2}
        rises = {}
        for i in range(tiles):
            if r.random() < 0.4:
                rises[i] = {w: {cb for cb in range(w >> 2, chunks, 2) if r.random() < 0.4} for w in range(WARPS)
                            if r.random() < 0.4}
        segments.append(Segment(tiles, chunks, edges, bad, r.random() < 0.3, rises))
    return segments


def failures(seeds, without=None):
    for seed in seeds:
        try:
            Cta(seed, random_segments(random.Random(seed)), without).run()
        except Wrong as e:
            yield seed, e.args


def test_the_source_has_the_barriers_of_the_model():
    assert counts() == {"k_full": 1, "k_empty": 1, "v_full": 1, "v_empty": 1, "s_full": 2, "p_full": 1, "pv_done": 1,
                        "q_full": WARPS, "o_full": 1, "o_free": WARPS, "drained": 1, "group": WARPS, "seg_full": 1,
                        "seg_empty": WARPS + 1}
    assert f"constexpr int kSegs8 = {SEGS};" in TEXT
    # every bounded wait and its parity
    for wait in ["&s->pv_done, (tile - 1) & 1u", "&s->s_full[buf], tile >> 1 & 1u", "&s->o_full, (seg - 1) & 1u",
                 "&s->group, (turns - 1) & 1u", "&s->q_full, seg & 1u", "&s->k_full[at], (tile + i) >> 1 & 1u",
                 "&s->o_free, (seg - 1) & 1u", "&s->v_full[at], last >> 1 & 1u", "&s->p_full, last & 1u",
                 "&s->seg_empty[seg % kSegs8], (seg / kSegs8 - 1) & 1u", "&s->seg_full[seg % kSegs8], seg / kSegs8 & 1u"]:
        assert wait in TEXT, wait


def test_every_schedule_reads_what_it_should_and_ends():
    assert list(failures(range(80))) == []


@pytest.mark.parametrize("without", ["p_full", "pv_done", "group"])
def test_the_model_sees_a_missing_wait(without):
    assert any(failures(range(300), without=without))
