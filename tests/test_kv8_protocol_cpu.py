"""The barrier protocol of the many-row attention kernel (csrc/kv8_prompt.cu), played on the CPU with random delays.

Every role is a generator that waits, arrives, reads and writes in the kernel's order; ring sizes and arrival counts are
read from the source.  A barrier answers a wait by its phase's parity, as the hardware does, so a wait that could pass
on another phase than its own is an error here; so is a slot, tile or place that is not what its reader expects, at
the start or at the end of the reading, and a role that never ends.
"""
import heapq
import os
import random
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "slot_decode_window_gb300", "csrc",
                      "kv8_prompt.cu")


def constants():
    text = open(SOURCE).read()
    c = {n: eval(re.search(r"constexpr int %s = ([\d +]+);" % n, text)[1]) for n in ("kSegs", "kRawStages", "kScores", "kSegReaders")}
    for n in ("kVStages", "kVParts"):
        a, b = re.search(r"%s = TWO \? (\d) : (\d);" % n, text).groups()
        c[n] = (int(b), int(a))
    c["kRawBars"] = int(re.search(r"kRawBars = (\d) \* kRawStages;", text)[1])
    count = {}
    for name, two, n in re.findall(r"mbar_init\(&?(\w+)(?:\[\w\])?, (TWO \? \d : )?(\w+)\)", text):
        n = c["kSegReaders"] if n == "kSegReaders" else int(n)
        count[name] = (n, int(re.search(r"\d", two)[0]) if two else n)
    c["count"] = count
    c["stats"] = int(re.search(r"kStats = .*// \[(\d)\]\[128\]", text)[1])
    c["rf"] = int(re.search(r"kRf = .*// \[(\d)\]\[128\]", text)[1])
    c["factors"] = int(re.search(r"kExp = .*// \[(\d)\]\[8\]", text)[1])
    return c


class Bar:
    def __init__(self, count):
        self.count, self.phase, self.n = count, 0, 0

    def arrive(self):
        self.n += 1
        assert self.n <= self.count
        if self.n == self.count:
            self.n, self.phase = 0, self.phase + 1


class Machine:
    """Generators yield ("wait", barrier, phase), ("arrive", barrier), ("work", mean), ("async", queue, mean, then)."""

    def __init__(self, seed):
        self.r, self.bars, self.mem = random.Random(seed), {}, {}
        self.events, self.order, self.now, self.queue_end, self.waiting, self.groups = [], 0, 0.0, {}, {}, {}

    def push(self, delay, fn):
        heapq.heappush(self.events, (self.now + delay, self.order, fn))
        self.order += 1

    def arrive(self, bar):
        b = self.bars[bar]
        b.arrive()
        for role, phase in [w for w in self.waiting.get(bar, [])]:
            if b.phase == phase + 1:
                self.waiting[bar].remove((role, phase))
                self.push(self.r.random(), lambda role=role: self.step(role))

    def expect(self, where, what):
        assert self.mem.get(where) == what, (where, self.mem.get(where), what)

    def step(self, role):
        try:
            x = next(role)
        except StopIteration:
            self.live -= 1
            return
        go = lambda: self.step(role)
        if x[0] == "wait":
            b = self.bars[x[1]]
            assert b.phase in (x[2], x[2] + 1), ("a wait for phase %d meets phase %d" % (x[2], b.phase), x[1])
            if b.phase == x[2] + 1:
                self.push(self.r.random(), go)
            else:
                self.waiting.setdefault(x[1], []).append((role, x[2]))
        elif x[0] == "arrive":
            self.arrive(x[1])
            self.push(0.1 * self.r.random(), go)
        elif x[0] == "work":
            self.push(self.r.expovariate(1 / (x[1] * self.r.choice([0.2, 1, 6]))), go)
        elif x[0] == "async":  # in order within a queue
            end = max(self.queue_end.get(x[1], 0.0), self.now) + self.r.expovariate(1 / x[2])
            self.queue_end[x[1]] = end
            self.push(end - self.now, x[3])
            self.push(0.1, go)
        elif x[0] == "meet":  # a barrier of some of the roles
            g = self.groups.setdefault(x[1], [])
            g.append(role)
            if len(g) == x[2]:
                self.groups[x[1]] = []
                for other in g:
                    self.push(self.r.random(), lambda other=other: self.step(other))

    def run(self, roles):
        self.live = len(roles)
        for role in roles:
            self.push(self.r.random(), lambda role=role: self.step(role))
        while self.events:
            self.now, _, fn = heapq.heappop(self.events)
            fn()
        assert self.live == 0, ("stuck", {b: w for b, w in self.waiting.items() if w})


def play(units, two, seed, raw_bars=None):
    """units: of each segment of a CTA's part of the list.  raw_bars: barriers of a side's copies, if not the kernel's."""
    c = constants()
    m = Machine(seed)
    places, stages, segs = c["kScores"], c["kRawStages"], c["kSegs"]
    vst, vparts = c["kVStages"][two], c["kVParts"][two]
    raws = raw_bars or c["kRawBars"] * stages
    size = dict(raw_full=raws, raw_empty=raws, k_full=2, k_empty=2, v_full=4, v_empty=4, s_full=places,
                p_full=places, place_free=places, u_full=1, u_empty=1, q_full=1, q_empty=1, seg_full=segs, seg_empty=segs)
    for name, n in size.items():
        for i in range(n):
            for side in ("K", "V") if name.startswith("raw") else ("",):
                m.bars[name, side, i] = Bar(c["count"][name][two])
    ends, total = [sum(units[:i + 1]) for i in range(len(units))], sum(units)
    begin = [0] + ends[:-1]

    def bar(name, i=0, side=""):
        return (name, side, i)

    def wait(name, number, ring, side=""):
        """For use `number` of a ring of barriers."""
        return "wait", bar(name, number % ring, side), number // ring

    def seg_wait(i):
        return wait("seg_full", i, segs)

    def seg_done(i):
        m.expect(("seg", i % segs), i)
        return "arrive", bar("seg_empty", i % segs)

    def copies(side):
        h = 0
        for i, n in enumerate(units):
            if side == "K":
                if i >= segs:
                    yield wait("seg_empty", i - segs, segs)
                m.mem["seg", i % segs] = i
                yield "arrive", bar("seg_full", i % segs)
            else:
                yield seg_wait(i)
            for _ in range(2 * n):
                if h >= stages:
                    yield wait("raw_empty", h - stages, raws, side)

                def land(h=h):
                    m.mem["raw", side, h % stages] = h
                    m.arrive(bar("raw_full", h % raws, side))
                m.mem["raw", side, h % stages] = None
                yield "async", ("tma", side, h), 20, land
                h += 1
            yield seg_done(i)

    def convert(side, w):
        half = w >> 1
        for i, n in enumerate(units):
            yield seg_wait(i)
            if side == "K":
                if i > 0:
                    yield wait("q_empty", i - 1, 1)
                m.mem["q", w] = m.mem["rf", i % c["rf"], w] = i
                yield "work", 8
                yield "arrive", bar("q_full")
            for at in range(begin[i], ends[i]):
                st = at % (vst if side == "V" else 2)
                if side == "K" and at >= 2:
                    yield wait("k_empty", at - 2, 2)
                elif side == "V" and at >= vst:
                    yield wait("v_empty", at - vst, vst) if not two else ("wait", bar("v_empty", half), at - 1)
                if side == "K" and w == 0:
                    m.mem["factors", at % c["factors"]] = at
                h = 2 * at + half
                yield wait("raw_full", h, raws, side)
                m.expect(("raw", side, h % stages), h)
                yield "work", 1
                m.expect(("raw", side, h % stages), h)
                yield "arrive", bar("raw_empty", h % raws, side)
                m.mem["tile", side, st, w] = None
                yield "work", 6
                m.mem["tile", side, st, w] = at
                yield "arrive", bar("k_full", st) if side == "K" else bar("v_full", half if two else st)
            yield seg_done(i)

    def products_s():
        for i in range(len(units)):
            yield seg_wait(i)
            yield seg_done(i)
            yield wait("q_full", i, 1)
            for at in range(begin[i], ends[i]):
                if at >= places:
                    yield wait("place_free", at - places, places)
                yield wait("k_full", at, 2)

                def look(at=at, i=i):
                    for w in range(4):
                        m.expect(("tile", "K", at % 2, w), at)
                        m.expect(("q", w), i)

                def done(at=at, i=i, look=look):
                    look()
                    for w in range(4):
                        m.mem["place", at % places, w] = ("S", at)
                    m.arrive(bar("s_full", at % places))
                    m.arrive(bar("k_empty", at % 2))
                    if at + 1 == ends[i]:
                        m.arrive(bar("q_empty"))
                look()
                for w in range(4):
                    m.mem["place", at % places, w] = None
                yield "async", "S", 8, done

    def products_u():
        for at in range(total):
            yield wait("p_full", at, places)
            if at >= 1:
                yield wait("u_empty", at - 1, 1)
            for part in range(vparts):
                v = part if two else at % vst
                yield ("wait", bar("v_full", v), at if two else at // vst)
                mine = [w for w in range(4) if not two or w >> 1 == part]

                def look(at=at, mine=mine):
                    for w in mine:
                        m.expect(("tile", "V", at % vst, w), at)
                    for w in range(4):
                        m.expect(("place", at % places, w), ("P", at))

                def done(at=at, part=part, v=v, look=look):
                    look()
                    if part == vparts - 1:
                        m.mem["u"] = at
                        m.arrive(bar("u_full"))
                        m.arrive(bar("place_free", at % places))
                    m.arrive(bar("v_empty", v))
                look()
                m.mem["u"] = None
                yield "async", "U", 8, done

    def softmax(odd, w):
        for i in range(len(units)):
            yield seg_wait(i)
            first = True
            for at in range(begin[i], ends[i]):
                if at & 1 != odd:
                    continue
                yield wait("s_full", at, places)
                if first:
                    m.expect(("rf", i % c["rf"], w), i)
                    first = False
                for _ in range(2):
                    m.expect(("place", at % places, w), ("S", at))
                    m.expect(("factors", at % c["factors"]), at)
                    yield "work", 10
                m.expect(("place", at % places, w), ("S", at))
                m.expect(("factors", at % c["factors"]), at)
                m.mem["place", at % places, w] = ("P", at)
                m.mem["stats", at % c["stats"], w] = at
                yield "arrive", bar("p_full", at % places)
            yield seg_done(i)

    def correction(w):
        for i in range(len(units)):
            yield seg_wait(i)
            yield "meet", "correction", 4
            for at in range(begin[i], ends[i]):
                yield wait("u_full", at, 1)
                m.expect(("stats", at % c["stats"], w), at)
                m.expect("u", at)
                yield "work", 4
                m.expect("u", at)
                yield "arrive", bar("u_empty")
                yield "work", 4
            yield seg_done(i)

    m.run([copies("K"), copies("V"), products_s(), products_u()] + [convert(s, w) for s in "KV" for w in range(4)] +
          [softmax(o, w) for o in range(2) for w in range(4)] + [correction(w) for w in range(4)])


@pytest.mark.parametrize("two", [0, 1])
@pytest.mark.parametrize("mix", [[1], [1, 1, 2], [3, 5, 9], [30]])
def test_every_wait_meets_its_own_phase(two, mix):
    r = random.Random(len(mix))
    for seed in range(40):
        play([r.choice(mix) for _ in range(r.choice([1, 2, 12, 25]) if max(mix) < 30 else 2)], two, seed)


@pytest.mark.parametrize("two", [0, 1])
def test_the_play_finds_barriers_shared_by_the_halves(two):
    """What it is for: with one barrier a stage for the copies of both halves, whose warps each skip the other's phases,
    a wait can meet an earlier phase of the same parity."""
    with pytest.raises(AssertionError, match="a wait for phase"):
        for seed in range(40):
            play([9, 9], two, seed, raw_bars=constants()["kRawStages"])
