"""The barriers of the tensor-core attention kernel (attn_tc.cu), restated: warps that load, look at values, issue the
MMAs of two streams and take their exponentials, over units of one and of two tiles in any order. Under random schedules
no warp waits for ever, and none takes a block, a product or a statistic of another step for its own. Barriers are told
apart by their phase's parity alone, as on the device; MMAs of a warp end in order, copies in any order."""
import random

import pytest


class Barrier:
    def __init__(self, count):
        self.count, self.phase, self.left = count, 0, count

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.phase, self.left = self.phase + 1, self.count

    def done(self, parity):
        return (self.phase & 1) != (parity & 1)


def first(unit, pos, t):
    """Stream t's first block of a unit (blocks, two tiles) that begins at block `pos` of the CTA; its step is 1 or 2."""
    return 0 if unit[1] else (pos ^ t) & 1


class Cta:
    def __init__(self, units, slots):
        pair = lambda n=1: [Barrier(n), Barrier(n)]                          # noqa: E731
        ring = lambda n: [Barrier(n) for _ in range(slots)]                  # noqa: E731
        self.units, self.slots = units, slots
        self.kfull, self.kfree, self.vfull, self.vfree, self.fixed = ring(1), ring(2), ring(1), ring(2), ring(1)
        self.qfull, self.qfree, self.sfull, self.pfull, self.ofull, self.go = pair(), pair(), pair(), pair(), pair(), pair()
        self.mfull, self.mfree, self.reached = Barrier(1), Barrier(1), [0, 0]
        self.k, self.v, self.q, self.s, self.p, self.o, self.stats = [None] * slots, [None] * slots, [None] * 2, [None] * 2, [None] * 2, [None] * 2, None
        self.copies, self.mmas = [], [[], []]

    def copy(self, where, i, what, bar):
        def end():
            where[i] = what
            bar.arrive()
        where[i] = None
        self.copies.append(end)

    def keys(self):
        n, alone, pos, used = 0, False, 0, [0, 0]
        for u, unit in enumerate(self.units):
            for b in range(unit[0]):
                slot, phase = n % self.slots, n // self.slots
                while not self.kfree[slot].done(phase + 1):
                    yield False
                self.copy(self.k, slot, (u, b), self.kfull[slot])
                n += 1
                if b != (0 if alone else min(1, unit[0] - 1)):
                    continue
                for t in (0, 1):
                    if first(unit, pos, t) < unit[0]:
                        while not self.qfree[t].done(used[t] + 1):
                            yield False
                        used[t] += 1
                        self.copy(self.q, t, u, self.qfull[t])
            alone = not unit[1]
            pos += unit[0]

    def values(self):
        n = 0
        for u, unit in enumerate(self.units):
            for b in range(unit[0]):
                slot, phase = n % self.slots, n // self.slots
                while not self.vfree[slot].done(phase + 1):
                    yield False
                self.copy(self.v, slot, (u, b), self.vfull[slot])
                n += 1
                yield True

    def look(self):
        n = 0
        for u, unit in enumerate(self.units):
            for b in range(unit[0]):
                slot, phase = n % self.slots, n // self.slots
                while not self.vfull[slot].done(phase):
                    yield False
                assert self.v[slot] == (u, b)
                self.v[slot] = (u, b, "looked at")
                self.fixed[slot].arrive()
                n += 1
                yield True

    def issue(self, t):
        units, slots = self.units, self.slots
        at = dict(u=0, pos=0, b=first(units[0], 0, t), q=0, own=(1 << slots) - 1)  # of the scores, a step ahead
        turns, steps, pos = 1 - t, 0, 0

        def operands():
            while at["u"] < len(units) and at["b"] >= units[at["u"]][0]:
                unit = units[at["u"]]
                if not unit[1] and first(unit, at["pos"], 1 - t) < unit[0]:
                    at["own"] &= 0x5 if t == 0 else 0xa
                at["pos"] += unit[0]
                at["u"] += 1
                if at["u"] < len(units):
                    at["b"] = first(units[at["u"]], at["pos"], t)
            if at["u"] == len(units):
                self.reached[t] = 1 << 32
                return
            unit, pos = units[at["u"]], at["pos"] + at["b"]
            self.reached[t] = pos
            slot = pos % slots
            if not at["own"] >> slot & 1 and pos >= slots:
                while not self.reached[1 - t] > pos - slots:
                    yield False
            at["own"] |= 1 << slot
            if at["b"] < (1 if unit[1] else 2):
                while not self.qfull[t].done(at["q"]):
                    yield False
                at["q"] += 1
            while not self.kfull[slot].done(pos // slots):
                yield False

        def scores():
            u, b, slot = at["u"], at["b"], (at["pos"] + at["b"]) % slots

            def end():
                assert self.k[slot] == (u, b) and self.q[t] == u
                self.s[t] = (u, b)
                self.sfull[t].arrive()
            self.mmas[t].append(end)

        def scores_done():
            unit, slot = units[at["u"]], (at["pos"] + at["b"]) % slots
            self.mmas[t] += [self.kfree[slot].arrive] * (1 if unit[1] else 2)
            at["b"] += 1 if unit[1] else 2
            if at["b"] >= unit[0]:
                self.mmas[t].append(self.qfree[t].arrive)

        def product(u, b, slot):
            def end():
                assert self.v[slot] == (u, b, "looked at") and self.p[t] == (u, b)
                self.o[t] = (u, b)
            self.mmas[t].append(end)

        yield from operands()
        if at["u"] < len(units):
            scores()
            scores_done()
        for u, unit in enumerate(units):
            for b in range(first(unit, pos, t), unit[0], 1 if unit[1] else 2):
                slot, phase = (pos + b) % slots, (pos + b) // slots
                yield from operands()
                while not self.fixed[slot].done(phase):
                    yield False
                while not self.pfull[t].done(steps):
                    yield False
                if unit[1]:
                    while not self.go[t].done(turns):
                        yield False
                    turns += 1
                product(u, b, slot)
                if b + (1 if unit[1] else 2) >= unit[0]:
                    self.mmas[t].append(self.ofull[t].arrive)
                more = at["u"] < len(units)
                if more:
                    scores()
                if unit[1]:
                    self.go[1 - t].arrive()
                self.mmas[t] += [self.vfree[slot].arrive] * (1 if unit[1] else 2)
                if more:
                    scores_done()
                steps += 1
                yield True
            pos += unit[0]

    def softmax(self, t):
        pos = steps = mine_used = other_used = merges = 0
        for u, unit in enumerate(self.units):
            b0, stride = first(unit, pos, t), 1 if unit[1] else 2
            mine, other = b0 < unit[0], first(unit, pos, 1 - t) < unit[0]
            last = [[(u, b) for b in range(first(unit, pos, x), unit[0], stride)][-1:] for x in (0, 1)]
            for b in range(b0, unit[0], stride):
                while not self.sfull[t].done(steps):
                    yield False
                assert self.s[t] == (u, b)
                self.p[t] = (u, b)
                self.pfull[t].arrive()
                steps += 1
                yield True
            merge = not unit[1] and mine and other
            if not unit[1] and b0 != 0:     # the other stream's warps write the rows
                if merge:
                    self.stats = u
                    self.mfull.arrive()
                    while not self.mfree.done(merges):
                        yield False
            else:
                if mine:
                    while not self.ofull[t].done(mine_used):
                        yield False
                    assert [self.o[t]] == last[t]
                if merge:
                    while not self.mfull.done(merges):
                        yield False
                    while not self.ofull[1 - t].done(other_used):
                        yield False
                    assert [self.o[1 - t]] == last[1 - t] and self.stats == u
                    yield True
                    assert [self.o[1 - t]] == last[1 - t]
                    self.mfree.arrive()
            mine_used, other_used, merges, pos = mine_used + mine, other_used + other, merges + merge, pos + unit[0]

    def run(self, r):
        warps = dict(keys=self.keys(), values=self.values(), look=self.look(), issue0=self.issue(0), issue1=self.issue(1),
                     softmax0=self.softmax(0), softmax1=self.softmax(1))
        speed = {w: r.choice([1, 1, 5, 25]) for w in [*warps, "copies", 0, 1]}
        idle = 0
        while warps:
            able = [*warps] + ["copies"] * bool(self.copies) + [t for t in (0, 1) if self.mmas[t]]
            w = r.choices(able, [speed[x] for x in able])[0]
            idle += 1
            if w == "copies":
                self.copies.pop(r.randrange(len(self.copies)))()
                idle = 0
            elif w in (0, 1):
                self.mmas[w].pop(0)()
                idle = 0
            else:
                try:
                    if next(warps[w]):
                        idle = 0
                except StopIteration:
                    del warps[w]
                    idle = 0
            assert idle < 3000, f"{sorted(warps)} wait for ever: {self.units}"


@pytest.mark.parametrize("slots", [2, 4])
def test_any_order_of_units(slots):
    r = random.Random(slots)
    for _ in range(250):
        most = r.choice([2, 3, 6])
        Cta([(r.randint(1, most), r.random() < r.choice([0.2, 0.5, 0.8])) for _ in range(r.randint(1, 14))], slots).run(r)


@pytest.mark.parametrize("slots,units", [(2, [(3, True), (1, False), (2, True)]), (4, [(3, False), (1, True)]),
                                         (2, [(1, False), (2, True), (1, False), (2, False)]), (4, [(1, True), (1, True), (2, False)])])
def test_orders_that_need_care(slots, units):
    """A unit of one tile between units of two; units of one tile first; results joined right behind other units."""
    for seed in range(60):
        Cta(units, slots).run(random.Random(seed))
