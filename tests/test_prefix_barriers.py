"""A model of the barriers of the shared-prefix attention kernel: its roles step in random order, copies land in random
order, matrix products of different shapes complete in random order, and every read is checked to find what it is meant
to find.  The order in which the copying warps take their steps, and whether scores wait for the weights in their place
to be done with, is read from the kernel's source."""

import os
import random
import re

import pytest

from linear_attention_decode_02_gb300 import build

SOURCE = open(os.path.join(build.CSRC, "kda_prefix.cu")).read()
WARPS = 2  # that copy; the kernel has four


def section(start, end):
    return SOURCE[SOURCE.index(start):SOURCE.index(end)]


def copy_steps():
    """What a copying warp does for a tile: 'room' (waits for the next half's slot), 'mask', 'keys', 'values'."""
    names = {"wait_or_abort(&empty": "room", "mbar_arrive(&live_full": "mask", "copy_half(a.kp": "keys",
             "copy_half(a.vp": "values"}
    found = re.findall("|".join(re.escape(n) for n in names), section("// ---------------- copies", "// ---------------- queries"))
    return [names[n] for n in found]


def scores_wait():
    return "wait_or_abort(&o_done" in section("const auto scores", "const auto output")


class Barrier:
    """As an mbarrier: `count` arrivals end a phase; a wait for a parity passes when the current phase has the other one."""

    def __init__(self, count):
        self.count = self.left = count
        self.phase = 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left = self.count
            self.phase += 1

    def over(self, parity):
        return self.phase & 1 != parity & 1


class Pipe:
    """A lane's tensor operations: those of one kind complete in order; a commit's arrival follows all before it."""

    def __init__(self):
        self.queue = []

    def step(self, rng):
        kinds = [kind for kind, _ in self.queue]
        first = {kind: kinds.index(kind) for kind in kinds}
        if first.get("commit") != 0:
            first.pop("commit", None)
        if first:
            self.queue.pop(rng.choice(list(first.values())))[1]()


class Model:
    def __init__(self, counts, seed, RT, LANES, STEPS, SLOTS, QSLOTS, steps, wait):
        self.scores_wait = wait
        self.rng, self.counts, self.shape, self.loader_steps = random.Random(seed), counts, (RT, LANES, STEPS, SLOTS, QSLOTS), steps
        self.split = RT < LANES
        bars = lambda n, count: [Barrier(count) for _ in range(n)]  # noqa: E731
        self.full, self.empty = bars(SLOTS, WARPS), bars(SLOTS, RT)
        self.s_full, self.p_full, self.o_done = bars(2 * LANES, 1), bars(2 * LANES, 1), bars(2 * LANES, 1)
        self.q_full, self.q_empty = bars(QSLOTS, 1), bars(QSLOTS, LANES)
        self.live, self.x_full, self.x_empty = bars(16, WARPS), Barrier(1), Barrier(1)
        self.ring = [[None] * SLOTS for _ in range(WARPS)]
        self.mask, self.S, self.O, self.Q = [None] * 16, [None] * (2 * LANES), [None] * LANES, [None] * QSLOTS
        self.exchange, self.flight, self.wrong = None, [], []
        self.pipes = [Pipe() for _ in range(LANES)]

    def need(self, found, wanted, what):
        if found != wanted:
            self.wrong.append(f"{what}: {found} in the place of {wanted}")

    def wait(self, bar, parity):
        while not bar.over(parity):
            yield

    def copies(self, w):
        SLOTS, half, tile = self.shape[3], 0, 0
        for count in self.counts:
            for _ in range(count):
                for step in self.loader_steps:
                    if step == "room":
                        if half >= SLOTS:
                            yield from self.wait(self.empty[half % SLOTS], half // SLOTS - 1)
                    elif step == "mask":
                        self.mask[tile % 16] = tile
                        self.live[tile % 16].arrive()
                    else:
                        self.ring[w][half % SLOTS] = ("under way", half)
                        self.flight.append((w, half))
                        half += 1
                    yield
                tile += 1

    def land(self):
        w, half = self.flight.pop(self.rng.randrange(len(self.flight)))
        self.ring[w][half % self.shape[3]] = half
        self.full[half % self.shape[3]].arrive()

    def queries(self):
        QSLOTS = self.shape[4]
        for unit in range(len(self.counts)):
            q = unit % QSLOTS
            if unit >= QSLOTS:
                yield from self.wait(self.q_empty[q], unit // QSLOTS - 1)
            self.Q[q] = unit
            yield
            self.q_full[q].arrive()
            yield

    def steps_of(self, count, me):
        return ((count + 1 - me) // 2 if self.split else count) * self.shape[2]

    def tile_of(self, i, me):
        return i // self.shape[2] * (2 if self.split else 1) + (me if self.split else 0)

    def products(self, me):
        _, _, STEPS, SLOTS, QSLOTS = self.shape
        half = tile = job = 0
        issue = self.pipes[me].queue.append

        def used(h):
            issue(("commit", self.empty[h % SLOTS].arrive))

        def scores(unit, i):
            q, j, b, sub = unit % QSLOTS, self.tile_of(i, me), 2 * me + (job + i) % 2, i % STEPS
            h = half + 2 * j
            if i == 0:
                yield from self.wait(self.q_full[q], unit // QSLOTS)
            if sub == 0:
                yield from self.wait(self.live[(tile + j) % 16], (tile + j) // 16)
                self.need(self.mask[(tile + j) % 16], tile + j, "mask")
                yield from self.wait(self.full[h % SLOTS], h // SLOTS)
            if self.scores_wait and job + i >= 2:
                yield from self.wait(self.o_done[b], (job + i) // 2 - 1)

            def run():
                self.need(self.Q[q], unit, "queries")
                self.need([r[h % SLOTS] for r in self.ring], [h] * WARPS, "keys")
                self.S[b] = ("scores", unit, i)

            issue(("scores", run))
            issue(("commit", self.s_full[b].arrive))
            if sub == STEPS - 1:
                used(h)

        def output(unit, i):
            b, sub, h = 2 * me + (job + i) % 2, i % STEPS, half + 2 * self.tile_of(i, me) + 1
            if sub == 0:
                yield from self.wait(self.full[h % SLOTS], h // SLOTS)
            yield from self.wait(self.p_full[b], (job + i) // 2)

            def run():
                self.need([r[h % SLOTS] for r in self.ring], [h] * WARPS, "values")
                self.need(self.S[b], ("weights", unit, i), "weights")
                if i > 0:
                    self.need(self.O[me], ("output", unit, i - 1), "output so far")
                self.O[me] = ("output", unit, i)

            issue(("output", run))
            issue(("commit", self.o_done[b].arrive))
            if sub == STEPS - 1:
                used(h)

        for unit, count in enumerate(self.counts):
            steps = self.steps_of(count, me)
            for i in range(steps + 1):
                first = self.split and i % STEPS == 0
                if first and i > 0:
                    yield from output(unit, i - 1)
                yield
                if i < steps:
                    yield from scores(unit, i)
                yield
                if not first and i > 0:
                    yield from output(unit, i - 1)
                yield
            if steps == 0:
                yield from self.wait(self.q_full[unit % QSLOTS], unit // QSLOTS)
            issue(("commit", self.q_empty[unit % QSLOTS].arrive))
            half, tile, job = half + 2 * count, tile + count, job + steps
            yield

    def softmax(self, me):
        tile = job = 0
        for unit, count in enumerate(self.counts):
            steps = self.steps_of(count, me)
            for i in range(steps):
                b, j = 2 * me + job % 2, tile + self.tile_of(i, me)
                yield from self.wait(self.s_full[b], job // 2)
                if i % self.shape[2] == 0:
                    yield from self.wait(self.live[j % 16], j // 16)
                self.need(self.S[b], ("scores", unit, i), "scores")
                self.need(self.mask[j % 16], j, "mask of the softmax")
                if i > 0 and self.rng.random() < .5:  # rescales
                    yield from self.wait(self.o_done[2 * me + (job - 1) % 2], (job - 1) // 2)
                    self.need(self.O[me], ("output", unit, i - 1), "output to be rescaled")
                yield
                self.S[b] = ("weights", unit, i)
                if self.split and me == 1 and i == 0 and unit > 0:
                    yield from self.wait(self.x_empty, unit - 1)
                self.p_full[b].arrive()
                job += 1
                yield
            if steps > 0:
                yield from self.wait(self.o_done[2 * me + (job - 1) % 2], (job - 1) // 2)
                self.need(self.O[me], ("output", unit, steps - 1), "output at the unit's end")
            if self.split and me == 1:
                if steps == 0 and unit > 0:
                    yield from self.wait(self.x_empty, unit - 1)
                self.exchange = unit
                self.x_full.arrive()
            elif self.split:
                yield from self.wait(self.x_full, unit)
                self.need(self.exchange, unit, "the other lane's statistics")
                if count > 1:
                    self.need(self.O[1], ("output", unit, self.steps_of(count, 1) - 1), "the other lane's output")
                yield
                self.x_empty.arrive()
            tile += count
            yield

    def run(self, most=400000):
        """What was found wrong, nothing where all is well."""
        rng, LANES = self.rng, self.shape[1]
        roles = [self.queries(), *(self.copies(w) for w in range(WARPS)), *(self.products(m) for m in range(LANES)),
                 *(self.softmax(m) for m in range(LANES))]
        weight = {id(r): rng.choice([1, 1, 3, 10]) for r in roles}
        lands, tensor = rng.choice([.02, .2, .5]), rng.choice([.1, .3, .6])
        for _ in range(most):
            if self.wrong:
                return self.wrong
            if not roles and not self.flight and not any(p.queue for p in self.pipes):
                return []
            if self.flight and (rng.random() < lands or not roles):
                self.land()
            elif rng.random() < tensor or not roles:
                rng.choice(self.pipes).step(rng)
            else:
                role = rng.choices(roles, [weight[id(r)] for r in roles])[0]
                if next(role, roles) is roles:
                    roles.remove(role)
        return ["a role waits for ever"]


SHAPES = {"one row tile": (1, 2, 2, 5, 2), "one row tile, 64 channels": (1, 2, 2, 12, 2), "two row tiles": (2, 2, 2, 5, 1),
          "two row tiles, 64 channels": (2, 2, 2, 12, 1), "256 channels": (1, 1, 1, 5, 1)}


def sweep(name, steps, wait, runs=150):
    found = []
    for seed in range(runs):
        rng = random.Random(seed * 7 + 1)
        counts = [rng.choice([1, 1, 2, 3, 3, 5, rng.randint(1, 9)]) for _ in range(rng.randint(1, 9))]
        if seed % 5 == 0:
            counts = [1] * rng.randint(1, 9)
        found += [(counts, w) for w in Model(counts, seed, *SHAPES[name], steps, wait).run()[:1]]
    return found


def test_the_source_has_the_steps_of_the_model():
    assert sorted(copy_steps()) == ["keys", "mask", "room", "room", "values"]


@pytest.mark.parametrize("name", SHAPES)
def test_every_read_finds_what_it_waits_for(name):
    assert sweep(name, copy_steps(), scores_wait()) == []


def test_a_mask_given_before_the_values_have_room_is_noticed():
    found = sweep("one row tile", ["room", "mask", "keys", "room", "values"], True, 400)
    assert any("values" in w for _, w in found)


@pytest.mark.parametrize("name", SHAPES)
def test_scores_that_go_where_weights_are_still_read_are_noticed(name):
    found = sweep(name, copy_steps(), False)
    assert any("weights" in w for _, w in found)
