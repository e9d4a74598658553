"""The waits of the tcgen05 attention kernel with tiles that need a mask, on the
CPU, for both caches.

As in test_attend_pipeline_protocol the kernel's roles and the tensor cores run
as coroutines in random order and waits are by parity.  Here a tile that needs
a mask has its values looked at by all softmax warps of its slot, those without
valid rows among them (they skip the softmax, so they run ahead), and on bf16
the rows past the end are set to zero in the stage the product reads.

Units of 128 rows: the two slots take alternate tiles.  Operand stages: bf16,
head_dim 128: four in turn, keys 0 and 2, values 1 and 3, filled by the copy
engine.  e4m3: one for the keys with a full barrier per slot, one per slot for
the values, filled by converters from an input ring.

Units of 256 rows: both slots use every tile, and their issuing threads take
turns.  Operand stages in turn, four (bf16) or three (e4m3, with an input ring
of three), keys and values alike.

The order that is checked is the kernel's: whether the wait for a tile's scores
comes before the wait for its values is read from its source.
"""
import os
import random
import re

import pytest

from test_attend_pipeline_protocol import Bar, wait

SOURCE = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "lossless_bit_weight_w12_gb300", "csrc",
                      "kernels_attend_tc.cu")


def kernel_waits_for_scores_first():
    text = open(SOURCE).read()
    softmax = text[text.index("-- softmax"):text.index("-- converters")]
    masked = re.search(r"if \(masked\) \{\s*wait_operand\(i, 1\);", softmax)
    scores = softmax.index("att_wait(&s_full[slot]")
    assert masked, "the wait for a masked tile's values"
    return scores < masked.start()


WARPS = 2  # softmax warps of a slot: one with valid rows, one without


class Blocks:
    def __init__(self, segments, masked, e4m3, scores_first, seed):
        self.segments, self.masked, self.e4m3, self.scores_first = segments, masked, e4m3, scores_first
        self.rnd = random.Random(seed)
        self.tiles = sum(segments)
        bars = lambda n, arrivals=1: [Bar(arrivals) for _ in range(n)]  # noqa: E731
        self.stages = 4  # of the input ring (e4m3)
        self.in_full, self.in_empty, self.ring = bars(4), bars(4), [None] * 4
        self.op_full, self.op_empty, self.op = bars(4), bars(4), [None] * 4
        self.s_full, self.o_done = bars(2), bars(2)
        self.p_full, self.q_full = bars(2, WARPS), bars(2, WARPS)
        self.scales_full, self.key_scales, self.value_scales = bars(4), [None] * 4, [None] * 4
        self.scores, self.weights, self.output, self.result = [None] * 2, [None] * 2, [[], []], []
        self.cleared = [[] for _ in range(4)]
        self.copies, self.products = [], []
        self.together = {}

    # operand stage of tile i's keys (0) or values (1), its full barrier, the
    # phase of either barrier that the tile's turn is
    def stage(self, i, kv):
        return (1 + (i & 1) if kv else 0) if self.e4m3 else (2 * i + kv) % 4

    def full(self, i, kv):
        if self.e4m3:
            return self.op_full[1 + (i & 1) if kv else 3 * (i & 1)], i >> 1
        return self.op_full[(2 * i + kv) % 4], (2 * i + kv) // 4

    def turn(self, i, kv):
        return (i >> 1 if kv else i) if self.e4m3 else (2 * i + kv) // 4

    def fill(self, i, kv):
        s = self.stage(i, kv)
        assert self.op[s] == "on its way"
        self.op[s], self.cleared[s] = (i, kv), []
        self.full(i, kv)[0].arrive()

    def copy(self, kv):
        for i in range(self.tiles):
            if self.e4m3:
                h, s = 2 * i + kv, (2 * i + kv) % self.stages
                if h >= self.stages:
                    yield from wait(self.in_empty[s], h // self.stages - 1)
                self.ring[s] = "on its way"
            else:
                s, turn = self.stage(i, kv), self.turn(i, kv)
                if turn:
                    yield from wait(self.op_empty[s], turn - 1)
                self.op[s] = "on its way"
            yield
            self.copies.append((i, kv))

    def copy_engine(self):
        while True:
            if self.copies:
                i, kv = self.copies.pop(self.rnd.randrange(len(self.copies)))
                if self.e4m3:
                    self.ring[(2 * i + kv) % self.stages] = (i, kv)
                    self.in_full[(2 * i + kv) % self.stages].arrive()
                else:
                    self.fill(i, kv)
            yield

    def convert(self, kv):
        if not self.e4m3:
            return
        for i in range(self.tiles):
            h, s = 2 * i + kv, (2 * i + kv) % self.stages
            yield from wait(self.in_full[s], h // self.stages)
            assert self.ring[s] == (i, kv)
            if kv:
                self.value_scales[i % 4] = i
                self.scales_full[i % 4].arrive()
            to, turn = self.stage(i, kv), self.turn(i, kv)
            if turn:
                yield from wait(self.op_empty[to], turn - 1)
            if not kv:
                self.key_scales[i % 4] = i
            self.op[to] = "on its way"
            yield
            self.fill(i, kv)
            self.ring[s] = None
            self.in_empty[s].arrive()
            yield

    def parts(self, slot):
        """(first tile of the slot, end) of each segment; None: no tile."""
        t = 0
        for n in self.segments:
            first = t + (1 if (t & 1) != slot else 0)
            yield (first, t + n) if first < t + n else None
            t += n

    def meet(self, key, n):
        """A barrier of n coroutines, named by what they meet for."""
        self.together[key] = self.together.get(key, 0) + 1
        while self.together[key] < n:
            yield

    def softmax(self, slot, valid):
        tiles = segs = 0
        for g, part in enumerate(self.parts(slot)):
            for k in range(2):  # both slots copy the queries
                yield from self.meet(("queries", g, k), 2 * WARPS)
            if not part:
                continue
            if valid:
                self.output[slot] = []
            self.q_full[slot].arrive()
            for i in range(part[0], part[1], 2):
                if self.scores_first:
                    yield from wait(self.s_full[slot], tiles)
                if i in self.masked:
                    bar, phase = self.full(i, 1)
                    yield from wait(bar, phase)
                    s = self.stage(i, 1)
                    assert self.op[s] == (i, 1)
                    yield
                    assert self.op[s] == (i, 1)
                    if self.e4m3:
                        assert self.value_scales[i % 4] == i
                    else:
                        self.cleared[s].append(i)
                    yield from self.meet(("masked", i), WARPS)
                if not self.scores_first:
                    yield from wait(self.s_full[slot], tiles)
                tiles += 1
                if valid:
                    assert self.scores[slot] == i
                    yield
                    if self.e4m3:
                        assert self.key_scales[i % 4] == i
                        yield from wait(self.scales_full[i % 4], i // 4)
                        assert self.value_scales[i % 4] == i
                        yield
                        assert self.value_scales[i % 4] == i and self.key_scales[i % 4] == i
                    assert self.scores[slot] == i
                    self.weights[slot] = i
                self.p_full[slot].arrive()
                yield
            yield from wait(self.o_done[slot], segs)
            segs += 1
            if valid:
                self.result.extend(self.output[slot])
            yield

    def issue(self, slot):
        def scores(i):
            def run():
                assert self.op[self.stage(i, 0)] == (i, 0)
                self.scores[slot] = i
                self.s_full[slot].arrive()
                self.op_empty[self.stage(i, 0)].arrive()
            self.products.append(run)

        def outputs(i):
            def run():
                s = self.stage(i, 1)
                assert self.op[s] == (i, 1) and self.weights[slot] == i
                if not self.e4m3:
                    assert self.cleared[s] == ([i] * WARPS if i in self.masked else [])
                self.output[slot].append(i)
                self.op_empty[s].arrive()
            self.products.append(run)

        tiles = segs = 0
        for part in self.parts(slot):
            if not part:
                continue
            yield from wait(self.q_full[slot], segs)
            segs += 1
            yield from wait(*self.full(part[0], 0))
            scores(part[0])
            yield
            for i in range(part[0], part[1], 2):
                more = i + 2 < part[1]
                yield from wait(*self.full(i, 1))
                if more and not self.e4m3:
                    yield from wait(*self.full(i + 2, 0))
                yield from wait(self.p_full[slot], tiles)
                tiles += 1
                outputs(i)
                yield
                if more:
                    if self.e4m3:
                        yield from wait(*self.full(i + 2, 0))
                    scores(i + 2)
                else:
                    self.products.append(self.o_done[slot].arrive)
                yield

    def tensor_cores(self):
        while True:
            if self.products:
                self.products.pop(0)()
            yield

    def run(self):
        roles = [f(x) for f in (self.copy, self.convert, self.issue) for x in (0, 1)]
        roles += [self.softmax(slot, valid) for slot in (0, 1) for valid in (True, False)]
        engines = [self.tensor_cores(), self.copy_engine()]
        speed = {r: self.rnd.choice([1, 1, 3, 10]) for r in roles}
        lag = self.rnd.choice([0.1, 0.3, 0.5])  # how often the engines get on
        for _ in range(self.tiles * 8000 + 40000):
            if not roles:
                break
            if self.rnd.random() < lag:
                next(self.rnd.choice(engines))
                continue
            r = self.rnd.choices(roles, [speed[x] for x in roles])[0]
            if next(r, self) is self:
                roles.remove(r)
        assert not roles, "no progress"
        assert sorted(self.result) == self.results()

    def results(self):
        return list(range(self.tiles))


class Wide(Blocks):
    """Units of 256 rows."""

    def __init__(self, segments, masked, e4m3, scores_first, seed):
        super().__init__(segments, masked, e4m3, scores_first, seed)
        bars = lambda n, arrivals=1: [Bar(arrivals) for _ in range(n)]  # noqa: E731
        self.operands, self.stages = (3 if e4m3 else 4), 3
        writers = 2 if e4m3 else 1  # converter warps, each in the order of the tiles
        self.op_full, self.op_empty = bars(self.operands, writers), bars(self.operands, 2)
        self.in_empty = bars(self.stages, writers)
        self.scales_full, self.token = bars(4, writers), bars(2)
        self.half = [[] for _ in range(self.operands)]

    def stage(self, i, kv):
        return (2 * i + kv) % self.operands

    def full(self, i, kv):
        return self.op_full[self.stage(i, kv)], (2 * i + kv) // self.operands

    def turn(self, i, kv):
        return (2 * i + kv) // self.operands

    def convert(self, warp):
        if not self.e4m3:
            return
        for h in range(2 * self.tiles):
            i, kv, s = h // 2, h % 2, h % self.stages
            yield from wait(self.in_full[s], h // self.stages)
            assert self.ring[s] == (i, kv)
            if kv:
                self.value_scales[i % 4] = i
                self.scales_full[i % 4].arrive()
            to, turn = self.stage(i, kv), self.turn(i, kv)
            if turn:
                yield from wait(self.op_empty[to], turn - 1)
            if not kv:
                self.key_scales[i % 4] = i
            if self.op[to] != ("half", i, kv):
                self.op[to], self.half[to], self.cleared[to] = ("half", i, kv), [], []
            yield
            assert self.ring[s] == (i, kv) and self.op[to] == ("half", i, kv)
            self.half[to].append(warp)
            if len(self.half[to]) == 2:
                self.op[to] = (i, kv)
            self.op_full[to].arrive()
            self.in_empty[s].arrive()
            yield

    def parts(self, slot):
        t = 0
        for n in self.segments:
            yield (t, t + n)
            t += n

    def softmax(self, slot, valid):
        tiles = 0
        for segs, part in enumerate(self.parts(slot)):
            yield from self.meet(("queries", segs, slot), WARPS)
            if valid:
                self.output[slot] = []
            self.q_full[slot].arrive()
            for i in range(*part):
                if self.scores_first:
                    yield from wait(self.s_full[slot], tiles)
                if i in self.masked:
                    bar, phase = self.full(i, 1)
                    yield from wait(bar, phase)
                    s = self.stage(i, 1)
                    assert self.op[s] == (i, 1)
                    yield
                    assert self.op[s] == (i, 1)
                    if self.e4m3:
                        assert self.value_scales[i % 4] == i
                    else:
                        self.cleared[s].append(i)
                    yield from self.meet(("masked", i), 2 * WARPS)
                if not self.scores_first:
                    yield from wait(self.s_full[slot], tiles)
                tiles += 1
                if valid:
                    assert self.scores[slot] == i
                    yield
                    if self.e4m3:
                        assert self.key_scales[i % 4] == i
                        yield from wait(self.scales_full[i % 4], i // 4)
                        assert self.value_scales[i % 4] == i
                        yield
                        assert self.value_scales[i % 4] == i and self.key_scales[i % 4] == i
                    self.weights[slot] = i
                self.p_full[slot].arrive()
                yield
            yield from wait(self.o_done[slot], segs)
            if valid:
                self.result.extend(self.output[slot])
            yield

    def issue(self, slot):
        def scores(i, hand_on):
            def run():
                assert self.op[self.stage(i, 0)] == (i, 0)
                self.scores[slot] = i
                self.s_full[slot].arrive()
                self.op_empty[self.stage(i, 0)].arrive()
            self.products.append(run)
            if hand_on:
                self.token[slot ^ 1].arrive()

        def outputs(i):
            def run():
                s = self.stage(i, 1)
                assert self.op[s] == (i, 1) and self.weights[slot] == i
                if not self.e4m3:
                    assert self.cleared[s] == ([i] * 2 * WARPS if i in self.masked else [])
                self.output[slot].append(i)
                self.op_empty[s].arrive()
            self.products.append(run)

        tiles = 0
        for segs, part in enumerate(self.parts(slot)):
            yield from wait(self.q_full[slot], segs)
            yield from wait(*self.full(part[0], 0))
            scores(part[0], False)
            yield
            for i in range(*part):
                more = i + 1 < part[1]
                yield from wait(*self.full(i, 1))
                if more and not self.e4m3:
                    yield from wait(*self.full(i + 1, 0))
                yield from wait(self.p_full[slot], tiles)
                tiles += 1
                if i or slot:
                    yield from wait(self.token[slot], (2 * i + slot - 1) // 2)
                outputs(i)
                if not more:
                    self.token[slot ^ 1].arrive()
                yield
                if more:
                    if self.e4m3:
                        yield from wait(*self.full(i + 1, 0))
                    scores(i + 1, True)
                else:
                    self.products.append(self.o_done[slot].arrive)
                yield

    def results(self):
        return sorted(list(range(self.tiles)) * 2)


def problem(kind, seed, e4m3, scores_first):
    """Segments of a CTA; the last tiles of some of them (a request's newest keys) are masked."""
    r = random.Random(seed)
    segments = [r.choice([1, 1, 2, 3, 4, 5, 9, 16]) for _ in range(r.randrange(1, 6))]
    masked, t = set(), 0
    for n in segments:
        t += n
        masked |= set(range(t - min(n, r.choice([0, 1, 1, 2])), t))
    return kind(segments, masked, e4m3, scores_first, seed)


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("kind", [Blocks, Wide], ids=["128", "256"])
def test_masked_tiles_in_the_kernels_order(kind, e4m3):
    for seed in range(300):
        problem(kind, seed, e4m3, kernel_waits_for_scores_first()).run()


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_waiting_for_the_values_first_is_not_safe(e4m3):
    """A warp without valid rows never waited for the stage's values before, and
    takes the phase before for this one."""
    wrong = 0
    for seed in range(300):
        try:
            problem(Blocks, seed, e4m3, False).run()
        except AssertionError:
            wrong += 1
    assert wrong > 10
