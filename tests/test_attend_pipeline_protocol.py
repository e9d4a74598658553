"""The waits of the tcgen05 attention kernel's e4m3 pipeline, on the CPU.

The kernel's roles (copies of keys and of values, their converters, two
softmax groups, two issuing threads) and the tensor cores run as coroutines in
random order; waits are by parity, as an mbarrier's.  Checked: every stage and
scale table holds what its reader expects, and every schedule ends.  Stages as
in the kernel: an input ring of an even number of stages (each the keys' or the
values'), one operand stage for the keys with a full barrier per slot, one per
slot for the values, scale tables of four tiles.
"""
import random

import pytest


class Bar:
    """An mbarrier; done(parity) is what a wait on that parity sees."""

    def __init__(self, n=1):
        self.n, self.pending, self.phase = n, n, 0

    def arrive(self):
        assert self.pending > 0
        self.pending -= 1
        if self.pending == 0:
            self.phase, self.pending = self.phase + 1, self.n

    def done(self, parity):
        return (self.phase & 1) != (parity & 1)


def wait(bar, count):
    """Until the barrier's phase `count` has completed, as far as its parity tells."""
    while not bar.done(count):
        yield


class Pipeline:
    def __init__(self, segments, stages, seed):
        self.segments, self.stages, self.rnd = segments, stages, random.Random(seed)
        self.tiles = sum(segments)
        bars = lambda n: [Bar() for _ in range(n)]  # noqa: E731
        self.in_full, self.in_empty = bars(stages), bars(stages)
        self.key_full, self.value_full, self.key_empty, self.value_empty = bars(2), bars(2), Bar(), bars(2)
        self.s_full, self.p_full, self.q_full, self.o_done, self.scales_full = bars(2), bars(2), bars(2), bars(2), bars(4)
        self.ring, self.keys, self.values = [None] * stages, None, [None, None]
        self.key_scales, self.value_scales = [None] * 4, [None] * 4
        self.scores, self.weights, self.output, self.result = [None] * 2, [None] * 2, [[], []], []
        self.named, self.copies, self.products = [0, 0], [], []

    def copy(self, kv):
        for i in range(self.tiles):
            h, s = 2 * i + kv, (2 * i + kv) % self.stages
            if h >= self.stages:
                yield from wait(self.in_empty[s], h // self.stages - 1)
            self.ring[s] = "on its way"
            yield
            self.copies.append((s, (i, kv)))

    def copy_engine(self):
        while True:
            if self.copies:
                s, what = self.copies.pop(self.rnd.randrange(len(self.copies)))
                assert self.ring[s] == "on its way"
                self.ring[s] = what
                self.in_full[s].arrive()
            yield

    def convert(self, kv):
        for i in range(self.tiles):
            h, s = 2 * i + kv, (2 * i + kv) % self.stages
            yield from wait(self.in_full[s], h // self.stages)
            assert self.ring[s] == (i, kv)
            if kv:
                self.value_scales[i % 4] = i
                self.scales_full[i % 4].arrive()
                if i >= 2:
                    yield from wait(self.value_empty[i & 1], i // 2 - 1)
                self.values[i & 1] = "half written"
                yield
                self.values[i & 1] = i
                self.value_full[i & 1].arrive()
            else:
                if i:
                    yield from wait(self.key_empty, i - 1)
                self.key_scales[i % 4] = i
                self.keys = "half written"
                yield
                self.keys = i
                self.key_full[i & 1].arrive()
            assert self.ring[s] == (i, kv)
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

    def softmax(self, slot):
        tiles = segs = syncs = 0
        for part in self.parts(slot):
            for _ in range(2):  # both slots copy the queries
                syncs += 1
                self.named[slot] += 1
                while self.named[slot ^ 1] < syncs:
                    yield
            if not part:
                continue
            self.output[slot] = []
            self.q_full[slot].arrive()
            for i in range(part[0], part[1], 2):
                yield from wait(self.s_full[slot], tiles)
                tiles += 1
                assert self.scores[slot] == i and self.key_scales[i % 4] == i
                yield
                assert self.key_scales[i % 4] == i
                yield from wait(self.scales_full[i % 4], i // 4)
                assert self.value_scales[i % 4] == i
                if self.rnd.random() < 0.2:  # a masked tile: the values are looked at
                    yield from wait(self.value_full[i & 1], i // 2)
                    assert self.values[i & 1] == i
                yield
                assert self.value_scales[i % 4] == i and self.scores[slot] == i
                self.weights[slot] = i
                self.p_full[slot].arrive()
                yield
            yield from wait(self.o_done[slot], segs)
            segs += 1
            self.result.extend(self.output[slot])
            yield

    def issue(self, slot):
        def scores(i):
            def run():
                assert self.keys == i
                self.scores[slot] = i
                self.s_full[slot].arrive()
                self.key_empty.arrive()
            self.products.append(run)

        def outputs(i):
            def run():
                assert self.values[i & 1] == i and self.weights[slot] == i
                self.output[slot].append(i)
                self.value_empty[i & 1].arrive()
            self.products.append(run)

        tiles = segs = 0
        for part in self.parts(slot):
            if not part:
                continue
            yield from wait(self.q_full[slot], segs)
            segs += 1
            yield from wait(self.key_full[part[0] & 1], part[0] // 2)
            scores(part[0])
            yield
            for i in range(part[0], part[1], 2):
                yield from wait(self.value_full[i & 1], i // 2)
                yield from wait(self.p_full[slot], tiles)
                tiles += 1
                outputs(i)
                yield
                if i + 2 < part[1]:
                    yield from wait(self.key_full[i & 1], i // 2 + 1)
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
        roles = [f(x) for f in (self.copy, self.convert, self.softmax, self.issue) for x in (0, 1)]
        engines = [self.tensor_cores(), self.copy_engine()]
        speed = {r: self.rnd.choice([1, 1, 3, 10]) for r in roles}
        for _ in range(self.tiles * 4000 + 20000):
            if not roles:
                break
            if self.rnd.random() < 0.3:
                next(self.rnd.choice(engines))
                continue
            r = self.rnd.choices(roles, [speed[x] for x in roles])[0]
            if next(r, self) is self:
                roles.remove(r)
        assert not roles, "no progress"
        assert sorted(self.result) == list(range(self.tiles))


@pytest.mark.parametrize("stages", [4, 8])
def test_every_schedule_ends_with_the_right_contents(stages):
    for seed in range(300):
        r = random.Random(seed)
        Pipeline([r.choice([1, 1, 2, 3, 4, 5, 9]) for _ in range(r.randrange(1, 6))], stages, seed).run()


def test_an_odd_number_of_stages_is_not_safe():
    """Keys and values would take turns in a stage, and a parity wait can pass a phase early."""
    with pytest.raises(AssertionError):
        for seed in range(300):
            r = random.Random(seed)
            Pipeline([r.choice([4, 5, 9]) for _ in range(3)], 3, seed).run()
