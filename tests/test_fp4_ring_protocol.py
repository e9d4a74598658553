"""The ring of the 4-bit products on mma.sync (kernels_fp4.cu), on the CPU.

A stage has a unit's weights, which a bulk copy brings (its warp arrives once and
the bytes are counted), and its tokens, which another warp stores and arrives for
on the same barrier; eight warps multiply (two here) and release the stage.  The roles run as coroutines in random
order, copies land after random times, waits are by parity, and in half of the
runs a random waiter gives up at a random time: from then on nobody waits, and the
warp of the copies lets those under way land before it ends, with arrivals of its
own for units whose tokens will not come.  Checked:
 - a warp multiplies its unit's weights and tokens, landed and not yet replaced;
 - no barrier gets more arrivals than its phase has left (an arrival on a phase
   that only waits for bytes is undefined);
 - no copy is under way when its warp ends.
Whether the warp of the tokens stops where a wait of its own, or another's, has given
up is read from the kernel's source.
"""
import os
import random
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "lossless_bit_weight_w12_gb300", "csrc", "kernels_fp4.cu")


def tokens_stop():
    text = open(SOURCE).read()
    tokens = text[text.index("-- tokens"):text.rindex("-- products")]
    assert "mbar_wait(&empty[s]" in tokens
    stop = re.search(r"bool (\w+) = i >= S && \(!mbar_wait\(&empty\[s\].*\|\| aborted\(&ctl\)\);", tokens)
    return bool(stop) and f"if (__any_sync(0xFFFFFFFFu, {stop.group(1)})) break;" in tokens


class Bar:
    def __init__(self, count):
        self.count = self.pending = count
        self.tx = self.phase = 0

    def settle(self):
        if self.pending == 0 and self.tx == 0:
            self.phase, self.pending = self.phase + 1, self.count

    def arrive(self, tx=0):
        assert self.pending > 0, "an arrival too many"
        self.tx += tx
        self.pending -= 1
        self.settle()

    def landed(self):
        self.tx -= 1
        self.settle()

    def passed(self, phase):
        return (self.phase & 1) != (phase & 1)


class Ring:
    WARPS = 2

    def __init__(self, S, units, stop, seed, abort_at):
        self.S, self.U, self.stop, self.rnd, self.abort_at = S, units, stop, random.Random(seed), abort_at
        self.aborted, self.steps = False, 0
        self.stored = None  # units whose tokens have come, once no more do
        self.full = [Bar(2) for _ in range(S)]
        self.empty = [Bar(self.WARPS) for _ in range(S)]
        self.w, self.x = [None] * S, [None] * S
        self.copies = []  # [steps left, stage, unit]

    def wait(self, bar, phase):
        while not bar.passed(phase):
            if self.aborted:
                return False
            if self.steps > self.abort_at:
                self.aborted = True
                return False
            yield
        return True

    def weights(self):
        issued = 0
        for u in range(self.U):
            s = u % self.S
            if u >= self.S:
                ok = yield from self.wait(self.empty[s], u // self.S - 1)
                if not ok or self.aborted:
                    break
            self.full[s].arrive(tx=1)
            self.w[s] = "on its way"
            self.copies.append([self.rnd.randint(1, 30), s, u])
            issued += 1
            yield
        if self.aborted:
            while self.stored is None:
                yield
            for k in range(max(0, issued - self.S, self.stored), issued):
                self.full[k % self.S].arrive()
            for k in range(max(0, issued - self.S), issued):
                for _ in range(500):  # (bounded)
                    if self.full[k % self.S].passed(k // self.S):
                        break
                    yield
            assert not self.copies, "a copy under way as its warp ends"

    def tokens(self):
        u = 0
        while u < self.U:
            s = u % self.S
            if u >= self.S:
                ok = yield from self.wait(self.empty[s], u // self.S - 1)
                if self.stop and (not ok or self.aborted):
                    break
            self.x[s] = u
            yield
            self.full[s].arrive()
            u += 1
        self.stored = u

    def multiply(self):
        for u in range(self.U):
            s = u % self.S
            yield from self.wait(self.full[s], u // self.S)
            if not self.aborted:
                assert self.w[s] == u and self.x[s] == u
                yield
                assert self.aborted or (self.w[s] == u and self.x[s] == u)
            self.empty[s].arrive()
            for _ in range(self.rnd.randint(0, 5)):
                yield

    def run(self):
        roles = [self.weights(), self.tokens()] + [self.multiply() for _ in range(self.WARPS)]
        pace = [self.rnd.choice([1, 1, 5]) for _ in roles]
        while roles or self.copies:
            self.steps += 1
            assert self.steps < 100000, "stuck"
            for c in self.copies:
                c[0] -= 1
            for c in [c for c in self.copies if c[0] <= 0]:
                self.copies.remove(c)
                self.w[c[1]] = c[2]
                self.full[c[1]].landed()
            if not roles:
                continue
            k = self.rnd.choices(range(len(roles)), weights=pace)[0]
            try:
                next(roles[k])
            except StopIteration:
                del roles[k], pace[k]


@pytest.mark.parametrize("S", [3, 4, 5])
@pytest.mark.parametrize("give_up", [False, True], ids=["", "gives up"])
def test_ring(S, give_up):
    stop = tokens_stop()
    for seed in range(300):
        rnd = random.Random(seed)
        Ring(S, rnd.randint(1, 30), stop, seed, rnd.randint(0, 200) if give_up else 10 ** 9).run()


def test_the_model_sees_an_arrival_too_many():
    with pytest.raises(AssertionError, match="too many"):
        for seed in range(300):
            Ring(4, 30, False, seed, 40).run()
