"""When the tcgen05 product kernels (kernels_tc.cu, kernels_fp4_tc.cu) give their
tensor memory back, on the CPU.

After a wait that gave up every role runs to its end without waiting, so no wait
that the abort flag cuts short can tell an issuer that the other warps are done:
a store to tensor memory that has been freed is an error of the whole context.
The roles run as coroutines in random order -- producers reduced to their pace,
warps that expand weights (they store A buffers and read sums), issuers -- and a
random waiter gives up at a random time.  What an issuer waits for before it
frees is read from the kernels' source.
"""
import os
import random
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "lossless_bit_weight_w12_gb300", "csrc")


class Bar:
    def __init__(self, count):
        self.count = self.pending = count
        self.phase = 0

    def arrive(self):
        self.pending -= 1
        assert self.pending >= 0
        if self.pending == 0:
            self.phase, self.pending = self.phase + 1, self.count

    def passed(self, parity):
        return (self.phase & 1) != parity


def last_wait(name, barriers):
    """(the call, the barrier) of an issuer's last wait before it frees."""
    text = open(os.path.join(CSRC, name)).read()
    before = text[:text.index("tcgen05.dealloc")]
    calls = re.findall(r"(mbar_wait|mbar_drain)\(&(?:bar\.)?(\w+)", before)
    call, bar = calls[-1]
    assert bar in barriers, bar
    return call, bar


class Cta:
    """pieces: units per piece.  The two issuers' UMMAs of a unit need both
    groups' A buffers (two per tile, units in turn)."""

    def __init__(self, pieces, wait, seed, abort):
        self.pieces, self.wait_kind, self.rnd = pieces, wait, random.Random(seed)
        self.aborted, self.abort_at = False, abort
        self.steps, self.freed, self.freed_by = 0, False, 0
        self.warps = 4  # that expand: two groups of two
        self.a_full = [Bar(2) for _ in range(2)]
        self.a_empty = [Bar(2) for _ in range(2)]
        self.sum_full, self.sum_empty = Bar(2), Bar(4)
        self.out = Bar(4)
        self.umma = 0  # products under way

    def wait(self, bar, phase):  # bounded: cut short by the abort
        while not bar.passed(phase & 1):
            if self.aborted:
                return
            if self.steps > self.abort_at:
                self.aborted = True  # this waiter gave up
                return
            yield

    def drain(self, bar, phase):
        while not bar.passed(phase & 1):
            yield

    def touch(self):
        assert not self.freed, "tensor memory is used after it was freed"

    def warp(self, grp):
        i, last = 0, len(self.pieces) - 1
        for piece, n in enumerate(self.pieces):
            for unit in range(i, i + n):
                if unit % 2 != grp:
                    continue
                for _ in range(self.rnd.randint(0, 12)):
                    yield
                if unit >= 2:
                    yield from self.wait(self.a_empty[grp], unit // 2 - 1)
                self.touch()
                self.a_full[grp].arrive()
            i += n
            yield from self.wait(self.sum_full, piece)
            self.touch()
            yield
            self.touch()
            self.sum_empty.arrive()
            if piece == last:
                self.out.arrive()

    def issuer(self):
        i = 0
        for piece, n in enumerate(self.pieces):
            if piece:
                yield from self.wait(self.sum_empty, piece - 1)
            for unit in range(i, i + n):
                yield from self.wait(self.a_full[unit % 2], unit // 2)
                yield
                self.touch()
                self.a_empty[unit % 2].arrive()
            i += n
            self.sum_full.arrive()
        call, bar = self.wait_kind
        if bar == "out":
            assert call == "mbar_drain"
            yield from self.drain(self.out, 0)
        else:
            yield from (self.wait if call == "mbar_wait" else self.drain)(self.sum_empty, len(self.pieces) - 1)
        self.freed_by += 1
        if self.freed_by == 2:
            self.freed = True

    def run(self):
        roles = [self.warp(g) for g in (0, 0, 1, 1)] + [self.issuer(), self.issuer()]
        pace = [self.rnd.choice([1, 1, 4]) for _ in roles]
        while roles:
            self.steps += 1
            assert self.steps < 200000, "stuck"
            k = self.rnd.choices(range(len(roles)), weights=pace)[0]
            try:
                next(roles[k])
            except StopIteration:
                del roles[k], pace[k]
        assert self.freed


@pytest.mark.parametrize("name", ["kernels_fp4_tc.cu", "kernels_tc.cu"])
@pytest.mark.parametrize("give_up", [False, True], ids=["", "gives up"])
def test_freed_after_the_last_use(name, give_up):
    wait = last_wait(name, {"out", "sum_empty", "acc_empty"})
    for seed in range(300):
        rnd = random.Random(seed)
        pieces = [rnd.choice([1, 2, 3, 8]) for _ in range(rnd.randint(1, 4))]
        Cta(pieces, wait, seed, rnd.randint(0, 120) if give_up else 10 ** 9).run()


def test_the_model_sees_a_wait_that_the_abort_cuts_short():
    with pytest.raises(AssertionError, match="after it was freed"):
        for seed in range(300):
            Cta([3, 8], ("mbar_wait", "sum_empty"), seed, 20).run()
