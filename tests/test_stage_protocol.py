"""The barriers between the warps of the grouped products (csrc/grouped_gemm.cu), on the
CPU: a model of each role's waits, arrivals and copies, run with every role as the slowest
in turn and in random orders.

A parity wait passes while the barrier's last completed phase has that parity, so a role
may wait only on a barrier that cannot complete two phases without it.  The model has the
kernel's rules; `late_follower` is a rule that breaks this (a warp that follows `empty`
although only some steps need it), which the model must find.
"""
import os
import random
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "moe_finalize_rmsnorm_gb300", "csrc", "grouped_gemm.cu")
STEP = 64


class Barrier:
    def __init__(self, count):
        self.count, self.pending, self.bytes, self.phases = count, count, 0, 0

    def passes(self, parity):
        return self.phases % 2 != parity

    def arrive(self, expect=0):
        self.bytes += expect
        self.pending -= 1
        self._complete()

    def landed(self, bytes_):
        self.bytes -= bytes_
        self._complete()

    def _complete(self):
        if self.pending == 0 and self.bytes == 0:
            self.phases += 1
            self.pending = self.count


class Model:
    """One CTA of the weights' gradient.  `sums` are its tiles' summed values; the bytes of
    a whole step and of a last one are units: one per copying warp."""

    def __init__(self, sums, stages, gather=0, segment=None, late_follower=False):
        self.sums, self.stages, self.gather = sums, stages, gather
        self.segment = segment
        self.late_follower = late_follower
        self.full = [Barrier(1) for _ in range(stages)]
        self.empty = [Barrier(1) for _ in range(stages)]
        self.tail = [Barrier(1) for _ in range(stages)]
        self.acc_full = [Barrier(1) for _ in range(2)]
        self.acc_empty = [Barrier(1) for _ in range(2)]
        self.flights = []          # copies under way
        self.stage_step = [None] * stages   # the step whose copies a stage takes
        self.used = []
        self.roles = {"blocks": self.blocks(), "products": self.products(),
                      "results": self.results()}
        if gather:
            for sub in range(gather):
                for stage in range(stages):
                    self.roles[f"gather{stage}.{sub}"] = self.rows(stage)
        else:
            self.roles["last rows"] = (self.follow_empty() if late_follower
                                       else self.last_rows())

    def steps(self, summed):
        return (summed + STEP - 1) // STEP

    def copy(self, stage, step):
        assert self.stage_step[stage] in (None, step), "a stage is filled by two steps"
        self.flights.append((stage, step))

    def land(self, i):
        stage, step = self.flights.pop(i)
        self.full[stage].landed(1)

    def blocks(self):
        it = 0
        for summed in self.sums:
            for s in range(self.steps(summed)):
                stage, parity = it % self.stages, it // self.stages % 2
                yield self.empty[stage], parity ^ 1
                whole = (s + 1) * STEP <= summed
                # this warp's block of the step (all of it, or the half that is not gathered;
                # a last step's comes from the others), and the gathering warps' or the tail's
                expect = 1 if not self.gather else self.gather + (1 if whole else 0)
                self.stage_step[stage] = it
                self.full[stage].arrive(expect)
                if whole:
                    self.copy(stage, it)
                elif not self.gather:
                    self.tail[stage].arrive()
                it += 1
        for p in range(max(0, it - self.stages), it):
            yield self.empty[p % self.stages], p // self.stages % 2

    def last_rows(self):
        it, phases = 0, [0] * self.stages
        for summed in self.sums:
            it += self.steps(summed)
            if summed % STEP == 0:
                continue
            stage = (it - 1) % self.stages
            yield self.tail[stage], phases[stage]
            phases[stage] ^= 1
            self.copy(stage, it - 1)

    def follow_empty(self):
        it = 0
        for summed in self.sums:
            for s in range(self.steps(summed)):
                yield self.empty[it % self.stages], it // self.stages % 2 ^ 1
                if (s + 1) * STEP > summed:
                    self.copy(it % self.stages, it)
                it += 1

    def rows(self, stage):
        it = stage
        for _ in range(stage, sum(map(self.steps, self.sums)), self.stages):
            yield self.empty[stage], it // self.stages % 2 ^ 1
            self.copy(stage, it)
            it += self.stages

    def products(self):
        it = acc = 0
        for summed in self.sums:
            steps = self.steps(summed)
            for s in range(steps):
                first = s % self.segment == 0 if self.segment else s == 0
                if first:
                    yield self.acc_empty[acc % 2], acc // 2 % 2 ^ 1
                stage = it % self.stages
                yield self.full[stage], it // self.stages % 2
                assert self.stage_step[stage] == it, "a product of another step's operands"
                self.used.append(it)
                self.stage_step[stage] = None
                self.empty[stage].arrive()
                if s + 1 == steps or self.segment and s % self.segment == self.segment - 1:
                    self.acc_full[acc % 2].arrive()
                    acc += 1
                it += 1

    def results(self):
        acc = 0
        for summed in self.sums:
            steps = self.steps(summed)
            for _ in range(0, steps, self.segment or max(steps, 1)):
                yield self.acc_full[acc % 2], acc // 2 % 2
                self.acc_empty[acc % 2].arrive()
                acc += 1

    def run(self, choose):
        """Until every role has ended; False if none can go on."""
        waits = {}
        for name, role in list(self.roles.items()):
            waits[name] = next(role, None)
        while True:
            waits = {n: w for n, w in waits.items() if w is not None}
            if not waits and not self.flights:
                return self.used == list(range(sum(map(self.steps, self.sums))))
            ready = [n for n, (bar, parity) in waits.items() if bar.passes(parity)]
            ready += ["copy"] * bool(self.flights)
            if not ready:
                return False
            name = choose(ready)
            if name == "copy":
                self.land(0)
            else:
                waits[name] = next(self.roles[name], None)


def orders(model_of):
    """Every role as the slowest, every role as the fastest, and random orders."""
    names = [*model_of().roles, "copy"]
    for slow in names:
        yield lambda ready, slow=slow: min(ready, key=lambda n: (n == slow, n))
        yield lambda ready, slow=slow: min(ready, key=lambda n: (n != slow, n))
    for seed in range(40):
        yield random.Random(seed).choice


TILES = [[128, 70, 0, 64, 1, 640, 130, 63, 65] * 3, [1] * 20, [64] * 20, [1000, 0, 1000],
         [64 * 7, 1] * 8, [0, 0, 5]]


@pytest.mark.parametrize("sums", TILES)
@pytest.mark.parametrize("stages", [4, 6])
@pytest.mark.parametrize("gather,segment", [(0, None), (0, 10), (1, 10), (2, None), (0, 1)])
def test_every_order_ends(sums, stages, gather, segment):
    def model():
        return Model(sums, stages, gather, segment)
    for choose in orders(model):
        assert model().run(choose)


def test_the_model_finds_a_follower_that_is_late():
    def model():
        return Model(TILES[0], 6, late_follower=True)
    assert not all(model().run(choose) for choose in orders(model))


def test_the_kernel_has_the_rule_of_the_model():
    """The warp that copies a sum's last rows waits on `tail` alone."""
    text = open(SOURCE).read()
    role = text[text.index("KIND == kWgrad && !GATHER && warp == 2"):]
    waits = re.findall(r"mbar_wait_long\((\w+) \+", role[:role.index("atomicOr")])
    assert waits == ["tail"]


def test_signals_between_the_ctas_of_a_pair_have_cluster_scope():
    """Every barrier but `tail` is signalled by the other CTA of a pair too."""
    waits = re.findall(r"mbar_wait_long(<PAIR>)?\((\w+) \+", open(SOURCE).read())
    assert {bar for _, bar in waits} == {"full", "empty", "tail", "acc_full", "acc_empty"}
    assert all((scope == "<PAIR>") == (bar != "tail") for scope, bar in waits)
    helpers = open(SOURCE.replace("grouped_gemm.cu", "experts.cuh")).read()
    arrive = helpers[helpers.index("void mbar_arrive_cluster"):]
    assert re.search(r"mbarrier\.arrive\.\w+\.(\w+)", arrive).group(1) == "cluster"
    assert "try_wait.parity.acquire.cluster" in helpers
