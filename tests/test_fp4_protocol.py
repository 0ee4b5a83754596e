"""The barriers between the warps of the 4-bit floating point product (csrc/fp4_gemm.cu), on
the CPU: a model of each role's waits, arrivals and copies, run with every role as the
slowest in turn and in random orders.

A parity wait passes while the barrier's last completed phase has that parity, so a role
may wait only on a barrier that cannot complete two phases without it.  The model has the
kernel's rules; the planted rules break them, which the model must find.
"""
import os
import random
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "moe_finalize_rmsnorm_gb300", "csrc", "fp4_gemm.cu")


class Barrier:
    def __init__(self, count):
        self.count, self.pending, self.bytes, self.phases = count, count, 0, 0

    def passes(self, parity):
        return self.phases % 2 != parity

    def arrive(self, expect=0):
        self.bytes += expect
        self.pending -= 1
        self._complete()

    def landed(self):
        self.bytes -= 1
        self._complete()

    def _complete(self):
        if self.pending == 0 and self.bytes == 0:
            self.phases += 1
            self.pending = self.count


class Model:
    """One CTA with BF16 results.  `tiles` are their rows; `second` is the second
    accumulator's first column."""

    def __init__(self, tiles, steps, stages, group, second, gather=0, planted=None):
        self.tiles, self.steps, self.stages, self.group = tiles, steps, stages, group
        self.second, self.gather, self.planted = second, gather, planted
        idle_arrive = planted != "no arrival without rows"
        self.full = [Barrier(1 + (gather if idle_arrive else 0)) for _ in range(stages)]
        self.empty = [Barrier(1) for _ in range(stages)]
        self.acc_full = [Barrier(1) for _ in range(2)]
        self.acc_empty = [Barrier(2) for _ in range(2)]
        self.shared = Barrier(2)
        self.scale_full = [Barrier(1) for _ in range(2)]
        self.scale_empty = [Barrier(1) for _ in range(2)]
        self.stage_step = [None] * stages      # the step whose copies a stage takes
        self.in_flight = [0] * stages
        self.flights = []
        self.scales = [None] * 2               # the group that a buffer holds
        self.columns = [None] * 512            # the tile whose sums a column holds
        self.issued = []                       # products and commits, in order
        self.roles = {"blocks": self.blocks(), "products": self.products(),
                      "results 0": self.results(0), "results 1": self.results(1),
                      "scales 0": self.team(0), "scales 1": self.team(1)}
        for w in range(gather):
            self.roles[f"gather {w}"] = self.rows(w)

    def quads(self, n, w):
        return max(0, (n // 8 - w + self.gather - 1) // self.gather)

    def copy(self, stage, step):
        assert self.stage_step[stage] in (None, step), "a stage is filled by two steps"
        self.stage_step[stage] = step
        self.in_flight[stage] += 1
        self.flights.append(stage)

    def land(self, i):
        stage = self.flights.pop(i)
        self.in_flight[stage] -= 1
        self.full[stage].landed()

    def blocks(self):
        it = 0
        for n in self.tiles:
            copies = 1 + sum(self.quads(n, w) > 0 for w in range(self.gather))
            for _ in range(self.steps):
                stage = it % self.stages
                yield self.empty[stage], it // self.stages % 2 ^ 1
                self.full[stage].arrive(copies)
                self.copy(stage, it)
                it += 1
        for p in range(max(0, it - self.stages), it):
            yield self.empty[p % self.stages], p // self.stages % 2

    def rows(self, w):
        it = 0
        for n in self.tiles:
            for _ in range(self.steps):
                stage = it % self.stages
                yield self.empty[stage], it // self.stages % 2 ^ 1
                if self.quads(n, w):
                    self.copy(stage, it)
                if self.planted != "no arrival without rows":
                    self.full[stage].arrive()
                it += 1

    def team(self, team):
        groups = len(self.tiles) * -(-self.steps // self.group)
        n = 0
        for g in range(team, groups, 2):
            yield self.scale_empty[team], n % 2 ^ 1
            assert self.scales[team] is None, "scales that are still to be read"
            self.scales[team] = g
            self.scale_full[team].arrive()
            n += 1
        if n:
            yield self.scale_empty[team], n % 2 ^ 1

    def products(self):
        it = group = 0
        before = 0
        for t, n in enumerate(self.tiles):
            a = t % 2
            for s in range(self.steps):
                if s % self.group == 0:
                    yield self.scale_full[group % 2], group // 2 % 2
                if s == 0:
                    waits = [(self.acc_empty[a], t // 2 % 2 ^ 1)]
                    if (before if a else n) > self.second and t > 0:
                        waits.append((self.shared, a ^ 1))
                    if self.planted == "shared columns not waited for":
                        waits = waits[:1]
                    if self.planted == "shared columns first":
                        waits.reverse()
                    for wait in waits:
                        yield wait
                    before = n
                yield self.full[it % self.stages], it // self.stages % 2
                group_end = s + 1 == self.steps or (s + 1) % self.group == 0
                self.issued.append((it, group, t, n, group_end, s + 1 == self.steps))
                group += group_end
                it += 1

    def run_products(self):
        it, group, t, n, group_end, end = self.issued.pop(0)
        stage = it % self.stages
        assert self.stage_step[stage] == it and self.in_flight[stage] == 0, "operands"
        assert self.scales[group % 2] == group, "scales"
        at = self.second if t % 2 else 0
        for c in range(at, at + n):
            assert self.columns[c] in (None, t), "sums that are still to be moved"
            self.columns[c] = t
        self.stage_step[stage] = None
        self.empty[stage].arrive()
        if group_end:
            self.scales[group % 2] = None
            self.scale_empty[group % 2].arrive()
        if end:
            self.acc_full[t % 2].arrive()

    def results(self, half):
        """Half of the warps: every other 32 rows, two at a time."""
        for t, n in enumerate(self.tiles):
            a = t % 2
            yield self.acc_full[a], t // 2 % 2
            for p in (half, half + 4):
                for at in (p, p + 2):
                    r = 32 * (at if a else 7 - at)
                    for c in range(r, min(r + 32, n)):
                        col = c + (self.second if a else 0)
                        assert self.columns[col] == t, "another tile's sums"
                        self.columns[col] = None
                if p == half:
                    self.shared.arrive()
                    yield None   # the rest may take its time
            self.acc_empty[a].arrive()

    def run(self, pick):
        waiting = {name: next(role, "done") for name, role in self.roles.items()}
        while True:
            ready = [n for n, w in waiting.items()
                     if w != "done" and (w is None or w[0].passes(w[1]))]
            ready += ["land"] * bool(self.flights) + ["tensor cores"] * bool(self.issued)
            if not ready:
                left = [n for n, w in waiting.items() if w != "done"]
                assert not left, f"stuck: {left}"
                return
            name = pick(ready)
            if name == "land":
                self.land(random.randrange(len(self.flights)))
            elif name == "tensor cores":
                self.run_products()
            else:
                waiting[name] = next(self.roles[name], "done")


MIXED = [256, 32, 224, 32, 256, 256, 64, 160, 32, 256, 192, 96, 256]
FORMATS = [(4, 160), (8, 208)]   # steps of a group, second accumulator's column: E4M3, E8M0


def schedules(model, seeds=6):
    """Every role (and the copies, and the tensor cores) as the slowest, then random orders."""
    names = list(model().roles) + ["land", "tensor cores"]
    for slow in names:
        def pick(ready, slow=slow):
            others = [r for r in ready if r != slow]
            return random.choice(others or ready)
        random.seed(slow)
        model().run(pick)
    for seed in range(seeds):
        random.seed(seed)
        weight = {}

        def pick(ready):
            for r in ready:
                weight.setdefault(r, random.choice([0.02, 0.2, 1, 5]))
            return random.choices(ready, [weight[r] for r in ready])[0]
        model().run(pick)


@pytest.mark.parametrize("group,second", FORMATS)
@pytest.mark.parametrize("steps", [1, 2, 4, 5, 9])
@pytest.mark.parametrize("gather", [0, 6])
def test_no_schedule_stops_or_overwrites(group, second, steps, gather):
    schedules(lambda: Model(MIXED, steps, 5, group, second, gather))


@pytest.mark.parametrize("planted,gather", [("no arrival without rows", 6),
                                            ("shared columns not waited for", 0),
                                            ("shared columns first", 0)])
def test_the_model_finds_broken_rules(planted, gather):
    with pytest.raises(AssertionError):
        for steps in (1, 2, 9):
            schedules(lambda: Model(MIXED * 3, steps, 5, 4, 160, gather, planted), seeds=40)


def test_the_kernel_has_these_sizes():
    with open(SOURCE) as f:
        text = f.read()
    assert re.search(r"kRows = SUMS \? 192 : 256;", text)
    assert re.search(r"kStages = SUMS \? 6 : 5;", text)
    assert re.search(r"kGatherWarps = 6;", text)
    assert re.search(r"mbar_init\(full \+ 8 \* i, 1 \+ \(GATHER \? 2 \* W::kGatherWarps : 0\)\)", text)
