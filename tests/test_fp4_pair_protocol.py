"""The barriers of the 4-bit floating point product (csrc/fp4_gemm.cu) over both CTAs of a
pair, on the CPU: a model of each role's waits, arrivals and copies, and of what each wait
orders, run with every role as the slowest in turn and in random orders.

CTA 0 issues the products, which read both CTAs' shared memory, and its barriers take both
CTAs' arrivals; the tensor cores' completions go to both.  The scales are written by ordinary
stores, so each copy of a block to TMEM needs the stores of either CTA ordered before it: by
arrivals that release, at a scope that holds the waiting thread, to a wait that acquires.  A
role knows the stores that are its own and those that it learned of so; a relaxed arrival
hands on nothing.
"""
import os
import random
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "moe_finalize_rmsnorm_gb300", "csrc", "fp4_gemm.cu")


def source():
    with open(SOURCE) as f:
        return f.read()


class Barrier:
    def __init__(self, count):
        self.count, self.pending, self.bytes, self.phases = count, count, 0, 0
        self.handed, self.known = [], []   # (scope, stores): of this phase, of those before

    def passes(self, parity):
        return self.phases % 2 != parity

    def arrive(self, expect=0, scope=None, stores=()):
        """scope: the release's, "cluster" or a CTA's number; None: relaxed."""
        if scope is not None:
            self.handed.append((scope, frozenset(stores)))
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
            self.known, self.handed = self.handed, []

    def learned(self, cta):
        """The stores that a wait of a thread of `cta` orders before it."""
        return set().union(*(stores for scope, stores in self.known if scope in ("cluster", cta)))


class Model:
    """A pair.  `tiles` are their rows; `second` is the second accumulator's first column;
    `segment` the steps after which the sums leave the tensor cores (None: at the end);
    `scope` that of the release with which a team hands its scales over ("cta": its own;
    None: no release)."""

    def __init__(self, tiles, steps, stages, group, second, gather=0, segment=None,
                 scope="cluster", planted=None):
        self.tiles, self.steps, self.stages, self.group = tiles, steps, stages, group
        self.second, self.gather, self.segment = second, gather, segment
        self.scope, self.planted = scope, planted
        pair = range(2)
        self.full = [Barrier(1 + 2 * gather) for _ in range(stages)]            # CTA 0's
        self.empty = [[Barrier(1) for _ in range(stages)] for _ in pair]
        self.acc_full = [[Barrier(1) for _ in pair] for _ in pair]
        self.acc_empty = [Barrier(2 if planted == "half of the results" else 4) for _ in pair]
        self.shared = Barrier(2 if planted == "half of the shared columns" else 4)  # CTA 0's, too
        self.scale_full = [Barrier(2) for _ in pair]                           # CTA 0's
        self.scale_empty = [[Barrier(1) for _ in pair] for _ in pair]
        self.stage_step = [[None] * stages for _ in pair]   # the step whose copies a stage takes
        self.in_flight = [[0] * stages for _ in pair]
        self.flights = []
        self.scales = [[None] * 2 for _ in pair]            # the group that a buffer holds
        self.columns = [[None] * 512 for _ in pair]         # the sums that a column holds
        self.issued = []                                    # products and commits, in order
        self.roles, self.cta, self.stores = {}, {}, {}
        for cta in pair:
            self.add(f"blocks {cta}", cta, self.blocks(cta))
            for i in pair:
                self.add(f"results {cta} {i}", cta, self.results(cta, i))
                self.add(f"scales {cta} {i}", cta, self.team(cta, i))
            for w in range(gather):
                self.add(f"gather {cta} {w}", cta, self.rows(cta, w))
        self.add("products", 0, self.products())

    def add(self, name, cta, role):
        self.roles[name], self.cta[name], self.stores[name] = role, cta, set()

    def groups(self):
        return len(self.tiles) * -(-self.steps // self.group)

    def quads(self, n, w):
        return max(0, (n // 8 - w + self.gather - 1) // self.gather)

    def copy(self, cta, stage, step):
        assert self.stage_step[cta][stage] in (None, step), "a stage is filled by two steps"
        self.stage_step[cta][stage] = step
        self.in_flight[cta][stage] += 1
        self.flights.append((cta, stage))

    def land(self, i):
        cta, stage = self.flights.pop(i)
        self.in_flight[cta][stage] -= 1
        self.full[stage].landed()

    def blocks(self, cta):
        it = 0
        for n in self.tiles:
            copies = 1 + sum(self.quads(n, w) > 0 for w in range(self.gather))
            for _ in range(self.steps):
                stage = it % self.stages
                yield self.empty[cta][stage], it // self.stages % 2 ^ 1
                if cta == 0:
                    self.full[stage].arrive(2 * copies)
                self.copy(cta, stage, it)
                it += 1
        for p in range(max(0, it - self.stages), it):
            yield self.empty[cta][p % self.stages], p // self.stages % 2

    def rows(self, cta, w):
        it = 0
        for n in self.tiles:
            for _ in range(self.steps):
                stage = it % self.stages
                yield self.empty[cta][stage], it // self.stages % 2 ^ 1
                if self.quads(n, w):
                    self.copy(cta, stage, it)
                self.full[stage].arrive()
                it += 1

    def team(self, cta, team):
        name = f"scales {cta} {team}"
        n = 0
        for g in range(team, self.groups(), 2):
            yield self.scale_empty[cta][team], n % 2 ^ 1
            assert self.scales[cta][team] is None, "scales that are still to be read"
            self.scales[cta][team] = g
            self.stores[name].add((cta, g))
            self.scale_full[team].arrive(scope=cta if self.scope == "cta" else self.scope,
                                         stores=self.stores[name])
            n += 1
        if n:
            yield self.scale_empty[cta][team], n % 2 ^ 1

    def products(self):
        it = group = acc = 0
        before = 0
        for t, n in enumerate(self.tiles):
            in_segment = 0
            for s in range(self.steps):
                a = acc % 2
                if s % self.group == 0:
                    yield self.scale_full[group % 2], group // 2 % 2
                    assert {(0, group), (1, group)} <= self.stores["products"], \
                        "scales whose stores this copy is not ordered behind"
                if in_segment == 0:
                    if self.planted != "accumulator not waited for":
                        yield self.acc_empty[a], acc // 2 % 2 ^ 1
                    shared = self.segment is None   # whole accumulators share none
                    if shared and (before if a else n) > self.second and acc > 0:
                        if self.planted != "shared columns not waited for":
                            yield self.shared, a ^ 1
                    before = n
                yield self.full[it % self.stages], it // self.stages % 2
                in_segment += 1
                group_end = s + 1 == self.steps or (s + 1) % self.group == 0
                end = s + 1 == self.steps or in_segment == self.segment
                self.issued.append((it, group, acc, n, in_segment == 1, group_end, end))
                group += group_end
                if end:
                    acc, in_segment = acc + 1, 0
                it += 1

    def run_products(self):
        it, group, acc, n, first, group_end, end = self.issued.pop(0)
        stage = it % self.stages
        at = self.second if acc % 2 else 0
        for cta in range(2):
            assert self.stage_step[cta][stage] == it and not self.in_flight[cta][stage], "operands"
            assert self.scales[cta][group % 2] == group, "scales"
            for c in range(at, at + n):
                assert self.columns[cta][c] == (None if first else acc), \
                    "sums that are still to be moved"
                self.columns[cta][c] = acc
            self.stage_step[cta][stage] = None
            if group_end:
                self.scales[cta][group % 2] = None
            if cta and self.planted == "commits to one CTA":
                continue
            self.empty[cta][stage].arrive()
            if group_end:
                self.scale_empty[cta][group % 2].arrive()
            if end:
                self.acc_full[cta][acc % 2].arrive()

    def move(self, cta, acc, r, n):
        for c in range(r, min(r + 32, n)):
            col = c + (self.second if acc % 2 else 0)
            assert self.columns[cta][col] == acc, "another tile's sums"
            self.columns[cta][col] = None

    def results(self, cta, half):
        """Half of the warps: every other 32 rows, two at a time where the sums stay."""
        acc = 0
        for n in self.tiles:
            for _ in range(-(-self.steps // (self.segment or self.steps))):
                a = acc % 2
                yield self.acc_full[cta][a], acc // 2 % 2
                if self.segment:
                    for r in range(32 * half, n, 64):
                        self.move(cta, acc, r, n)
                        yield None
                else:
                    for p in (half, half + 4):
                        for at in (p, p + 2):
                            self.move(cta, acc, 32 * (at if a else 7 - at), n)
                        if p == half:
                            self.shared.arrive()
                            yield None   # the rest may take its time
                self.acc_empty[a].arrive()
                acc += 1

    def step(self, name):
        return next(self.roles[name], "done")

    def run(self, pick):
        waiting = {name: self.step(name) for name in self.roles}
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
                if waiting[name] is not None:
                    self.stores[name] |= waiting[name][0].learned(self.cta[name])
                waiting[name] = self.step(name)


MIXED = [256, 32, 224, 32, 256, 256, 160, 192, 96, 256]
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


def hand_over():
    """The scope of the release with which the kernel hands the scales over."""
    text = source()
    scales = text[text.index("// Scales.  Two teams"):text.index("// Rows by number, four a copy")]
    assert "scale_full_at = map_to_cta(scale_full, 0)" in scales
    call = re.search(r"fence_proxy_async_smem\(\);\s*__syncwarp\(\);\s*if \(lane == 0\) (\w+)"
                     r"\(scale_full_at \+ 8 \* team\);", scales)[1]
    with open(os.path.join(os.path.dirname(SOURCE), "experts.cuh")) as f:
        body = re.search(rf"void {call}\(uint32_t remote_bar\) \{{(.*?)\n\}}", f.read(), re.S)[1]
    if re.search(r'"fence\.release\.sync_restrict::shared::cta\.cluster;"', body):
        assert re.search(r"fence\.release.*mbar_arrive_cluster\(remote_bar\);", body, re.S)
        return "cluster"
    assert "mbarrier.arrive.relaxed.cluster" in body
    return None


@pytest.mark.parametrize("group,second", FORMATS)
@pytest.mark.parametrize("steps", [1, 4, 9])
@pytest.mark.parametrize("gather", [0, 6])
def test_every_copy_of_scales_is_ordered_behind_their_stores(group, second, steps, gather):
    scope = hand_over()
    schedules(lambda: Model(MIXED, steps, 5, group, second, gather, scope=scope), seeds=4)


@pytest.mark.parametrize("scope", [None, "cta"])
def test_the_model_finds_stores_that_are_not_ordered(scope):
    with pytest.raises(AssertionError, match="not ordered behind"):
        schedules(lambda: Model(MIXED, 9, 5, 4, 160, scope=scope))


SUMS = [(4, 224), (8, 272)]      # the same of moved sums, whose tiles have 192 rows at most


@pytest.mark.parametrize("group,second", SUMS)
@pytest.mark.parametrize("steps", [1, 9, 10, 11, 20, 23])
@pytest.mark.parametrize("gather", [0, 6])
def test_sums_that_leave_the_tensor_cores_on_their_way(group, second, steps, gather):
    """Several accumulators a tile, and segments of ten steps that end inside groups."""
    tiles = [192, 32, 160, 192, 64]
    schedules(lambda: Model(tiles, steps, 6, group, second, gather, segment=10), seeds=4)


@pytest.mark.parametrize("planted", ["commits to one CTA", "shared columns not waited for",
                                     "accumulator not waited for", "half of the results",
                                     "half of the shared columns"])
def test_the_model_finds_broken_rules(planted):
    with pytest.raises(AssertionError):
        schedules(lambda: Model(MIXED * 2, 9, 5, 4, 160, planted=planted), seeds=40)


@pytest.mark.parametrize("planted", ["commits to one CTA", "accumulator not waited for",
                                     "half of the results"])
def test_the_model_finds_broken_rules_of_moved_sums(planted):
    with pytest.raises(AssertionError):
        schedules(lambda: Model([192] * 4, 23, 6, 4, 224, segment=10, planted=planted), seeds=40)


def test_the_kernel_has_these_rules():
    """What the model takes from the source: who arrives on each barrier and how often, the
    sizes, and the waits before an accumulator is written."""
    text = " ".join(source().split())
    for barrier, count in (("empty + 8 * i", "1"), ("acc_full + 8 * i", "1"),
                           ("acc_empty + 8 * i", "kEpilogueWarps * 2"),
                           ("scale_full + 8 * i", "4 * 2"), ("scale_empty + 8 * i", "1"),
                           ("shared_empty", "kEpilogueWarps * 2")):
        assert f" mbar_init({barrier}, {count});" in text, barrier
    for rule in (
            "kRows = SUMS ? 192 : 256;", "kStages = SUMS ? 6 : 5;", "constexpr int kSegment = 10;",
            "kBytes = FORMAT == kMx ? 8 : 16;", "kSteps = 64 / kBytes;", "kColumns = 12 * kWords;",
            "kColumn = kTmemColumns - 2 * kColumns;",
            "kSecond = Scales<FORMAT>::kColumn - Shape<SUMS>::kRows;",
            # the products' waits
            "warp_wait(scale_full + 8 * (group_n & 1), group_n >> 1 & 1, a.timeout_ns)",
            "warp_wait(acc_empty + 8 * (acc_n & 1), (acc_n >> 1 & 1) ^ 1, a.timeout_ns)",
            "if (Acc::kShared > 0 && (acc_n & 1 ? before : n) > Acc::kSecond && acc_n > 0 && "
            "!warp_wait(shared_empty, (acc_n & 1) ^ 1, a.timeout_ns)) return false; before = n;",
            "if (!warp_wait(full + 8 * stage, phase, a.timeout_ns)) return false;",
            # and their completions, to both CTAs
            "const bool group_end = left == 1 || in_group == Sc::kSteps;",
            "const bool end = left == 1 || (SUMS && in_segment == kSegment);",
            "mma_commit<2>(bar); if (group_end) mma_commit<2>(scale_empty + 8 * (group_n & 1)); "
            "if (end) mma_commit<2>(acc_full + 8 * (acc_n & 1));",
            # the results' arrivals, on CTA 0's barriers
            "done_at = map_to_cta(acc_empty, 0);", "shared_at = map_to_cta(shared_empty, 0);",
            "r[i] = 32 * (second ? at : kAll - 1 - at);",
            "if (p == group) { tcgen05_fence_before(); __syncwarp(); "
            "if (lane == 0) mbar_arrive_cluster(shared_at); } "
            "if (p + 2 * kGroups >= kAll) give_back();",
            # the scales' wait, and the copies'
            "ok = warp_wait(scale_empty + 8 * team, (n & 1) ^ 1, a.timeout_ns);",
            "ok = warp_wait(empty + 8 * stage, phase, a.timeout_ns);"):
        assert rule in text, rule
