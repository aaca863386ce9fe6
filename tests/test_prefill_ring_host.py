"""The prompt kernel's ring of K and V tiles, modelled on the CPU: five slots
filled by the copying warp, read by one matrix thread per query tile and passed
by the warp that zeroes rows of V.  Every role only waits on barriers that keep
their last two phases apart, so a role that falls two laps behind takes an old
phase for its own, or waits for one that never ends.  The model runs the roles
in schedules that hold one of them back for as long as any other can move, with
copies that land in any order, and checks what each role finds in its slot.

The number of arrivals that free a slot is read from the kernel's source."""
import os
import random
import re

import pytest

import top_retrieval_sparse_gb300.build as build

SLOTS = 5


class Wrong(Exception):
    pass


class Barrier:
    def __init__(self, count):
        self.count, self.left, self.phase = count, count, 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left, self.phase = self.count, self.phase + 1

    def passed(self, parity):  # what a wait for a phase of this parity sees
        return (self.phase + 1) % 2 == parity


class Ring:
    """n key tiles; edges: tiles whose V is zeroed in part; x: matrix threads."""

    def __init__(self, n, edges, x, counted):
        self.n, self.edges, self.x, self.counted = n, edges, x, counted
        self.full = [Barrier(1) for _ in range(SLOTS)]
        self.empty = [Barrier(x + counted) for _ in range(SLOTS)]
        self.clean = [Barrier(1) for _ in range(SLOTS)]
        self.holds = [None] * SLOTS      # the tile that has landed in a slot
        self.flying = []                 # copies on their way: (slot, item)
        self.zeroed, self.used = set(), {}

    def copy(self):
        for it in range(2 * self.n):
            s = it % SLOTS
            if it >= SLOTS:
                yield lambda: self.empty[s].passed((it // SLOTS - 1) & 1)
                if self.used.get(it - SLOTS, 0) != self.x:
                    raise Wrong("a slot is filled while it is read")
            self.holds[s] = None
            self.flying.append((s, it))

    def land(self, rng):
        s, it = self.flying.pop(rng.randrange(len(self.flying)))
        self.holds[s] = it
        self.full[s].arrive()

    def find(self, it):
        if self.holds[it % SLOTS] != it:
            raise Wrong(f"item {it} is not in its slot")

    def matrix(self, x):
        def read(it):
            self.find(it)
            self.used[it] = self.used.get(it, 0) + 1
            self.empty[it % SLOTS].arrive()

        yield lambda: self.full[0].passed(0)
        read(0)
        for j in range(self.n):
            it = 2 * j + 1
            yield lambda: self.full[it % SLOTS].passed((it // SLOTS) & 1)
            if j in self.edges:
                yield lambda: self.clean[j % SLOTS].passed((j // SLOTS) & 1)
                if j not in self.zeroed:
                    raise Wrong(f"V tile {j} is used before its rows are zeroed")
            read(it)
            if j + 1 < self.n:
                yield lambda: self.full[(it + 1) % SLOTS].passed(((it + 1) // SLOTS) & 1)
                read(it + 1)

    def zero(self):
        for j in range(self.n):
            it = 2 * j + 1
            if self.counted:
                yield lambda: self.full[(it - 1) % SLOTS].passed(((it - 1) // SLOTS) & 1)
                self.empty[(it - 1) % SLOTS].arrive()
            yield lambda: self.full[it % SLOTS].passed((it // SLOTS) & 1)
            if j in self.edges:
                self.find(it)
                self.zeroed.add(j)
            self.clean[j % SLOTS].arrive()
            if self.counted:
                self.empty[it % SLOTS].arrive()

    def run(self, rng, held=None, hold=0):
        """One schedule; role `held` only moves when it is drawn in one of `hold`
        turns, or nothing else can."""
        roles = {"copy": self.copy(), "zero": self.zero()}
        roles.update({f"matrix{x}": self.matrix(x) for x in range(self.x)})
        waits = {name: None for name in roles}
        while roles or self.flying:
            ready = [r for r in roles if waits[r] is None or waits[r]()]
            moves = ready + (["land"] if self.flying else [])
            others = [m for m in moves if m != held]
            if others and held is not None and rng.randrange(hold + 1):
                moves = others
            if not moves:
                raise Wrong(f"nothing can move: {sorted(roles)} wait")
            m = rng.choice(moves)
            if m == "land":
                self.land(rng)
                continue
            try:
                waits[m] = next(roles[m])
            except StopIteration:
                del roles[m]


def schedules(counted, x, runs):
    for seed in range(runs):
        rng = random.Random(seed)
        n = rng.randrange(1, 24)
        edges = {0, n - 1, rng.randrange(n), rng.randrange(n)}
        held = rng.choice([None, "zero", "copy", "matrix0", "land"])
        Ring(n, edges, x, counted).run(rng, held, rng.choice([1, 10, 10 ** 9]))


def arrivals(two):
    src = open(os.path.join(build.CSRC, "window_prefill.cu")).read()
    a, b = re.search(r"mbar_init\(&bar\.empty\[i\], two \? (\d) : (\d)\);", src).groups()
    return int(a if two else b)


@pytest.mark.parametrize("x", [1, 2])
def test_no_schedule_breaks_the_ring(x):
    schedules(arrivals(x == 2) - x, x, 4000)


@pytest.mark.parametrize("x", [1, 2])
def test_the_model_sees_a_reader_that_is_not_counted(x):
    with pytest.raises(Wrong):
        schedules(0, x, 4000)
