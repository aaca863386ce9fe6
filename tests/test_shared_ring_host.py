"""The rings of the kernel over shared rows, modelled on the CPU: slots of K and V tiles (8-bit
caches: slots of codes, widened into slots of operands) that two streams of matrix instructions
read, both of them or by turns, and that the zeroing warp passes in order.

Barriers keep their last two phases apart and no more.  A stream passes by the tiles that are
the other's alone, so after a run of units of one key tile it is far ahead of the ring, and must
not wait for a slot before the slot's tile of the lap before is known to have landed.  The model
runs the roles in schedules that hold one of them back for as long as any other can move, with
copies that land in any order, and checks what every role finds in its slot.

Slots, arrivals and how far ahead of the zeroing warp a stream may wait are read from the
kernel's source."""
import os
import random
import re

import pytest

import top_retrieval_sparse_gb300.build as build


def source(name):
    return open(os.path.join(build.CSRC, name)).read()


def number(name, pattern):
    return int(re.search(pattern, source(name)).group(1))


def slots(q8):
    a, b = re.search(r"kSlots = FMT == kFmtBf16 \? (\d) : (\d);", source("shared_prefix.cu")).groups()
    return int(b if q8 else a)


# ------------------------------------------------------------ the list of work
def shares_of(cu, shared, G, Hkv):
    """What every share has, [(key tiles, both streams on every tile, V's last rows zeroed)], as
    the list kernel cuts it."""
    src = "shared_attn.h"
    n_shares = number(src, r"kSharedShares = (\d+);")
    unit = number(src, r"kUnitRows = (\d+);")
    both, alone = (number(src, rf"{x} = (\d+)") for x in ("kCostBoth", "kCostAlone"))
    units, cost, columns, groups = [], 0, 0, 0
    for n, P in enumerate(shared):
        rows = (cu[n + 1] - cu[n]) * G
        if P <= 0 or rows == 0:
            continue
        groups += 1
        columns += -(-rows // unit)
        for t in range(0, rows, unit):
            w = both if min(unit, rows - t) > 128 else alone
            for _ in range(Hkv):
                tiles = -(-P // 128)
                units.append((cost, tiles, w, P % 128 > 0))
                cost += tiles * w
    shares = n_shares
    if groups == 1:
        even = n_shares // columns * columns if columns <= n_shares else 0
        shares = even if even * 10 >= n_shares * 9 else n_shares
    shares = max(1, min(shares, cost // both))
    out = []
    for s in range(shares):
        at, end = -(-cost * s // shares), -(-cost * (s + 1) // shares)
        mine = []
        for c0, tiles, w, tail in units:
            j0 = max(0, -(-(at - c0) // w))
            j1 = min(tiles, -(-(end - c0) // w))
            if j0 < j1:
                mine.append((j1 - j0, w == both, tail and j1 == tiles))
        out.append(mine)
    return out


def passed_by(share):
    """The most tiles in a row of `share` that are the first stream's alone, before one that is
    the second's."""
    most = run = 0
    for tiles, both, _ in share:
        if not both and tiles == 1:
            run += 1
        else:
            most, run = max(most, run), 0
    return most


# ------------------------------------------------------------ the ring
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
    """The segments of a share, [(key tiles, both streams, V's last rows zeroed)].  `lag`: tiles
    that a stream may wait ahead of the zeroing warp's count; None: a wait by parity in its
    place (what the count is there for).  `returned`: codes are given back when their loads have
    returned; else a load may find what its slot holds later."""

    def __init__(self, segs, q8, lag, returned=True):
        self.segs, self.q8, self.lag, self.returned = segs, q8, lag, returned
        self.S, self.raw = slots(q8), number("shared_prefix.cu", r"kRawSlots = (\d)")
        self.tiles = []                     # of every tile: (both, stream, zeroed)
        for n, both, tail in segs:
            for j in range(n):
                self.tiles.append((both, 0 if both else j & 1, tail and j == n - 1))
        bar = lambda count, n: [Barrier(count) for _ in range(n)]  # noqa: E731
        src = source("shared_prefix.cu")
        count = lambda name: int(re.search(  # noqa: E731
            rf"mbar_init\(&bar\.{name}\[i\], (\d)\);", src).group(1))
        self.full = bar(4 if q8 else 1, self.S)
        self.empty, self.raw_full = bar(count("empty"), self.S), bar(count("raw_full"), self.raw)
        self.raw_empty, self.scale = bar(count("raw_empty"), self.raw), bar(count("scale"), self.raw)
        self.clean, self.turn = bar(1, self.S), bar(1, 2)
        self.q, self.s, self.p, self.o = (bar(1, 2) for _ in range(4))
        self.holds = [[None] * 4 for _ in range(self.S)]  # the item in a slot, by quarters
        self.raw_holds = [None] * self.raw
        self.scale_holds = [None] * self.raw
        self.flying = []                    # copies on their way: (slot, item)
        self.queue = [[], []]               # matrix instructions and arrivals, in order
        self.passed, self.zeroed = 0, set()
        self.used, self.taken, self.done = {}, {}, [0, 0]

    # -- what a slot is asked for
    def readers(self, tile):
        return 2 if self.tiles[tile][0] else 1

    def free(self, it):
        if it >= self.S and self.used.get(it - self.S, 0) != self.readers((it - self.S) // 2):
            raise Wrong(f"slot of item {it - self.S} is filled while it is read")

    def read(self, x, it):
        if self.holds[it % self.S] != [it] * 4:
            raise Wrong(f"stream {x} wants item {it}, its slot holds {self.holds[it % self.S]}")
        tile = it // 2
        if it & 1 and not self.q8 and self.tiles[tile][2] and tile not in self.zeroed:
            raise Wrong(f"V tile {tile} is used before its rows are zeroed")
        self.used[it] = self.used.get(it, 0) + 1
        self.empty[it % self.S].arrive()

    def full_of(self, it):
        return lambda: self.full[it % self.S].passed(it // self.S & 1)

    # -- the roles
    def copy(self):
        n = self.raw if self.q8 else self.S
        for it in range(2 * len(self.tiles)):
            if it >= n:
                bar = (self.raw_empty if self.q8 else self.empty)[it % n]
                yield lambda: bar.passed(it // n & 1 ^ 1)
            if self.q8:
                if it >= n and self.taken.get(it - n, 0) != 4:
                    raise Wrong("codes are overwritten while they are read")
                self.raw_holds[it % n] = None
            else:
                self.free(it)
                self.holds[it % n] = [None] * 4
            self.flying.append((it % n, it))

    def land(self, rng):
        s, it = self.flying.pop(rng.randrange(len(self.flying)))
        if self.q8:
            self.raw_holds[s] = it
            self.raw_full[s].arrive()
        else:
            self.holds[s] = [it] * 4
            self.full[s].arrive()

    def widen(self, w):
        for it in range(2 * len(self.tiles)):
            tile, r = it // 2, it % self.raw
            if w == 0 and not it & 1:
                old = tile - self.raw
                if old >= 0 and self.taken.get(("scale", old), 0) != self.readers(old):
                    raise Wrong("scales are overwritten while they are read")
                self.scale_holds[tile % self.raw] = tile
                self.scale[tile % self.raw].arrive()
            yield lambda: self.raw_full[r].passed(it // self.raw & 1)
            if it >= self.S:
                yield lambda: self.empty[it % self.S].passed(it // self.S & 1 ^ 1)
            self.taken[it] = self.taken.get(it, 0) + 1
            if not self.returned:
                self.raw_empty[r].arrive()
                yield lambda: True
            if self.raw_holds[r] != it:
                raise Wrong("codes of another tile are widened")
            if self.returned:
                self.raw_empty[r].arrive()
            self.free(it)
            self.holds[it % self.S][w] = it
            self.full[it % self.S].arrive()

    def zero(self):
        for tile, (both, _, tail) in enumerate(self.tiles):
            def give(it):
                for _ in range(1 if both else 2):
                    self.empty[it % self.S].arrive()
            yield self.full_of(2 * tile)
            give(2 * tile)
            yield self.full_of(2 * tile + 1)
            if self.holds[(2 * tile + 1) % self.S] != [2 * tile + 1] * 4:
                raise Wrong("rows of another tile are zeroed")
            if tail:
                self.zeroed.add(tile)
            self.clean[tile % self.S].arrive()
            self.passed = tile + 1
            give(2 * tile + 1)

    def known(self, tile):
        if self.lag is not None:
            return lambda: self.passed + self.lag >= tile
        return lambda: tile < 2 or self.clean[(tile - 2) % self.S].passed((tile - 2) // self.S & 1)

    def known_clean(self, tile):
        if self.lag is not None:
            return lambda: self.passed >= tile + 1
        return lambda: self.clean[tile % self.S].passed(tile // self.S & 1)

    def matrix(self, x):
        do = self.queue[x].append

        def qk(it):
            def run():
                self.read(x, it)
                self.done[x] += 1
                self.s[x].arrive()
            do(run)

        tiles = segs = turns = at = 0
        for all_, both, tail in self.segs:
            n = all_ if both else (all_ - x + 1) // 2
            of = lambda j: at + (j if both else 2 * j + x)  # noqa: E731
            if n:
                it = 2 * of(0)
                yield lambda: self.q[x].passed(segs & 1)
                yield self.known(of(0))
                yield self.full_of(it)
                if both and x:
                    yield lambda: self.turn[1].passed(turns & 1)
                qk(it)
                if both:
                    self.turn[x ^ 1].arrive()
            for j in range(n):
                it = 2 * of(j) + 1
                yield self.full_of(it)
                if not self.q8 and tail and of(j) == at + all_ - 1:
                    yield self.known_clean(of(j))
                yield lambda: self.p[x].passed(tiles + j & 1)
                if both:
                    yield lambda: self.turn[x].passed(turns + j + x & 1)
                do(lambda it=it: self.read(x, it))
                if j + 1 < n:
                    yield self.known(of(j + 1))
                    yield self.full_of(2 * of(j + 1))
                    qk(2 * of(j + 1))
                else:
                    do(self.o[x].arrive)
                if both:
                    self.turn[x ^ 1].arrive()
            if both:
                if x == 0:
                    yield lambda: self.turn[0].passed(turns + n & 1)
                turns += n + 1
            tiles, segs, at = tiles + n, segs + (n > 0), at + all_

    def softmax(self, x):
        tiles = segs = at = 0
        for all_, both, _ in self.segs:
            n = all_ if both else (all_ - x + 1) // 2
            if n:
                self.q[x].arrive()
            for j in range(n):
                tile = at + (j if both else 2 * j + x)
                yield lambda: self.s[x].passed(tiles + j & 1)
                if self.done[x] < tiles + j + 1:
                    raise Wrong("logits of another tile are read")
                if self.q8:
                    yield lambda: self.scale[tile % self.raw].passed(tile // self.raw & 1)
                    if self.scale_holds[tile % self.raw] != tile:
                        raise Wrong("scales of another tile are read")
                    key = ("scale", tile)
                    self.taken[key] = self.taken.get(key, 0) + 1
                self.p[x].arrive()
            if n:
                yield lambda: self.o[x].passed(segs & 1)
            tiles, segs, at = tiles + n, segs + (n > 0), at + all_

    def run(self, rng, held=None, hold=0):
        """One schedule; role `held` only moves when it is drawn in one of `hold` turns, or
        nothing else can."""
        roles = {"copy": self.copy(), "zero": self.zero()}
        for x in range(2):
            roles[f"matrix{x}"], roles[f"softmax{x}"] = self.matrix(x), self.softmax(x)
        for w in range(4 if self.q8 else 0):
            roles[f"widen{w}"] = self.widen(w)
        waits = {name: None for name in roles}
        while roles or self.flying or any(self.queue):
            moves = [r for r in roles if waits[r] is None or waits[r]()]
            moves += ["land"] * bool(self.flying)
            moves += [f"tensor{x}" for x in range(2) if self.queue[x]]
            others = [m for m in moves if m != held]
            if others and held is not None and rng.randrange(hold + 1):
                moves = others
            if not moves:
                raise Wrong(f"nothing can move: {sorted(roles)} wait")
            m = rng.choice(moves)
            if m == "land":
                self.land(rng)
            elif m.startswith("tensor"):
                self.queue[int(m[-1])].pop(0)()
            else:
                try:
                    waits[m] = next(roles[m])
                except StopIteration:
                    del roles[m]


def lag():
    """Tiles that the kernel lets a stream wait ahead of the zeroing warp's count."""
    return number("shared_prefix.cu", r"constexpr uint32_t kLag = (\d+);")


def loads_returned():
    """Whether who gives a slot of codes back depends on all that was loaded from it."""
    return re.search(r"any \|= c\[e\]\.x \| c\[e\]\.y \| c\[e\]\.z \| c\[e\]\.w;\s+"
                     r"const int by = __any_sync\(0xffffffffu, any != 0u\) \? 0 : 1;\s+"
                     r"__syncwarp\(\);\s+if \(lane == by\) mbar_arrive\(&bar\.raw_empty",
                     source("shared_prefix.cu")) is not None


HELD = [None, "copy", "zero", "land", "matrix0", "matrix1", "softmax0", "softmax1", "tensor0",
        "tensor1", "widen0", "widen3"]


def schedules(lists, q8, ahead, runs, returned=None):
    for seed in range(runs):
        rng = random.Random(seed)
        ring = Ring(lists(rng), q8, ahead, loads_returned() if returned is None else returned)
        ring.run(rng, rng.choice(HELD[: None if q8 else 10]), rng.choice([1, 10, 10 ** 9]))


def short_before_long(rng):
    """Units of one key tile, then a longer one; up to 30 tiles that one stream passes by."""
    return [(1, False, True)] * rng.randrange(31) + [(rng.randrange(2, 9), False, True)]


def mixed(rng):
    """Runs of units of one key tile, longer ones and ones of both streams, in any order."""
    out = []
    for _ in range(rng.randrange(1, 6)):
        kind = rng.randrange(4)
        if kind == 0:
            out += [(1, False, rng.random() < 0.5)] * rng.randrange(1, 20)
        else:
            out.append((rng.randrange(1, 9), kind == 3, rng.random() < 0.5))
    return out


@pytest.mark.parametrize("q8", [False, True], ids=["bf16", "8-bit"])
@pytest.mark.parametrize("lists", [short_before_long, mixed])
def test_no_schedule_breaks_the_ring(q8, lists):
    schedules(lists, q8, lag(), 1500)


@pytest.mark.parametrize("q8", [False, True], ids=["bf16", "8-bit"])
@pytest.mark.parametrize("lists", [short_before_long, mixed])
@pytest.mark.parametrize("ahead", [None, lambda: lag() + 1], ids=["parity", "too far ahead"])
def test_the_model_sees_a_stream_that_takes_another_lap(q8, lists, ahead):
    with pytest.raises(Wrong):
        schedules(lists, q8, ahead and ahead(), 1500)


def test_the_model_sees_codes_that_are_given_back_before_their_loads_return():
    with pytest.raises(Wrong, match="codes of another tile"):
        schedules(mixed, True, lag(), 1500, returned=False)


# Batches (sequences of every group, their shared rows, query heads of a KV head, KV heads) in
# which a share has short units before a long one.
SHORT_BEFORE_LONG = {
    "two short": ([2, 2, 2], [100, 100, 50000], 4, 8),
    "one short": ([4, 4], [100, 32768], 4, 8),
    "sixteen short": ([2] * 17, [100] * 16 + [131072], 4, 8),
    "between": ([2] * 3 + [3] + [2] * 3 + [40, 3], [128, 1, 77, 16384, 100, 128, 5, 700, 30000], 4, 8),
    "more queries": ([16, 1, 30, 16], [64, 128, 20000, 40000], 4, 8),
}


@pytest.mark.parametrize("name", SHORT_BEFORE_LONG)
def test_batches_with_short_units_before_a_long_one(name):
    """Their lists do what they are there for, and no schedule of such a share breaks the ring."""
    sizes, shared, G, Hkv = SHORT_BEFORE_LONG[name]
    cu = [sum(sizes[:i]) for i in range(len(sizes) + 1)]
    shares = shares_of(cu, shared, G, Hkv)
    assert sum(sum(n for n, _, _ in s) for s in shares) == Hkv * sum(
        -(-P // 128) * -(-S * G // 256) for S, P in zip(sizes, shared))
    worst = max(shares, key=passed_by)
    assert passed_by(worst) >= 4 and sum(passed_by(s) > 0 for s in shares) >= 1
    cut = [(min(n, 9 + n % 2), both, tail) for n, both, tail in worst]
    for q8 in (False, True):
        schedules(lambda rng: cut, q8, lag(), 60)


def test_the_list_of_random_batches_covers_every_tile_once():
    rng = random.Random(3)
    for _ in range(200):
        N, G, Hkv = rng.randrange(1, 9), rng.randrange(1, 9), rng.choice([1, 2, 4, 8])
        sizes = [rng.choice([0, 1, 2, 5, 16, 40, 70]) for _ in range(N)]
        shared = [rng.choice([0, 1, 127, 128, 129, rng.randrange(1, 9000)]) for _ in range(N)]
        cu = [sum(sizes[:i]) for i in range(N + 1)]
        shares = shares_of(cu, shared, G, Hkv)
        assert sum(sum(n for n, _, _ in s) for s in shares) == Hkv * sum(
            -(-P // 128) * -(-S * G // 256) for S, P in zip(sizes, shared))
