"""The page operators against a model of lists on the host: pages taken, given back,
shared, moved and copied.  Whole numbers throughout, so everything is equal."""
import ctypes
import random

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def tsa():
    import top_retrieval_sparse_gb300 as t
    t.lib()
    return t


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Model:
    """A pool by the definitions, one entry at a time."""

    def __init__(self, B, max_pages, n_pages, ps):
        self.table = [[-1] * max_pages for _ in range(B)]
        self.refs = [0] * n_pages
        self.ps, self.max = ps, max_pages

    def alloc(self, lo, hi):
        free = [p for p, r in enumerate(self.refs) if r == 0]
        cap, want = self.max * self.ps, []
        for b, (a, z) in enumerate(zip(lo, hi)):
            a, z = max(a, 0), min(z, cap)
            if a < z:
                want += [(b, j) for j in range(a // self.ps, -(-z // self.ps))
                         if self.table[b][j] < 0]
        if len(want) > len(free):
            return False
        for (b, j), p in zip(want, free):
            self.table[b][j], self.refs[p] = p, 1
        return True

    def free(self, lo, hi):
        for b, (a, z) in enumerate(zip(lo, hi)):
            for j in range(self.max):
                p = self.table[b][j]
                if p >= 0 and j * self.ps >= a and (j + 1) * self.ps <= z:
                    self.refs[p] -= 1
                    self.table[b][j] = -1

    def fork(self, parents, children, lens):
        free = iter([p for p, r in enumerate(self.refs) if r == 0])
        rows, moves = [], []
        for p, n in zip(parents, lens):
            full = n // self.ps
            row = self.table[p][:full] + [-1] * (self.max - full)
            src = dst = -1
            if n % self.ps and self.table[p][full] >= 0:
                src, dst = self.table[p][full], next(free)
                row[full] = dst
            rows.append(row)
            moves.append((src, dst))
        for c, row in zip(children, rows):
            for p in self.table[c]:
                if p >= 0:
                    self.refs[p] -= 1
            for p in row:
                if p >= 0:
                    self.refs[p] += 1
            self.table[c] = row
        return moves

    def compact(self):
        live = sum(r > 0 for r in self.refs)
        holes = [p for p in range(live) if self.refs[p] == 0]
        high = [p for p in range(live, len(self.refs)) if self.refs[p] > 0]
        to = dict(zip(high, holes))
        for a, z in to.items():
            self.refs[z], self.refs[a] = self.refs[a], 0
        self.table = [[to.get(p, p) for p in row] for row in self.table]
        return list(zip(high, holes))

    def same(self, pages):
        return pages.table.tolist() == self.table and pages.refs.tolist() == self.refs


@pytest.mark.parametrize("B,max_pages,n_pages,ps,seed", [
    (1, 1, 1, 16, 0), (3, 7, 10, 16, 1), (5, 40, 130, 64, 2), (40, 33, 700, 32, 3),
    (300, 9, 2100, 256, 4), (4, 3000, 5000, 16, 5), (17, 1025, 9000, 128, 6)])
def test_a_pool_over_many_calls(tsa, B, max_pages, n_pages, ps, seed):
    """Sequences grow, leave, are cut, forked and moved in any order."""
    rng = random.Random(seed)
    pages, m = tsa.Pages.empty(B, max_pages, n_pages, ps), Model(B, max_pages, n_pages, ps)
    cap = max_pages * ps
    lens = [0] * B
    for step in range(25):
        kind = rng.choice(["grow", "grow", "leave", "cut", "window", "fork", "compact"])
        if kind == "grow":
            new = [min(cap, n + rng.choice([0, 1, 1, ps, rng.randint(0, cap // 2)])) for n in lens]
            tsa.pages_alloc(pages, i32(lens), i32(new))
            good = m.alloc(lens, new)
            status = tsa.lib().tsa_workspace_status(pages.workspace.data_ptr(), 1, None)
            assert (status == 0) == good
            if good:
                lens = new
        elif kind in ("leave", "cut", "window"):
            some = [rng.random() < 0.4 for _ in range(B)]
            lo = [0] * B if kind == "leave" else [rng.randint(0, n) for n in lens]
            hi = [cap if kind != "window" else rng.randint(0, n) for n in lens]
            hi = [h if s else 0 for h, s in zip(hi, some)]
            tsa.pages_free(pages, i32(lo), i32(hi))
            m.free(lo, hi)
            if kind != "window":
                lens = [min(n, a) if s else n for n, a, s in zip(lens, lo, some)]
        elif kind == "fork":
            ids = rng.sample(range(B), rng.randint(0, B))
            kids = ids[: rng.randint(0, len(ids))]
            pool = ids[len(kids):]
            if not kids or not pool:
                continue
            par = [rng.choice(pool) for _ in kids]
            take = [rng.randint(0, lens[p]) for p in par]
            if sum(n % ps > 0 for n in take) > m.refs.count(0):
                continue
            src, dst = tsa.pages_fork(pages, i32(par), i32(kids), i32(take))
            assert list(zip(src.tolist(), dst.tolist())) == m.fork(par, kids, take)
            for c, n in zip(kids, take):
                lens[c] = n
        else:
            src, dst, count = tsa.pages_compact(pages)
            moves, k = m.compact(), int(count)
            assert list(zip(src.tolist(), dst.tolist()))[:k] == moves and k == len(moves)
            assert (src[k:] == -1).all() and (dst[k:] == -1).all()
        assert m.same(pages), (step, kind)
    assert tsa.workspace_status(pages.workspace) == 0


def test_a_large_pool(tsa):
    """A million pages: counts past one block's prefix, ranks in the last words."""
    B, per, n, ps = 64, 8192, (1 << 20) + 37, 16
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    perm = torch.randperm(n, generator=g, device=DEV)
    table = torch.full((B, per), -1, dtype=torch.int32, device=DEV)
    keep = torch.randint(0, per, (B,), generator=g, device=DEV)
    on = torch.arange(per, device=DEV) < keep[:, None]
    table[on] = perm[: int(on.sum())].int()
    refs = torch.zeros(n, dtype=torch.int32, device=DEV)
    refs[table[on].long()] = 1
    t0, r0 = table.clone(), refs.clone()
    pages = tsa.Pages(table, refs, ps)
    cap = i32([per * ps] * B)
    tsa.pages_alloc(pages, i32([0] * B), cap)
    free = (r0 == 0).nonzero().flatten()[: int((~on).sum())]
    want = t0.clone()
    want[~on] = free.int()
    assert torch.equal(table, want) and int(refs.sum()) == B * per
    # half of the sequences leave, the rest moves down
    tsa.pages_free(pages, i32([0] * B), i32([per * ps, 0] * (B // 2)))
    was, held = table.clone(), refs.clone()
    src, dst, count = tsa.pages_compact(pages)
    live = int((held > 0).sum())
    holes = (held[:live] == 0).nonzero().flatten()
    high = (held[live:] > 0).nonzero().flatten() + live
    k = int(count)
    assert k == len(holes) and torch.equal(src[:k].long(), high) and torch.equal(dst[:k].long(),
                                                                                 holes)
    to = torch.arange(n, device=DEV)
    to[high] = holes
    assert torch.equal(table, torch.where(was >= 0, to[was.clamp(min=0).long()].int(), was))
    assert (refs[:live] == 1).all() and (refs[live:] == 0).all()
    assert tsa.workspace_status(pages.workspace) == 0


def test_refused_calls_change_nothing(tsa):
    """Too few pages, children named twice, parents that are children, indices and
    lengths out of range, entries outside the pool."""
    def fresh():
        pages = tsa.Pages.empty(4, 8, 6, 16)
        tsa.pages_alloc(pages, i32([0] * 4), i32([40, 16, 0, 0]))   # 3 + 1 pages of 6
        assert tsa.workspace_status(pages.workspace) == 0
        return pages, pages.table.clone(), pages.refs.clone()

    def flagged(pages, t, r):
        assert int(tsa.lib().tsa_workspace_status(pages.workspace.data_ptr(), 1, None)) != 0
        assert torch.equal(pages.table, t) and torch.equal(pages.refs, r)

    pages, t, r = fresh()
    tsa.pages_alloc(pages, i32([0] * 4), i32([40, 16, 33, 0]))      # 3 more, 2 free
    flagged(pages, t, r)
    for par, kid, n in (([0, 0], [2, 2], [40, 40]), ([0, 2], [2, 3], [40, 0]), ([4], [2], [1]),
                        ([-1], [2], [1]), ([0], [4], [1]), ([0], [-1], [1]), ([0], [0], [8]),
                        ([0], [2], [129]), ([0], [2], [-1])):
        pages, t, r = fresh()
        src, dst = tsa.pages_fork(pages, i32(par), i32(kid), i32(n))
        assert (src == -1).all() and (dst == -1).all()
        flagged(pages, t, r)
    pages, t, r = fresh()
    src, dst = tsa.pages_fork(pages, i32([0, 1, 0]), i32([2, 3, 1]), i32([40, 8, 40]))
    assert (src == -1).all()                                        # 1 is parent and child
    flagged(pages, t, r)
    pages, t, r = fresh()
    pages.table[0, 1] = t[0, 1] = 6                                 # outside the pool
    src, dst = tsa.pages_fork(pages, i32([0]), i32([2]), i32([40]))
    assert (src == -1).all()
    flagged(pages, t, r)


def test_wrong_states_are_flagged_not_followed(tsa):
    """Entries outside the pool and counts that do not match the tables."""
    def status(pages):
        return int(tsa.lib().tsa_workspace_status(pages.workspace.data_ptr(), 1, None))

    pages = tsa.Pages(i32([[0, 9, 1], [1, -1, -1]]), i32([1, 1, 0, 0]), 16)
    tsa.pages_free(pages, i32([0, 0]), i32([48, 48]))
    # page 9 is outside, page 1 counts one entry and is named by two
    assert pages.refs.tolist() == [0, 0, 0, 0] and (pages.table == -1).all()
    assert status(pages) != 0
    pages = tsa.Pages(i32([[3, 7, 2, -1]]), i32([0, 0, 0, 1]), 16)
    src, dst, count = tsa.pages_compact(pages)
    # 3 moves to 0; 7 is outside, 2 counts as free
    assert int(count) == 1 and src[0] == 3 and dst[0] == 0
    assert pages.table.tolist() == [[0, 7, 2, -1]] and pages.refs.tolist() == [1, 0, 0, 0]
    assert status(pages) != 0
    pages = tsa.Pages.empty(2, 4, 8, 16)
    tsa.pages_alloc(pages, i32([-5, 0]), i32([10, 1000]))           # clipped to [0, 64)
    assert pages.table.tolist() == [[0, -1, -1, -1], [1, 2, 3, 4]]
    assert status(pages) != 0
    tsa.pages_alloc(pages, i32([60, 30]), i32([20, 30]))            # nothing
    tsa.pages_free(pages, i32([10, -3]), i32([5, 17]))
    assert pages.table.tolist() == [[0, -1, -1, -1], [-1, 2, 3, 4]]
    assert status(pages) == 0


@pytest.mark.parametrize("fmt,Hkv,ps,layers", [("bf16", 1, 16, 1), ("bf16", 8, 256, 2),
                                               ("int8", 1, 16, 3), ("int8", 3, 32, 1),
                                               ("e4m3", 4, 128, 40)])
def test_copy_moves_whole_pages_and_nothing_else(tsa, fmt, Hkv, ps, layers):
    """All layers in one call, scales of 4 bytes a page among them; pairs of -1 and
    behind the count do nothing; pages outside the pool are skipped and flagged."""
    g = torch.Generator(device=DEV)
    g.manual_seed(ps)
    n = 37
    pt = torch.zeros((1, 4), dtype=torch.int32, device=DEV)
    caches, bufs = [], []
    for _ in range(layers):
        if fmt == "bf16":
            k, v = (torch.randn((n, Hkv, ps, 128), generator=g, device=DEV).bfloat16()
                    for _ in range(2))
            caches.append(tsa.kv_paged(k, v, pt))
            bufs += [k, v]
        else:
            c = tsa.KV8.paged(n, Hkv, ps, pt, min(ps, 128), fmt)
            for x in (c.k, c.v):
                x.copy_(torch.randint(0, 256, x.shape, generator=g, device=DEV).byte())
            for x in (c.k_scale, c.v_scale):
                x.copy_(torch.rand(x.shape, generator=g, device=DEV))
            caches.append(c)
            bufs += [c.k, c.v, c.k_scale, c.v_scale]
    want = [b.clone() for b in bufs]
    perm = torch.randperm(n, generator=g, device=DEV)
    src, dst = perm[:12].int().contiguous(), perm[12:24].int().contiguous()
    src[3] = -1
    for w in want:
        for a, z in zip(src[:9].tolist(), dst[:9].tolist()):
            if a >= 0:
                w[z] = w[a]
    tsa.pages_copy(caches, src, dst, i32([9]))
    assert all(torch.equal(b, w) for b, w in zip(bufs, want))
    for w in want:
        for a, z in zip(src[9:].tolist(), dst[9:].tolist()):
            w[z] = w[a]
    tsa.pages_copy(caches, src, dst, i32([99]))       # a count past the list: all of it
    tsa.pages_copy(caches, src, dst)
    tsa.pages_copy(caches, src, dst, i32([-1]))
    assert all(torch.equal(b, w) for b, w in zip(bufs, want))
    if fmt != "bf16":
        assert tsa.workspace_status(caches[0].status) == 0
    tsa.pages_copy(caches, i32([n, 0, 1]), i32([1, n, -1]))
    assert all(torch.equal(b, w) for b, w in zip(bufs, want))
    if fmt != "bf16":
        assert int(tsa.lib().tsa_workspace_status(caches[0].status.data_ptr(), 1, None)) != 0


def test_pages_on_streams_and_in_graphs(tsa):
    """Two graphs that share the workspace, replayed by turns, and a stream of its own."""
    B, per, n, ps = 6, 20, 100, 16
    pages, m = tsa.Pages.empty(B, per, n, ps), Model(B, per, n, ps)
    lo, hi, zero, cap = i32([0] * B), i32([100, 1, 0, 320, 17, 16]), i32([0] * B), i32([320] * B)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    tsa.pages_alloc(pages, lo, hi, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    m.alloc([0] * B, hi.tolist())
    assert m.same(pages)
    par, kid, take = i32([0, 3]), i32([1, 2]), i32([99, 48])
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    with torch.cuda.graph(graphs[0]):
        pages_out = tsa.pages_fork(pages, par, kid, take)
    with torch.cuda.graph(graphs[1]):
        tsa.pages_free(pages, zero, cap)
        tsa.pages_alloc(pages, lo, hi)
        moves = tsa.pages_compact(pages)
    for _ in range(3):
        graphs[0].replay()
        assert list(zip(*(x.tolist() for x in pages_out))) == m.fork([0, 3], [1, 2], [99, 48])
        assert m.same(pages)
        graphs[1].replay()
        m.free([0] * B, [320] * B)
        m.alloc([0] * B, hi.tolist())
        assert int(moves[2]) == len(m.compact())
        assert m.same(pages)
    assert tsa.workspace_status(pages.workspace) == 0


@pytest.mark.parametrize("entry", [1, 5, 6, 9], ids=["free below", "free above", "outside", "far outside"])
def test_compaction_flags_every_wrong_entry(tsa, entry):
    """One entry that names no page in use, the only wrong one: left as it is and flagged.  (A free
    page below those in use is a hole that another page moves into.)"""
    def run(last):
        pages = tsa.Pages(i32([[0, 2, 4, -1], [last, -1, -1, -1]]), i32([1, 0, 1, 0, 1, 0]), 16)
        src, dst, count = tsa.pages_compact(pages)
        assert src.tolist() == [4, -1, -1] and dst.tolist() == [1, -1, -1] and int(count) == 1
        assert pages.table.tolist() == [[0, 2, 1, -1], [last, -1, -1, -1]]
        assert pages.refs.tolist() == [1, 1, 1, 0, 0, 0]
        return int(tsa.lib().tsa_workspace_status(pages.workspace.data_ptr(), 1, None))

    assert run(-1) == 0 and run(-7) == 0
    assert run(entry) != 0


def test_large_calls_of_several_host_threads(tsa):
    """Pools and batches of different sizes, whose kernels ask for different amounts of shared
    memory, from two host threads at once: no launch is refused."""
    import threading
    L, codes = tsa.lib(), []

    def pools(n):
        pages = tsa.Pages.empty(2, 64, n, 16)
        lo, hi, st = i32([0, 0]), i32([16, 32]), torch.cuda.Stream()
        args = (pages._ref, lo.data_ptr(), hi.data_ptr(), pages._ws, pages._ws_bytes,
                st.cuda_stream)
        return L.pages_alloc, args, (pages, lo, hi, st)

    def steps(B):
        pt = torch.arange(B, dtype=torch.int32, device=DEV).view(B, 1)
        k = torch.zeros((B, 1, 16, 128), dtype=torch.bfloat16, device=DEV)
        q, lens = torch.zeros((B, 1, 128), dtype=torch.bfloat16, device=DEV), i32([3] * B)
        out, ws = torch.empty((B, 1, 128), device=DEV), tsa.attn_decode_workspace(B, 1, 1)
        kv, st = tsa.kv_paged(k, k, pt), torch.cuda.Stream()
        args = (q.data_ptr(), ctypes.byref(kv.struct), lens.data_ptr(), B, 1, 1, 128, 0, 1 << 30,
                0.1, out.data_ptr(), None, ws.data_ptr(), ws.nbytes, st.cuda_stream)
        return L.window_attn_decode, args, (pt, k, q, lens, out, ws, kv, st)

    def loop(fn, args):
        codes.append({fn(*args) for _ in range(4000)})

    for make, sizes in ((pools, (1 << 22, 1 << 23)), (steps, (4096, 3500))):
        calls = [make(n) for n in sizes]
        torch.cuda.synchronize()
        threads = [threading.Thread(target=loop, args=c[:2]) for c in calls]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        torch.cuda.synchronize()
    assert codes == [{0}] * 4


def test_copies_of_bf16_pages_report_to_the_pages(tsa):
    """A bf16 cache has no status word: pages outside the pool are flagged in the workspace of
    the Pages given."""
    k = torch.randn((7, 2, 16, 128), device=DEV).bfloat16()
    pages = tsa.Pages.empty(2, 4, 7, 16)
    kv = tsa.kv_paged(k, k.clone(), pages.table)
    want = k.clone()
    want[1] = want[0]
    tsa.pages_copy(kv, i32([0]), i32([1]), pages=pages)
    assert torch.equal(kv.k, want) and tsa.workspace_status(pages.workspace) == 0
    tsa.pages_copy([kv, kv], i32([7, 0, -1]), i32([2, 7, 9]), pages=pages)
    assert torch.equal(kv.k, want)
    assert int(tsa.lib().tsa_workspace_status(pages.workspace.data_ptr(), 1, None)) != 0
    cache = tsa.KV8.paged(7, 2, 16, pages.table, 16, "int8")
    tsa.pages_copy([kv, cache], i32([7]), i32([2]), pages=pages)   # a cache's own word first
    assert tsa.workspace_status(pages.workspace) == 0
    assert int(tsa.lib().tsa_workspace_status(cache.status.data_ptr(), 1, None)) != 0


def test_a_fork_onto_entries_that_name_free_pages(tsa):
    """A child's old entries may name pages that count as free (a state that no call leaves), the
    very page that the fork gives out among them: flagged, and the page counts once."""
    for row in ([-1, 2, -1, -1], [2, -1, -1, -1], [-1, -1, 2, -1], [-1, -1, 3, 9]):
        for _ in range(20):
            pages = tsa.Pages(i32([[0, 1, -1, -1], row]), i32([1, 1, 0, 0, 0, 0]), 16)
            src, dst = tsa.pages_fork(pages, i32([0]), i32([1]), i32([24]))
            assert (int(src), int(dst)) == (1, 2)
            assert pages.table.tolist() == [[0, 1, -1, -1], [0, 2, -1, -1]]
            assert pages.refs.tolist() == [2, 1, 1, 0, 0, 0]
            assert int(tsa.lib().tsa_workspace_status(pages.workspace.data_ptr(), 1, None)) != 0


def test_a_fork_of_entries_that_name_free_pages(tsa):
    """A parent's entry that names a page that counts as free: nothing changes, and it is
    flagged; behind the forked positions it does not matter."""
    for take, good in ((40, False), (48, False), (16, False), (33, False), (0, True)):
        pages = tsa.Pages(i32([[3, 1, 0, -1], [-1] * 4]), i32([1, 1, 0, 0, 0, 0]), 16)
        t, r = pages.table.clone(), pages.refs.clone()
        src, dst = tsa.pages_fork(pages, i32([0]), i32([1]), i32([take]))
        status = int(tsa.lib().tsa_workspace_status(pages.workspace.data_ptr(), 1, None))
        assert (status == 0) == good and int(src) == int(dst) == -1
        assert torch.equal(pages.table, t) and torch.equal(pages.refs, r)
    pages = tsa.Pages(i32([[0, 1, 3, -1], [-1] * 4]), i32([1, 1, 0, 0, 0, 0]), 16)
    src, dst = tsa.pages_fork(pages, i32([0]), i32([1]), i32([24]))
    assert (int(src), int(dst)) == (1, 2) and pages.refs.tolist() == [2, 1, 1, 0, 0, 0]
    assert tsa.workspace_status(pages.workspace) == 0


def test_a_pool_without_sequences(tsa):
    pages = tsa.Pages.empty(0, 4, 10, 16)
    none = i32([])
    tsa.pages_alloc(pages, none, none)
    tsa.pages_free(pages, none, none)
    assert tsa.pages_fork(pages, none, none, none)[0].numel() == 0
    src, dst, count = tsa.pages_compact(pages)
    assert int(count) == 0 and (src == -1).all() and (dst == -1).all()
    assert (pages.refs == 0).all() and tsa.workspace_status(pages.workspace) == 0
