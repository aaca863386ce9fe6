"""One decode step of groups that share their first rows, against 64-bit attention of every
sequence by itself over the group's rows and its own.

Half a step of rounding, relative to the value: bf16 2^-8, fp32 2^-24.
"""
import math

import pytest
import torch

from test_parity_cache_ops import (D, DEV, HALF, attend64, bf16_cache, decode_close, gen, i32,
                                   quant_cache, randn, small_weights, value_steps)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tsa():
    import top_retrieval_sparse_gb300 as t
    t.lib()
    return t


def members(B, cu):
    """(group, first sequence) of every sequence; (-1, itself) outside the groups."""
    out = [(-1, b) for b in range(B)]
    for n in range(len(cu) - 1):
        for b in range(cu[n], cu[n + 1]):
            out[b] = (n, cu[n])
    return out


def close16(out, lse, ref, rlse, pv, zabs, n, extra):
    # as decode_close, the weights in one part (half a step of 16 bits, the shared rows' at
    # most) and the output rounded to bf16
    eps = 2 * (zabs * 2.0 ** -19 + 2.0 ** -17 + 2.0 ** -20 + n * 2.0 ** -27)
    tol = pv * (eps[:, None] + HALF) + (ref.abs() + pv * HALF) * HALF + extra + 1e-30
    assert ((out.double() - ref).abs() <= tol).all()
    empty = rlse.isinf()
    assert torch.equal(lse.isinf(), empty) and (out[empty] == 0).all()
    assert ((lse.double() - rlse).abs()[~empty] <= (eps + rlse.abs() * 2.0 ** -22)[~empty]).all()


def check(q, rows, lens, cu, shared, Hkv, out, lse, scale=1 / math.sqrt(D), steps=None, only=None):
    """rows(b, h): K and V of a sequence and head in its own cache."""
    G = q.shape[1] // Hkv
    for b, (n, first) in enumerate(members(len(lens), cu)):
        if only is not None and b not in only:
            continue
        L, P = lens[b], (shared[n] if n >= 0 else 0)
        P = min(P, L)
        for h in range(Hkv):
            (k0, v0), (k1, v1) = rows(first, h), rows(b, h)
            k, v = torch.cat([k0[:P], k1[P:L]]), torch.cat([v0[:P], v1[P:L]])
            at = slice(h * G, h * G + G)
            seen = torch.ones((G, L), dtype=torch.bool, device=DEV)
            r = attend64(q[b, at], k, v, seen, scale)
            extra = 0.0
            if steps is not None and L:
                s = torch.cat([steps(first, h)[:P], steps(b, h)[P:L]])
                extra = small_weights(q[b, at], k, v, seen, scale, s)
            if out.dtype == torch.bfloat16:
                close16(out[b, at], lse[b, at], *r, n=L, extra=extra)
            else:
                decode_close(out[b, at], lse[b, at], *r, n=L, extra=extra)


CASES = [  # Hq, Hkv, cap, page, lens, cu, shared
    (4, 1, 64, 0, [1], [0, 1], [1]), (8, 1, 64, 16, [17, 30], [0, 2], [16]),
    (6, 2, 640, 0, [640, 520, 0], [0, 3], [513]),
    (5, 5, 1024, 64, [1000, 999], [0, 1, 2], [1000, 0]),
    # sequences outside the groups, groups of one and of none, nothing shared, nothing own
    (28, 4, 1024, 16, [700, 33, 1024, 130, 130, 500, 0, 6], [1, 1, 2, 6], [5, 33, 130]),
    (16, 2, 2048, 256, [2048, 1300, 1290, 1281], [0, 4], [1280]),
    (32, 8, 2048, 128, [2000, 1027, 1150, 1024, 2048], [0, 4], [1023]),
    # one to many tiles of queries (a tile: 128 / G sequences), ragged ends
    (7, 1, 512, 32, [300 + i for i in range(18)], [0, 18], [299]),
    (8, 2, 512, 16, [257 + i % 50 for i in range(33)], [0, 33], [257]),
    (12, 4, 1024, 64, [640 + 7 * i for i in range(43)], [0, 43], [640]),
    (4, 4, 512, 0, [140 + i for i in range(130)], [0, 129], [139]),
    (8, 1, 512, 16, [130] * 65, [0, 33, 65], [129, 130]),
    (28, 4, 768, 128, [400 + 3 * i for i in range(40)], [0, 37, 40], [400, 400]),
    # long shared rows of few sequences, and many groups of two
    (32, 4, 20480, 16, [20000, 20001, 20400], [0, 3], [19999]),
    (4, 1, 30000, 0, [29999, 29000], [0, 2], [28999]),
    (4, 2, 256, 16, [100 + i for i in range(60)], list(range(0, 61, 2)),
     [99 - 3 * (i % 30) for i in range(30)])]


def roomy(B, Hkv, cap, page, row_bytes):
    """A capacity past the 64 MiB up to which shared rows are read for every sequence."""
    unit = max(page, 128)
    need = (64 << 20) // (B * Hkv * row_bytes) + 1
    return max(cap, -(-need // unit) * unit)


@pytest.mark.parametrize("room", [False, True], ids=["small", "large"])
@pytest.mark.parametrize("out16", [False, True], ids=["fp32", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=range(len(CASES)))
def test_shared_attn_decode(tsa, case, out16, room):
    Hq, Hkv, cap, page, lens, cu, shared = case
    B = len(lens)
    cap = roomy(B, Hkv, cap, page, 512) if room else cap
    g = gen(cap + B)
    q = randn(g, B, Hq, D).bfloat16()
    kv, rows = bf16_cache(tsa, g, B, Hkv, cap, page)
    lse = torch.empty((B, Hq), device=DEV)
    out = torch.empty((B, Hq, D), dtype=torch.bfloat16 if out16 else torch.float32, device=DEV)
    ws = tsa.shared_attn_decode_workspace(B, len(shared), Hq, Hkv)
    args = (q, kv, i32(lens), i32(cu), i32(shared))
    tsa.shared_attn_decode(*args, out=out, lse_out=lse, workspace=ws)
    check(q, lambda b, h: (rows(kv.k, b, h), rows(kv.v, b, h)), lens, cu, shared, Hkv, out, lse)
    assert tsa.workspace_status(ws) == 0
    # the same call again on the same workspace, on one full of ones, without one: the same
    again = torch.empty_like(out)
    tsa.shared_attn_decode(*args, out=again, workspace=ws)
    assert torch.equal(out, again)
    ws[256:] = 255
    again.zero_()
    tsa.shared_attn_decode(*args, out=again, workspace=ws)
    assert torch.equal(out, again) and tsa.workspace_status(ws) == 0
    if not out16:
        assert torch.equal(out, tsa.shared_attn_decode(*args)[0])


@pytest.mark.parametrize("room", [False, True], ids=["small", "large"])
@pytest.mark.parametrize("fmt,block", [("int8", 16), ("int8", 64), ("e4m3", 32), ("e4m3", 128)])
@pytest.mark.parametrize("case", CASES, ids=range(len(CASES)))
def test_kv8_shared_attn_decode(tsa, case, fmt, block, room):
    Hq, Hkv, cap, page, lens, cu, shared = case
    B = len(lens)
    if page and block > page:
        block = page
    cap = -(-cap // 128) * 128 if page == 0 else cap
    cap = roomy(B, Hkv, cap, page, 256) if room else cap
    g = gen(cap + B + block)
    q = randn(g, B, Hq, D).bfloat16()
    cache, rows = quant_cache(tsa, g, B, Hkv, cap, block, fmt, page)
    lse = torch.empty((B, Hq), device=DEV)
    ws = tsa.shared_attn_decode_workspace(B, len(shared), Hq, Hkv)
    args = (q, cache, i32(lens), i32(cu), i32(shared))
    for dtype in (torch.float32, torch.bfloat16):
        out = torch.empty((B, Hq, D), dtype=dtype, device=DEV)
        tsa.shared_attn_decode(*args, out=out, lse_out=lse, workspace=ws)
        check(q, lambda b, h: (rows(0, b, h), rows(1, b, h)), lens, cu, shared, Hkv, out, lse,
              steps=lambda b, h: value_steps(cache, b, h))
        again = torch.empty_like(out)
        tsa.shared_attn_decode(*args, out=again, workspace=ws)
        assert torch.equal(out, again)
    assert tsa.workspace_status(ws) == 0


@pytest.mark.parametrize("cap", [1024, 4096], ids=["small", "large"])
@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
def test_other_scales(tsa, scale, cap):
    """Logits of hundreds, of both signs, and none at all."""
    g = gen(11)
    B, Hq, Hkv = 20, 8, 2
    lens, cu, shared = [600 + 9 * i for i in range(20)], [0, 20], [555]
    q = randn(g, B, Hq, D).bfloat16()
    kv, rows = bf16_cache(tsa, g, B, Hkv, cap, 64)
    lse = torch.empty((B, Hq), device=DEV)
    out, _ = tsa.shared_attn_decode(q, kv, i32(lens), i32(cu), i32(shared), scale=scale, lse_out=lse)
    check(q, lambda b, h: (rows(kv.k, b, h), rows(kv.v, b, h)), lens, cu, shared, Hkv, out, lse,
          scale=scale)


@pytest.mark.parametrize("cap", [2048, 16384], ids=["small", "large"])
def test_a_maximum_that_rises_with_every_row(tsa, cap):
    """Keys whose logits grow by 1 every 8 rows: the weights' maximum is raised many times,
    and most weight lies in the last shared rows, or the own ones."""
    g = gen(12)
    B, Hq, Hkv = 9, 8, 1
    q = torch.ones((B, Hq, D), device=DEV).bfloat16()
    k = (torch.arange(cap, device=DEV).clamp(max=2047) / 8.0)[:, None].expand(cap, D) / D
    k = k.expand(B, 1, cap, D).contiguous().bfloat16()
    v = randn(g, B, Hkv, cap, D).bfloat16()
    kv = tsa.kv_contiguous(k, v)
    lens, cu, shared = [2000] * 4 + [2040] * 5, [0, 9], [2000]
    lse = torch.empty((B, Hq), device=DEV)
    out, _ = tsa.shared_attn_decode(q, kv, i32(lens), i32(cu), i32(shared), scale=1.0, lse_out=lse)
    check(q, lambda b, h: (k[b, h], v[b, h]), lens, cu, shared, Hkv, out, lse, scale=1.0)


@pytest.mark.parametrize("out16", [False, True], ids=["fp32", "bf16"])
def test_values_of_one_sign_over_long_shared_rows(tsa, out16):
    """Sums that only grow: 300000 shared rows of values in [1, 2], 24 sequences."""
    g = gen(13)
    B, Hq, Hkv, cap, P = 24, 8, 1, 300032, 300000
    q = (randn(g, B, Hq, D) * 0.1).bfloat16()
    pool = (torch.rand((2, 1, Hkv, cap, D), generator=g, device=DEV) + 1).bfloat16()
    k = (pool[0] - 1.5).expand(B, -1, -1, -1)
    # (paged, so that the sequences need no copies)
    n = cap // 256
    kv = tsa.kv_paged(k[0].reshape(Hkv, n, 256, D).transpose(0, 1).contiguous(),
                      pool[1, 0].reshape(Hkv, n, 256, D).transpose(0, 1).contiguous(),
                      torch.arange(n, device=DEV).int().expand(B, n).contiguous())
    lens, cu, shared = [P + b % 3 for b in range(B)], [0, B], [P]
    lse = torch.empty((B, Hq), device=DEV)
    out = torch.empty((B, Hq, D), dtype=torch.bfloat16 if out16 else torch.float32, device=DEV)
    tsa.shared_attn_decode(q, kv, i32(lens), i32(cu), i32(shared), out=out, lse_out=lse)
    check(q, lambda b, h: (k[0, h], pool[1, 0, h]), lens, cu, shared, Hkv, out, lse,
          only=[0, 1, 7, 16, 23])


@pytest.mark.parametrize("cap", [512, 12288], ids=["small", "large"])
def test_invisible_rows_and_pages_do_not_matter(tsa, cap):
    """NaN behind every length and in the members' unread copies of shared rows; page table
    entries of nothing visible are not looked up."""
    g = gen(14)
    Hq, Hkv, page = 8, 2, 32
    lens, cu, shared = [200, 150, 130, 400, 300, 0], [0, 3, 5], [129, 299]
    B = len(lens)
    kv, rows = bf16_cache(tsa, g, B, Hkv, cap, page)
    q = randn(g, B, Hq, D).bfloat16()
    want, _ = tsa.shared_attn_decode(q, kv, i32(lens), i32(cu), i32(shared))
    pt = kv.page_table.clone()
    dirty = torch.ones(kv.k.shape[0], page, dtype=torch.bool, device=DEV)
    for b, (n, first) in enumerate(members(B, cu)):
        P = shared[n] if n >= 0 else 0
        for i in range(512):
            if (b == first and i < max(P, lens[b])) or (P <= i < lens[b]):
                dirty[pt[b, i // page].long(), i % page] = False
    for t in (kv.k, kv.v):
        t.masked_fill_(dirty[:, None, :, None], math.nan)
    for b, (n, first) in enumerate(members(B, cu)):
        P = shared[n] if n >= 0 else 0
        for j in range(cap // page):
            lo, hi = j * page, (j + 1) * page
            if not (lo < lens[b] and (b == first or hi > P)):
                pt[b, j] = -7
    kv2 = tsa.kv_paged(kv.k, kv.v, pt)
    ws = tsa.shared_attn_decode_workspace(B, 2, Hq, Hkv)
    got, _ = tsa.shared_attn_decode(q, kv2, i32(lens), i32(cu), i32(shared), workspace=ws)
    assert torch.equal(got, want) and tsa.workspace_status(ws) == 0


@pytest.mark.parametrize("cap", [256, 20480], ids=["small", "large"])
def test_bad_input_is_flagged(tsa, cap):
    def status(ws):
        return int(tsa.lib().tsa_workspace_status(ws.data_ptr(), 1, None))

    def same(a, b):
        # other rows in the batch cut the work elsewhere: sums in another order, each within
        # decode_close of 64 bits (values of order 1, zabs about 7: 4.4e-5)
        return torch.allclose(a, b, rtol=0, atol=1e-4)

    g = gen(15)
    Hq, Hkv, page = 4, 2, 16
    lens, cu, shared = [200, 150, 90, 100], [0, 2, 4], [100, 80]
    kv, rows = bf16_cache(tsa, g, 4, Hkv, cap, page)
    q = randn(g, 4, Hq, D).bfloat16()
    ws = tsa.shared_attn_decode_workspace(4, 2, Hq, Hkv)

    def run(lens=lens, cu=cu, shared=shared, kv=kv):
        lse = torch.empty((4, Hq), device=DEV)
        out, _ = tsa.shared_attn_decode(q, kv, i32(lens), i32(cu), i32(shared), lse_out=lse,
                                        workspace=ws)
        s = status(ws)
        nan = out.isnan().all(-1).all(-1)
        assert torch.equal(nan, out.isnan().any(-1).any(-1)) and torch.equal(nan, lse.isnan().all(1))
        return s, nan.tolist(), out

    s, nan, good = run()
    assert s == 0 and not any(nan)
    s, nan, out = run(lens=[200, 99, 90, 100])            # shorter than its shared rows
    assert s != 0 and nan == [False, True, False, False] and same(out[2:], good[2:])
    s, nan, out = run(lens=[200, 0, 90, 100])             # an empty place is none of these
    assert s == 0 and not any(nan) and (out[1] == 0).all() and same(out[0], good[0])
    s, nan, out = run(shared=[100, cap + 1])                  # past the cache
    assert s != 0 and nan == [False, False, True, True]
    s, nan, out = run(shared=[-1, 80])                    # clamped to 0
    assert s != 0 and not any(nan) and same(out[2:], good[2:])
    s, nan, out = run(lens=[200, 150, 90, cap + 44])           # clamped to the cache
    assert s != 0 and not nan[0] and not nan[1] and not nan[2] and same(out[:3], good[:3])
    for bad in ([0, 3, 2], [0, 2, 5], [-1, 2, 4], [4, 0, 4]):
        s, nan, out = run(cu=bad)
        assert s != 0 and all(nan)
    pt = kv.page_table.clone()
    pt[0, 3] = -1                                         # shared rows of group 0
    s, nan, out = run(kv=tsa.kv_paged(kv.k, kv.v, pt))
    assert s != 0 and nan == [True, True, False, False] and same(out[2:], good[2:])
    pt = kv.page_table.clone()
    pt[3, 6] = -1                                         # own rows of sequence 3
    s, nan, out = run(kv=tsa.kv_paged(kv.k, kv.v, pt))
    assert s != 0 and nan == [False, False, False, True] and same(out[:3], good[:3])


def test_without_groups_it_is_the_plain_step(tsa):
    g = gen(16)
    B, Hq, Hkv, cap = 5, 8, 2, 1024
    kv, rows = bf16_cache(tsa, g, B, Hkv, cap, 16)
    q, lens = randn(g, B, Hq, D).bfloat16(), [1024, 1, 0, 500, 77]
    lse = torch.empty((B, Hq), device=DEV)
    for cu, shared in (([0], []), ([5], []), ([0, 0, 0], [3, 4]), ([0, 5], [0])):
        out, _ = tsa.shared_attn_decode(q, kv, i32(lens), i32(cu), i32(shared), lse_out=lse)
        check(q, lambda b, h: (rows(kv.k, b, h), rows(kv.v, b, h)), lens, cu, shared, Hkv, out, lse)


@pytest.mark.parametrize("per", [2, 4], ids=["small", "large"])
def test_the_largest_batch(tsa, per):
    """4096 sequences in 512 groups of one page each."""
    g = gen(17)
    B, Hq, Hkv, ps = 4096, 4, 1, 16
    pt = torch.randperm(B * per, generator=g, device=DEV).view(B, per).int().contiguous()
    k, v = (randn(g, B * per, Hkv, ps, D).bfloat16() for _ in range(2))
    kv = tsa.kv_paged(k, v, pt)
    cu = list(range(0, B + 1, 8))
    shared = [n % 17 for n in range(512)]
    lens = [shared[b // 8] + b % 5 for b in range(B)]
    q = randn(g, B, Hq, D).bfloat16()
    lse = torch.empty((B, Hq), device=DEV)
    out, _ = tsa.shared_attn_decode(q, kv, i32(lens), i32(cu), i32(shared), lse_out=lse)
    flat = [t[pt.long()].reshape(B, per * ps, D) for t in (k, v)]
    check(q, lambda b, h: (flat[0][b], flat[1][b]), lens, cu, shared, Hkv, out, lse,
          only=set(range(0, B, 37)) | set(range(130)) | set(range(B - 20, B)))


@pytest.mark.parametrize("cap", [2048, 12288], ids=["small", "large"])
def test_streams_graphs_and_calls_of_all_sizes_share_a_workspace(tsa, cap):
    g = gen(18)
    Hq, Hkv = 16, 4
    kv, _ = bf16_cache(tsa, g, 40, Hkv, cap, 64)     # (small: 3 sequences' rows)
    cache, _ = quant_cache(tsa, g, 40, Hkv, cap, 32, "int8", 64)
    q = randn(g, 40, Hq, D).bfloat16()
    small = (q[:3], kv, i32([1500, 1400, 1300]), i32([0, 3]), i32([1299]))
    large = (q, cache, i32([1025 + i for i in range(40)]), i32([0, 33, 40]), i32([1000, 1024]))
    ws = tsa.shared_attn_decode_workspace(40, 2, Hq, Hkv)
    want = [tsa.shared_attn_decode(*a)[0] for a in (small, large)]
    for i in (0, 1, 1, 0, 1, 0, 0):
        assert torch.equal(tsa.shared_attn_decode(*(small, large)[i], workspace=ws)[0], want[i])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = tsa.shared_attn_decode(*large, stream=side)[0]
    other = tsa.shared_attn_decode(*small)[0]              # at the same time
    side.synchronize()
    assert torch.equal(got, want[1]) and torch.equal(other, want[0])
    graphs, outs = [], [torch.empty_like(w) for w in want]
    for a, o in zip((small, large), outs):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            tsa.shared_attn_decode(*a, out=o, workspace=ws)
        graphs.append(gr)
    for i in (0, 1, 1, 0):
        outs[i].zero_()
        graphs[i].replay()
        assert torch.equal(outs[i], want[i])
    # new lengths and groups under the captured call
    large[2].copy_(i32([600 + i for i in range(40)]))
    large[3].copy_(i32([0, 5, 39])), large[4].copy_(i32([600, 500]))
    graphs[1].replay()
    assert torch.equal(outs[1], tsa.shared_attn_decode(*large)[0])
    assert tsa.workspace_status(ws) == 0


@pytest.mark.parametrize("fmt", ["bf16", "int8", "e4m3"])
def test_random_batches_match_every_sequence_by_itself(tsa, fmt):
    """Groups of all sizes and lengths in one call, against the decode step of every sequence
    over tables that all name the shared pages; every kind of unit after every other."""
    g = gen(20)
    rng = __import__("random").Random(5)
    for turn in range(24):
        Hq, Hkv = rng.choice([(32, 8), (32, 4), (28, 4), (12, 4), (6, 2), (5, 5), (8, 1)])
        ps = rng.choice([16, 32, 64, 128, 256])
        N = rng.choice([1, 2, 5, 12])
        sizes = [rng.choice([0, 1, 2, 3, 7, 16, 30, 70]) for _ in range(N)]
        P = [rng.choice([0, 1, 127, 128, 129, rng.randint(1, 3000)]) for _ in range(N)]
        P = [x if s else 1 for x, s in zip(P, sizes)]     # (within the cache)
        cu = [rng.choice([0, 0, 2])]
        for s in sizes:
            cu.append(cu[-1] + s)
        B = cu[-1] + rng.choice([0, 1])
        if B == 0:
            continue
        start = [0] * B
        for n in range(N):
            start[cu[n]:cu[n + 1]] = [P[n]] * sizes[n]
        lens = [s + rng.choice([0, 1, 5, 200]) for s in start]
        per = max(-(-max(lens) // ps), (96 << 20) // (B * Hkv * 256 * ps) + 1)  # a large cache
        pages = tsa.Pages.empty(B, per, sum(-(-x // ps) for x in lens) + 5, ps)
        lead = [cu[n] for n in range(N) if sizes[n]]
        first = [lens[b] if b in lead or start[b] == 0 else 0 for b in range(B)]
        tsa.pages_alloc(pages, i32([0] * B), i32(first))
        kids = [b for b in range(B) if start[b] and b not in lead]
        if kids:
            par = [max(x for x in lead if x <= b) for b in kids]
            tsa.pages_fork(pages, i32(par), i32(kids), i32([start[b] // ps * ps for b in kids]))
            # (the partly shared page: a page of its own, its rows up to start not read)
            tsa.pages_alloc(pages, i32([start[b] // ps * ps if b in kids else 0 for b in range(B)]),
                            i32([lens[b] if b in kids else 0 for b in range(B)]))
        assert tsa.workspace_status(pages.workspace) == 0
        n_pages = pages.n_pages
        q = randn(g, B, Hq, D).bfloat16()
        k, v = (randn(g, n_pages, Hkv, ps, D).bfloat16() for _ in range(2))
        if fmt == "bf16":
            cache = tsa.kv_paged(k, v, pages.table)
        else:
            blk = min(ps, rng.choice([16, 32, 64, 128]))
            cache = tsa.KV8.paged(n_pages, Hkv, ps, pages.table, blk, fmt)
            for i in range(0, n_pages, 4096):              # every page a sequence of its own
                j = min(n_pages, i + 4096)
                ids = torch.arange(i, j, device=DEV).int().view(-1, 1)
                one = tsa.KV8(cache.k, cache.v, cache.k_scale, cache.v_scale, fmt, ids)
                flat = [x[i:j].transpose(1, 2).reshape(-1, Hkv, D) for x in (k, v)]
                tsa.kv8_append(one, *flat, i32([ps] * (j - i)))
            # (one scale, so that a child's block of shared and own rows has the leader's too)
            cache.k_scale.fill_(cache.k_scale.max())
            cache.v_scale.fill_(cache.v_scale.max())
        # rows before start in a child's own page are the leader's
        for b in kids:
            a, z = start[b] // ps * ps, start[b]
            if a < z:
                src, dst = (int(pages.table[x, a // ps]) for x in (max(x for x in lead if x <= b), b))
                for x in (cache.k, cache.v):
                    x[dst, :, : z - a] = x[src, :, : z - a]
        for dtype in (torch.float32, torch.bfloat16):
            out = torch.empty((B, Hq, D), dtype=dtype, device=DEV)
            lse, lse1 = (torch.empty((B, Hq), device=DEV) for _ in range(2))
            ws = tsa.shared_attn_decode_workspace(B, N, Hq, Hkv)
            tsa.shared_attn_decode(q, cache, i32(lens), i32(cu), i32(P), out=out, lse_out=lse,
                                   workspace=ws)
            assert tsa.workspace_status(ws) == 0
            step = tsa.window_attn_decode if fmt == "bf16" else tsa.kv8_attn_decode
            want, _ = step(q, cache, i32(lens), 0, None, lse_out=lse1)
            empty = lse1.isinf()
            assert torch.equal(lse.isinf(), empty) and (out[empty] == 0).all()
            assert ((lse - lse1).abs()[~empty] <= 1e-4).all()
            # fp32: both within decode_close of 64 bits (logits' terms add up to about 10, 4.4e-5
            # of values of at most 6 each); bf16: half a step of the weights and of the result
            vmax = 6.0 if fmt == "bf16" else float(max(6.0, 448 * cache.v_scale.max()))
            tol = 1e-4 * vmax if dtype == torch.float32 else 2 * HALF * vmax
            assert ((out.float() - want).abs() <= tol).all(), (turn, dtype)


def test_a_run_of_forked_sequences(tsa):
    """A prompt with an image is written into pages, forked for samples, and the samples go
    on: pages taken, keys rotated by axes and written, attended with the prompt's rows read
    once, against every sequence by itself; some samples leave and the pool is compacted in
    between."""
    g = gen(19)
    B, Hq, Hkv, ps, cap, n_pages = 6, 8, 2, 32, 1024, 100
    pages = tsa.Pages.empty(B, cap // ps, n_pages, ps)
    cache = tsa.KV8.paged(n_pages, Hkv, ps, pages.table, 16, "int8")
    table = tsa.RopeTable(128, 4096, 1e4, sections=(16, 24, 24), order="turns")
    P = 333

    def write(seqs, lens_now, n):
        lens = [0] * B
        had = [0] * B
        for b in seqs:
            lens[b], had[b] = lens_now[b], lens_now[b] - n
        tsa.pages_alloc(pages, i32(had), i32(lens))
        cu = [0]
        for b in range(B):
            cu.append(cu[-1] + (n if b in seqs else 0))
        qkv = randn(g, cu[-1], Hq + 2 * Hkv, D).bfloat16()
        pos = torch.randint(0, 4096, (3, cu[-1]), generator=g, device=DEV).int()
        q, _ = tsa.rope(qkv[:, :Hq], pos, table)
        tsa.kv8_append(cache, qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], i32(lens), i32(cu), n,
                       rope=table, positions=pos)
        return q, lens

    lens = [0] * B
    lens[0] = P
    write([0], lens, P)
    src, dst = tsa.pages_fork(pages, i32([0] * 5), i32([1, 2, 3, 4, 5]), i32([P] * 5))
    tsa.pages_copy(cache, src, dst)
    lens = [P] * B
    live = list(range(B))
    for step in range(40):
        for b in live:
            lens[b] += 1
        q, now = write(live, lens, 1)
        full = torch.zeros((B, Hq, D), dtype=torch.bfloat16, device=DEV)
        full[live] = q
        got, _ = tsa.shared_attn_decode(full, cache, i32(now), i32([0, B]), i32([P]))
        want, _ = tsa.kv8_attn_decode(full, cache, i32(now))
        # both within decode_close of 64 bits: logits' terms add up to about 10, 4.4e-5 each
        assert torch.allclose(got, want, rtol=0, atol=1e-4)
        if step == 20:
            live = [0, 2, 5]
            out = i32([0 if b in live else cap for b in range(B)])
            tsa.pages_free(pages, i32([0] * B), out)
            tsa.pages_copy(cache, *tsa.pages_compact(pages))
            used = int((pages.refs > 0).sum())
            assert int(pages.table.max()) == used - 1
    assert int(pages.refs.sum()) == int((pages.table >= 0).sum())
    assert tsa.workspace_status(pages.workspace) == 0 and tsa.workspace_status(cache.status) == 0


@pytest.mark.parametrize("cap", [256, 20480], ids=["small", "large"])
def test_shared_rows_past_the_cache_are_clamped(tsa, cap):
    """shared[n] and lens[b] beyond the capacity stand for the capacity, and are flagged; a
    sequence shorter than that is still shorter than its shared rows."""
    g = gen(21)
    Hq, Hkv, page = 4, 2, 16
    kv, _ = bf16_cache(tsa, g, 5, Hkv, cap, page)
    q = randn(g, 5, Hq, D).bfloat16()
    ws = tsa.shared_attn_decode_workspace(5, 2, Hq, Hkv)

    def run(lens, shared):
        lse = torch.empty((5, Hq), device=DEV)
        out, _ = tsa.shared_attn_decode(q, kv, i32(lens), i32([0, 3, 5]), i32(shared), lse_out=lse,
                                        workspace=ws)
        return out, lse, int(tsa.lib().tsa_workspace_status(ws.data_ptr(), 1, None))

    want, lse, s = run([cap, cap, cap, 90, 100], [cap, 80])
    assert s == 0 and not want.isnan().any()
    for lens, shared in (([cap] * 3, cap + 1), ([cap] * 3, 2 ** 31 - 1), ([cap + 5, cap, cap + 1], cap),
                         ([cap + 5] * 3, cap + 9)):
        out, l, s = run(lens + [90, 100], [shared, 80])
        assert s != 0 and torch.equal(out, want) and torch.equal(l, lse)
    out, l, s = run([cap, cap - 1, 0, 90, 100], [cap + 1, 80])
    assert s != 0 and out[1].isnan().all() and l[1].isnan().all() and (out[2] == 0).all()
    # (other own rows cut the work elsewhere: as in test_bad_input_is_flagged)
    assert torch.allclose(out[[0, 3, 4]], want[[0, 3, 4]], rtol=0, atol=1e-4)
