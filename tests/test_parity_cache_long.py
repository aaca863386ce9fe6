"""Long writes and prompts of the cache-side operators against 64 bits, and a
shared block whose scale grows under rotated keys."""
import math

import pytest
import torch

from test_parity_cache_ops import (D, DEV, attend64, bf16_cache, gen, grid8, i32, make_cache, place,
                                   prefill_close, randn, rates, scale64, seen_of, tsa,  # noqa: F401
                                   turn64, values)

pytestmark = pytest.mark.gpu


def rows_of(cache, b, lo, hi):
    at = [place(cache, b, p) for p in range(lo, hi)]
    return torch.tensor([x[0] for x in at]), torch.tensor([x[1] for x in at])


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("blk,rot,layout", [(16, 128, "half"), (64, 96, "interleaved"),
                                            (128, 32, "half"), (32, 128, "interleaved")])
def test_a_shared_block_grows_under_rotated_keys(tsa, fmt, blk, rot, layout):
    """Rows written into a block that older rows share, 1 to 200 times as large: the
    scale is the larger of both, the older rows are rounded once more to it."""
    g = gen(blk)
    B, Hkv, cap, page = 4, 3, 1024, 128
    cache = make_cache(tsa, g, B, Hkv, cap, blk, fmt, page)
    table = tsa.RopeTable(rot, cap, 1e4, layout)
    w, amp = rates(rot, 1e4, "none", 1.0, 0)
    lens, news = [blk - 3, 2 * blk + 1, 7 * blk // 2, blk], [2, 5, blk, 1]
    first = randn(g, sum(lens), Hkv, D).bfloat16()
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    tsa.kv8_append(cache, first, first, i32(lens), cu_new=i32(cu), max_new=max(lens), rope=table)
    for amp_b in (1.0, 5.0, 200.0):
        was, had = values(cache), cache.k_scale.double()
        n_at = [0]
        for n in news:
            n_at.append(n_at[-1] + n)
        x = (randn(g, sum(news), Hkv, D) * amp_b).bfloat16()
        start, lens = lens, [a + n for a, n in zip(lens, news)]
        tsa.kv8_append(cache, x, x, i32(lens), cu_new=i32(n_at), max_new=max(news), rope=table)
        now = values(cache)
        for b in range(B):
            pos = torch.arange(start[b], lens[b], device=DEV)
            part = x[n_at[b]:n_at[b + 1]]
            turned, mag = turn64(part, pos, rot, layout, w, amp)
            for j in range(start[b] // blk, (lens[b] - 1) // blk + 1):
                lo, hi = max(start[b], j * blk), min(lens[b], (j + 1) * blk)
                pi, ri = rows_of(cache, b, j * blk, hi)
                s = cache.k_scale.double()[pi[0], :, ri[0] // blk]             # [Hkv]
                need = turned[lo - start[b]:hi - start[b]].abs().amax(dim=(0, 2))
                low, high = scale64(need * (1 - 1e-5), fmt), scale64(need * (1 + 1e-5), fmt)
                if lo > j * blk:
                    old = had[pi[0], :, ri[0] // blk]
                    low, high = torch.maximum(low, old), torch.maximum(high, old)
                assert ((low <= s) & (s <= high)).all()
                n_old = lo - j * blk
                if n_old:   # exact: shifts and one rounding
                    before = was[0][pi[:n_old], :, ri[:n_old]]
                    after = now[0][pi[:n_old], :, ri[:n_old]]
                    assert torch.equal(after, grid8(before / s[None, :, None], fmt) *
                                       s[None, :, None])
                got = now[0][pi[n_old:], :, ri[n_old:]]
                ref = turned[lo - start[b]:hi - start[b]]
                half = s[None, :, None] * 0.5 if fmt == "int8" else \
                    torch.maximum(ref.abs() * 2.0 ** -4, s[None, :, None] * 2.0 ** -10)
                err = mag[lo - start[b]:hi - start[b]] * 2.0 ** -20
                assert ((got - ref).abs() <= half * (1 + 1e-6) + err).all()


@pytest.mark.parametrize("fmt,blk,page,L", [("int8", 64, 0, 100000), ("e4m3", 16, 16, 65537),
                                            ("int8", 128, 256, 70001)])
def test_a_long_write_is_exact(tsa, fmt, blk, page, L):
    g = gen(L)
    Hkv, cap = 2, -(-L // 256) * 256
    cache = make_cache(tsa, g, 1, Hkv, cap, blk, fmt, page)
    x = (randn(g, L, Hkv, D) * torch.exp(2 * randn(g, L, 1, 1))).bfloat16()
    y = randn(g, L, Hkv, D).bfloat16()
    tsa.kv8_append(cache, x, y, i32([L]))
    k, v = tsa.kv8_read(cache, i32([L]), n=L)
    for got, want in ((k, x), (v, y)):
        t = torch.zeros((-(-L // blk) * blk, Hkv, D), dtype=torch.float64, device=DEV)
        t[:L] = want.double()
        t = t.view(-1, blk, Hkv, D)
        s = scale64(t.abs().amax(dim=(1, 3)), fmt)[:, None, :, None]
        assert torch.equal(got.double(), (grid8(t / s, fmt) * s).view(-1, Hkv, D)[:L])


@pytest.mark.parametrize("Hq,Hkv,cap,page,lens,news,ni,nr", [
    (8, 2, 8192, 16, [8000, 5001], [6000, 5001], 4, 700),
    (7, 1, 9000, 0, [9000], [9000], 0, None),
    (4, 4, 4096, 256, [4096, 10, 4095], [4096, 3, 1], 130, 1025)])
def test_long_prompts(tsa, Hq, Hkv, cap, page, lens, news, ni, nr):
    """Prompts of thousands of tokens, ragged: a spread of their tokens."""
    B, G, T = len(lens), Hq // Hkv, sum(news)
    g = gen(cap)
    q = randn(g, T, Hq, D).bfloat16()
    kv, rows = bf16_cache(tsa, g, B, Hkv, cap, page)
    cu = [0]
    for n in news:
        cu.append(cu[-1] + n)
    lse = torch.empty((T, Hq), device=DEV)
    out, _ = tsa.window_attn_prefill(q, kv, i32(lens), ni, nr, i32(cu), max(news), lse_out=lse)
    w = cap if nr is None else nr
    for b, (L, n) in enumerate(zip(lens, news)):
        at = torch.unique(torch.cat([torch.arange(min(n, 70)), torch.arange(max(0, n - 70), n),
                                     torch.arange(0, n, 97)])).to(DEV)
        seen = seen_of(L - n + at, L, ni, w)
        for h in range(Hq):
            r = attend64(q[cu[b] + at, h], rows(kv.k, b, h // G)[:L], rows(kv.v, b, h // G)[:L],
                         seen, 1 / math.sqrt(D))
            prefill_close(out[cu[b] + at, h], lse[cu[b] + at, h], *r, n=L)
