"""Attention over 8-bit caches of which some blocks were never written: their
scales are the zeros that the cache was made with, and so are their values."""
import math

import pytest
import torch

from test_parity_cache_ops import (D, DEV, attend64, decode_close, gen, i32, make_cache, randn,
                                   seen_of, tsa, values)  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("page", [0, 64])
def test_an_unwritten_cache_attends_to_zeros(tsa, fmt, page):
    g = gen(page)
    B, Hq, Hkv, cap = 3, 6, 2, 640
    cache = make_cache(tsa, g, B, Hkv, cap, 32, fmt, page)
    q = randn(g, B, Hq, D).bfloat16()
    lse = torch.empty((B, Hq), device=DEV)
    ws = tsa.attn_decode_workspace(B, Hq, Hkv)
    lens = [1, 640, 77]
    out, _ = tsa.kv8_attn_decode(q, cache, i32(lens), lse_out=lse, workspace=ws)
    assert (out == 0).all()
    # bytes of 0 under scales of 0 (codes of -128 in int8): 448 * 2^-60 at most
    cache.k.zero_(), cache.v.zero_()
    zero, _ = tsa.kv8_attn_decode(q, cache, i32(lens))
    assert (zero.abs() <= 448 * 2.0 ** -60).all()
    k, v = tsa.kv8_read(cache, i32(lens), n=1)
    assert (k == 0).all() and (v == 0).all()
    want = torch.log(torch.tensor(lens, dtype=torch.float64, device=DEV))[:, None]
    assert ((lse.double() - want).abs() <= (1 + want) * 2.0 ** -20).all()
    assert tsa.workspace_status(ws) == 0


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("cap,at,n,big", [(640, 320, 100, 1.0), (640, 32, 600, 1e-6),
                                          (20000 // 32 * 32, 9000, 64, 100.0)])
def test_written_and_unwritten_blocks_together(tsa, fmt, cap, at, n, big):
    """Rows [at, at + n) written; the rows before and after, all seen, are zeros:
    logits of 0 and values of 0 that share the weights' sum."""
    g = gen(at)
    Hq, Hkv, blk = 8, 2, 32
    cache = make_cache(tsa, g, 1, Hkv, cap, blk, fmt, 32)
    x, y = (randn(g, n, Hkv, D).bfloat16() for _ in range(2))
    tsa.kv8_append(cache, x, (y * big).bfloat16(), i32([at + n]))
    val = values(cache)
    k, v = (t[cache.page_table[0].long()].transpose(0, 1).reshape(Hkv, cap, D) for t in val)
    q = randn(g, 1, Hq, D).bfloat16()
    lse = torch.empty((1, Hq), device=DEV)
    for ni, nr in ((0, None), (64, 400)):
        out, _ = tsa.kv8_attn_decode(q, cache, i32([cap - 3]), ni, nr, lse_out=lse)
        seen = seen_of([cap - 4], cap - 3, ni, cap if nr is None else nr).expand(4, cap - 3)
        for h in range(Hkv):
            r = attend64(q[0, 4 * h:4 * h + 4], k[h, :cap - 3], v[h, :cap - 3], seen,
                         1 / math.sqrt(D))
            # weights below 2^-32 of their warp's largest may be dropped: of values
            # up to max |v|, at most cap of them
            decode_close(out[0, 4 * h:4 * h + 4], lse[0, 4 * h:4 * h + 4], *r, n=cap,
                         extra=cap * 2.0 ** -32 * float(v.abs().max()))
