"""What the decode step's arithmetic promises, each part by inputs that show it:
softmax weights in 16-bit parts that add up to 22 bits and more, sums that are
folded with rounding before truncation adds up, and folded sums that follow the
running maximum.  All formats, against 64 bits."""
import math

import pytest
import torch

from test_parity_cache_ops import D, DEV, gen, i32, randn, tsa  # noqa: F401

pytestmark = pytest.mark.gpu
FORMATS = ["bf16", "int8", "e4m3"]
PARTS = {"bf16": 3, "int8": 2, "e4m3": 2}


def make(tsa, fmt, k, v):
    """A contiguous cache of k, v [B, Hkv, L, D] (what it holds: by `held`)."""
    if fmt == "bf16":
        return tsa.kv_contiguous(k.contiguous(), v.contiguous())
    B, Hkv, L, _ = k.shape
    cache = tsa.KV8.contiguous(B, Hkv, L, 16, fmt)
    step = 1 << 18
    for lo in range(0, L, step):
        n = min(step, L - lo)
        tsa.kv8_append(cache, *(x[:, :, lo:lo + n].transpose(1, 2).reshape(B * n, Hkv, D)
                                for x in (k, v)), i32([lo + n] * B))
    return cache


def held(cache, which, b, h):
    """Values of a sequence and head, 64 bits: which 0 keys, 1 values."""
    t = (cache.k, cache.v)[which][b, h]
    if t.dtype == torch.bfloat16:
        return t.double()
    s = (cache.k_scale, cache.v_scale)[which][b, h].double()
    x = t.double() - 128 if cache.fmt == "int8" else t.view(torch.float8_e4m3fn).double()
    return x * s.repeat_interleave(16)[:, None]


def step(tsa, fmt, *a, **kw):
    if fmt == "bf16":
        return tsa.window_attn_decode(*a, 0, None, **kw)[0]
    return tsa.kv8_attn_decode(*a, **kw)[0]


@pytest.mark.parametrize("fmt", FORMATS)
def test_weights_keep_22_bits(tsa, fmt):
    """Two rows: the first has the maximum and values of 0, the second a weight p
    and values of 1, so out = p / (1 + p) and nothing hides what p loses.  A row's
    logit is one product: exact.  Its exponent is rounded three times within
    2^-24 of |y| <= 1 or 2^-22 (y - m up to 8), the exponential is within 2^-22, parts,
    sums and the division within 2^-22 together: 2^-20 in all.  One part fewer
    would lose up to 2^-18 (bf16) or 2^-12 (fp16)."""
    B, H = 64, 32
    k = torch.zeros((B, H, 16, D), dtype=torch.bfloat16, device=DEV)
    v = torch.zeros_like(k)
    k[:, :, 1, 0] = -1
    v[:, :, 1] = 1
    q = torch.zeros((B, H, D), dtype=torch.bfloat16, device=DEV)
    q[..., 0] = torch.rand((B, H), generator=gen(1), device=DEV) * 0.69
    cache = make(tsa, fmt, k, v)
    assert (held(cache, 0, 0, 0)[1, 0] == -1) and (held(cache, 1, 0, 0)[1] == 1).all()
    out = step(tsa, fmt, q, cache, i32([2] * B), scale=1.0)
    p = torch.exp(-q[..., :1].double())
    off = (out.double() / (p / (1 + p)) - 1).abs()
    assert float(off.max()) <= 2.0 ** -20


def lean(out, ref):
    return float(((out.double() - ref) / ref).mean())


@pytest.mark.parametrize("fmt", FORMATS)
def test_sums_of_many_rows_lean_to_no_side(tsa, fmt):
    """4M rows of 8 heads, values of one sign.  A matrix instruction loses about 3
    steps of 2^-23 of its sum; between two folds are 16 slabs of as many instructions
    as there are parts, half of whose loss counts as the sum grows.  Roundings of the
    exponents and exponentials go both ways and are shared by a row's columns only."""
    g = gen(2)
    H, L = 8, 1 << 22
    k = torch.empty((1, H, L, D), dtype=torch.bfloat16, device=DEV)
    v = torch.empty_like(k)
    for h in range(H):
        k[0, h] = randn(g, L, D)
        v[0, h] = 1 + torch.rand((L, D), generator=g, device=DEV)
    cache = make(tsa, fmt, k, v)
    q = randn(g, 1, H, D).bfloat16()
    out = step(tsa, fmt, q, cache, i32([L]))
    del k, v
    limit = 16 * PARTS[fmt] * 3 * 2.0 ** -23 / 2
    for h in (0, 5):
        p = torch.softmax(held(cache, 0, 0, h) @ q[0, h].double() / math.sqrt(D), 0)
        assert abs(lean(out[0, h], p @ held(cache, 1, 0, h))) <= limit


@pytest.mark.parametrize("fmt", FORMATS)
def test_folded_sums_follow_the_maximum(tsa, fmt):
    """Every 8192 rows come 128 whose weights are 2^17 (2^16) times the others', with
    values of 1 among values of 3: the others' sums, folded by then, are scaled
    down and still count 1e-3 of the output."""
    H, L = 8, 1 << 20
    high = torch.arange(L, device=DEV) % 8192 >= 8064
    k = torch.zeros((1, H, L, D), dtype=torch.bfloat16, device=DEV)
    v = torch.empty_like(k)
    k[..., 0] = torch.where(high, 17.0, 0.0)
    v[:] = torch.where(high, 1.0, 3.0)[:, None]
    cache = make(tsa, fmt, k, v)
    del k, v
    big = 2.0 ** float(held(cache, 0, 0, 0)[8064, 0])   # (17 is not on e4m3's grid: 16)
    assert big == (2.0 ** 16 if fmt == "e4m3" else 2.0 ** 17)
    q = torch.zeros((1, H, D), dtype=torch.bfloat16, device=DEV)
    q[..., 0] = 1
    for L1 in (L, L - 64, 8064 + 3, 8192 * 3 + 5):
        lse = torch.empty((1, H), device=DEV)
        out = step(tsa, fmt, q, cache, i32([L1]), scale=math.log(2), lse_out=lse)
        n = int(high[:L1].sum())
        total = n * big + (L1 - n)
        ref = (n * big + 3 * (L1 - n)) / total
        # weights are powers of two within 2^-21 (the scale's rounding, the exponential);
        # sums as above, and both sums' roundings
        limit = 2.0 ** -21 + 16 * PARTS[fmt] * 3 * 2.0 ** -23 / 2 + 2.0 ** -20
        assert (out.double() / ref - 1).abs().max() <= limit
        assert (lse.double() - math.log(total)).abs().max() <= limit + math.log(total) * 2.0 ** -22
