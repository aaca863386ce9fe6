"""Attention over many rows whose values have one sign, where truncated sums
would be off in one direction: prompts and decode steps against 64 bits."""
import math

import pytest
import torch

from test_parity_cache_ops import (D, DEV, attend64, bf16_cache, gen, i32, prefill_close, randn,
                                   seen_of, tsa)  # noqa: F401

pytestmark = pytest.mark.gpu


def one_sign(g, *shape):
    """bf16 in [1, 2.5), a mean of its own in every column, so that rounded
    results fall anywhere between two steps."""
    return (1 + torch.rand((*shape[:-2], 1, D), generator=g, device=DEV) +
            0.5 * torch.rand(shape, generator=g, device=DEV)).bfloat16()


def test_prefill_sums_of_many_rows_lean_to_no_side(tsa):
    """Matrix instructions truncate.  Between two additions with rounding stand 128
    tiles, 1024 instructions of 16 products, each product's loss below a step of
    2^-23 of the sum and half of that on average over a sum that grows: 2^-10 in all.
    bf16's roundings go both ways: 2^-8 / sqrt(3) each, 6 standard deviations of a
    mean of n."""
    g = gen(1)
    Hq, Hkv, L, T = 32, 8, 1 << 19, 704
    kv = tsa.kv_contiguous(randn(g, 1, Hkv, L, D).bfloat16(), one_sign(g, 1, Hkv, L, D))
    q = randn(g, T, Hq, D).bfloat16()
    out, _ = tsa.window_attn_prefill(q, kv, i32([L]), 0, None)
    off = []
    for t in (0, 63, 350, 703):
        n = L - T + t + 1
        for h in range(0, Hq, 2):
            z = kv.k[0, h // 4, :n].double() @ q[t, h].double() / math.sqrt(D)
            o = torch.softmax(z, 0) @ kv.v[0, h // 4, :n].double()
            off.append((out[t, h].double() - o) / o)
    off = torch.stack(off)
    assert abs(float(off.mean())) <= 2.0 ** -10 + 6 * 2.0 ** -8 / math.sqrt(3 * off.numel())


@pytest.mark.parametrize("Hq,Hkv,T,L,rise", [(32, 32, 700, 36000, 0.0), (32, 32, 700, 36001, 40.0),
                                             (32, 32, 700, 36001, -40.0), (14, 2, 3, 1200000, 0.0),
                                             (4, 1, 100, 300000, 60.0)])
def test_prefill_sums_outside_tensor_memory(tsa, Hq, Hkv, T, L, rise):
    """More than 128 key tiles a CTA, whole and in parts, with logits that rise or
    fall along the rows (by `rise` from the first to the last), so that sums put aside
    are scaled again, and tokens that see nothing yet."""
    g = gen(T + L)
    k = randn(g, 1, Hkv, L, D)
    k[..., 0] = torch.linspace(0, rise, L, device=DEV)
    kv = tsa.kv_contiguous(k.bfloat16(), one_sign(g, 1, Hkv, L, D))
    q = randn(g, T, Hq, D).bfloat16()
    q[..., 0] = math.sqrt(D)
    ws = tsa.window_attn_prefill_workspace(1, Hq, Hkv, T, L, 0, None)
    lse = torch.empty((T, Hq), device=DEV)
    out, _ = tsa.window_attn_prefill(q, kv, i32([L]), 0, None, lse_out=lse, workspace=ws)
    at = torch.tensor([0, T // 2, T - 1], device=DEV)
    seen = seen_of(L - T + at, L, 0, L)
    for h in range(0, Hq, max(1, Hq // 4)):
        r = attend64(q[at, h], kv.k[0, h * Hkv // Hq], kv.v[0, h * Hkv // Hq], seen,
                     1 / math.sqrt(D))
        prefill_close(out[at, h], lse[at, h], *r, n=L)
    assert tsa.workspace_status(ws) == 0
    assert not ws[:1024].any()                   # the status word and the places are free
    # the same again, a smaller call between
    tsa.window_attn_prefill(q[:1], kv, i32([L]), 0, 300, workspace=ws)
    again, _ = tsa.window_attn_prefill(q, kv, i32([L]), 0, None, workspace=ws)
    assert torch.equal(out, again) and not ws[:1024].any()


def test_prefill_long_sums_of_tokens_before_the_first_row(tsa):
    """More tokens than positions beside a long sequence: rows that see nothing
    through every addition, and a value of infinity behind all of them."""
    g = gen(4)
    Hq, cap = 16, 24000
    kv, rows = bf16_cache(tsa, g, 2, Hq, cap, 16)
    lens, news = [23984, 30], [700, 700]
    kv.v[kv.page_table[0, cap // 16 - 1].long()] = math.inf
    q = randn(g, 1400, Hq, D).bfloat16()
    lse = torch.empty((1400, Hq), device=DEV)
    out, _ = tsa.window_attn_prefill(q, kv, i32(lens), 0, None, lse_out=lse)
    for b, (L, n) in enumerate(zip(lens, news)):
        at = torch.tensor([0, 1, 669, 670, 699], device=DEV)
        for h in (0, 7, 15):
            r = attend64(q[700 * b + at, h], rows(kv.k, b, h)[:L], rows(kv.v, b, h)[:L],
                         seen_of(L - n + at, L, 0, L), 1 / math.sqrt(D))
            prefill_close(out[700 * b + at, h], lse[700 * b + at, h], *r, n=L)
