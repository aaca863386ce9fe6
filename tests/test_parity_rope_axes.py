"""Rotary positions with several axes against 64-bit forms of the definition: applied to
q and k, and on the way into the 8-bit cache."""
import math

import pytest
import torch

from test_parity_cache_ops import (D, DEV, PlainCache, gen, i32, make_cache,
                                   randn, rates, rope_close)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tsa():
    import top_retrieval_sparse_gb300 as t
    t.lib()
    return t


def axis_of(sections, order):
    if order == "blocks":
        return [a for a, n in enumerate(sections) for _ in range(n)]
    out, left = [], list(sections)
    while sum(left):
        for a in range(len(left)):
            if left[a] > 0:
                out.append(a)
                left[a] -= 1
    return out


def axes_rates(rot, sections, order, own, theta, kind="none", f=1.0, orig=0):
    axis, seen = axis_of(sections, order), [0] * len(sections)
    if not own:
        return rates(rot, theta, kind, f, orig)
    per = [rates(2 * n, theta, kind, f, orig) for n in sections]
    w = []
    for a in axis:
        w.append(per[a][0][seen[a]])
        seen[a] += 1
    return torch.stack(w), per[0][1]


def turn64(x, pos, rot, layout, axis, w, amp, inverse=False):
    """Rotated rows and, per element, |a| + |b| of its pair; pos [axes, T]."""
    x = x.double()
    ang = pos.double()[torch.tensor(axis, device=DEV)].T * w * (-1 if inverse else 1)
    c, s = ang.cos()[:, None] * amp, ang.sin()[:, None] * amp
    y, mag = x.clone(), torch.zeros_like(x)
    ia = torch.arange(rot // 2, device=DEV)
    ia, ib = (ia, ia + rot // 2) if layout == "half" else (2 * ia, 2 * ia + 1)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    mag[..., ia] = mag[..., ib] = (a.abs() + b.abs()) * amp
    return y, mag


CASES = [  # T, Hq, Hkv, rot, sections, order, rates, layout, scaling, inverse
    (1, 4, 1, 128, (16, 24, 24), "blocks", "joint", "half", "none", False),
    (7, 28, 4, 128, (24, 20, 20), "turns", "joint", "interleaved", "yarn", False),
    (33, 5, 5, 64, (16, 16), "blocks", "own", "half", "none", True),
    (130, 32, 8, 96, (16, 17, 15), "turns", "own", "half", "linear", False),
    (1300, 6, 2, 128, (16, 16, 16, 16), "turns", "joint", "half", "by_parts", False),
    (2049, 3, 1, 16, (1, 7), "blocks", "joint", "interleaved", "none", False),
    (64, 2, 2, 32, (2, 3, 11), "turns", "own", "interleaved", "ntk", False),
    (50, 4, 4, 128, (64,), "blocks", "joint", "half", "none", False),
    (5000, 32, 8, 112, (1, 1, 54), "turns", "joint", "half", "none", True)]


@pytest.mark.parametrize("case", CASES, ids=range(len(CASES)))
def test_rope_axes(tsa, case):
    T, Hq, Hkv, rot, sections, order, rt, layout, kind, inverse = case
    g = gen(T + rot)
    q, k = randn(g, T, Hq, D).bfloat16(), randn(g, T, Hkv, D).bfloat16()
    top, f, orig, theta = 1 << 18, 4.0, 8192, 5e5
    wide = torch.randint(0, top, (len(sections), T + 3), generator=g, device=DEV).int()
    pos = wide[:, :T]                                     # rows with a stride
    table = tsa.RopeTable(rot, top, theta, layout, kind, f, orig, sections=sections, order=order,
                          rates=rt)
    qo, ko = tsa.rope(q, pos, table, k=k, inverse=inverse)
    w, amp = axes_rates(rot, sections, order, rt == "own", theta, kind, f, orig)
    axis = axis_of(sections, order)
    for x, y in ((q, qo), (k, ko)):
        ref, mag = turn64(x, pos, rot, layout, axis, w, amp, inverse)
        rope_close(y, ref, mag)
        assert torch.equal(y[..., rot:], x[..., rot:])


def test_equal_positions_and_one_axis_are_the_plain_rotation(tsa):
    """Bit for bit, whatever the order; a table of several axes takes [T] too."""
    g = gen(3)
    T = 300
    q = randn(g, T, 6, D).bfloat16()
    pos = torch.randint(0, 4096, (T,), generator=g, device=DEV).int()
    plain, _ = tsa.rope(q, pos, tsa.RopeTable(128, 4096, 1e4))
    for sections, order in (((16, 24, 24), "blocks"), ((24, 20, 20), "turns"), ((64,), "turns")):
        table = tsa.RopeTable(128, 4096, 1e4, sections=sections, order=order)
        same = pos.expand(len(sections), T).contiguous()
        assert torch.equal(tsa.rope(q, same, table)[0], plain)
        assert torch.equal(tsa.rope(q, pos, table)[0], plain)
        if len(sections) > 1:                             # a stride of 0
            assert torch.equal(tsa.rope(q, pos[None].expand(len(sections), T), table)[0], plain)


def test_positions_out_of_range_blank_their_axis(tsa):
    """In place on a slice of a fused projection; other pairs and rows keep their values."""
    g = gen(5)
    T, sections = 9, (10, 30, 24)
    qkv = randn(g, T, 12, D).bfloat16()
    was = qkv.clone()
    pos = torch.randint(0, 1000, (3, T), generator=g, device=DEV).int()
    good = tsa.rope(was[:, :8], pos, tsa.RopeTable(128, 1000, 1e4, sections=sections),
                    k=was[:, 8:10])
    pos[1, 4], pos[2, 6], pos[0, 7] = 1000, -1, 1 << 30
    table = tsa.RopeTable(128, 1000, 1e4, sections=sections)
    tsa.rope(qkv[:, :8], pos, table, k=qkv[:, 8:10], q_out=qkv[:, :8], k_out=qkv[:, 8:10])
    want = torch.cat([*good, was[:, 10:]], dim=1)
    for t, a, z in ((4, 10, 40), (6, 40, 64), (7, 0, 10)):
        for lo in (0, 64):
            want[t, :10, lo + a: lo + z] = math.nan
    assert torch.equal(qkv.isnan(), want.isnan())
    assert torch.equal(qkv.nan_to_num(), want.nan_to_num())


def test_inverse_is_the_gradient_and_turns_back(tsa):
    """<R x, y> = <x, R^-1 y> in 64 bits on values that bf16 holds, by differences of the
    64-bit form; and back again within two roundings."""
    g = gen(8)
    T, sections = 40, (16, 24, 24)
    x, y = randn(g, T, 2, D).bfloat16(), randn(g, T, 2, D).bfloat16()
    pos = torch.randint(0, 4096, (3, T), generator=g, device=DEV).int()
    table = tsa.RopeTable(128, 4096, 1e4, sections=sections, order="turns")
    w, amp = axes_rates(128, sections, "turns", False, 1e4)
    axis = axis_of(sections, "turns")
    grad = torch.zeros_like(x, dtype=torch.float64)
    for j in range(0, D, 7):                              # d <R x, y> / d x_j, R being linear
        e = torch.zeros_like(grad)
        e[..., j] = 1
        up, down = (turn64(x.double() + s * e, pos, 128, "half", axis, w, amp)[0] for s in (1, -1))
        grad[..., j] = ((up - down) * y.double()).sum(-1) / 2
    back, _ = tsa.rope(y, pos, table, inverse=True)
    ref, mag = turn64(y, pos, 128, "half", axis, w, amp, inverse=True)
    rope_close(back, ref, mag)
    cols = torch.arange(0, D, 7, device=DEV)
    assert torch.allclose(grad[..., cols], ref[..., cols], rtol=0, atol=1e-12)
    there, _ = tsa.rope(x, pos, table)
    again, _ = tsa.rope(there, pos, table, inverse=True)
    # half a step of bf16 in there (turned back: of |a| + |b|), half a step at the end
    _, mag = turn64(x, pos, 128, "half", axis, w, amp)
    assert ((again.double() - x.double()).abs() <= mag * (2.0 ** -7 + 2.0 ** -19) * 1.01).all()


@pytest.mark.parametrize("fmt,block,page,layout,order", [
    ("int8", 16, 16, "half", "blocks"), ("e4m3", 64, 64, "interleaved", "turns"),
    ("int8", 128, 0, "half", "turns"), ("e4m3", 32, 256, "interleaved", "blocks"),
    ("int8", 64, 128, "interleaved", "turns"), ("e4m3", 128, 128, "half", "blocks")])
def test_append_rotates_keys_by_axes(tsa, fmt, block, page, layout, order):
    """Codes and scales are those of keys turned in 64 bits, but where a turned key lies
    within 2^-20 of the border of a code or a scale."""
    g = gen(block + page)
    B, Hkv, cap, sections = 3, 2, 512, (20, 24, 20)
    cache = make_cache(tsa, g, B, Hkv, cap, block, fmt, page)
    table = tsa.RopeTable(128, 1 << 16, 1e4, layout, sections=sections, order=order)
    w, amp = axes_rates(128, sections, order, False, 1e4)
    axis, lens = axis_of(sections, order), [0, 0, 0]
    plain = PlainCache(B, Hkv, cap, block, fmt)
    for news in ([200, 77, 0], [1, 1, 1], [130, 300, 33]):
        T, cu = sum(news), [0, news[0], news[0] + news[1], sum(news)]
        k, v = randn(g, T, Hkv, D).bfloat16(), randn(g, T, Hkv, D).bfloat16()
        pos = torch.randint(0, 1 << 16, (3, T), generator=g, device=DEV).int()
        lens = [a + n for a, n in zip(lens, news)]
        tsa.kv8_append(cache, k, v, i32(lens), i32(cu), max(news), rope=table, positions=pos)
        turned, _ = turn64(k, pos, 128, layout, axis, w, amp)
        for b in range(B):
            part = slice(cu[b], cu[b + 1])
            if news[b]:
                plain.append(b, lens[b] - news[b], torch.stack([turned[part], v[part].double()]))
    cu = [0, *[sum(lens[:i + 1]) for i in range(B)]]
    got_k, got_v = tsa.kv8_read(cache, i32(lens), cu=i32(cu), n=max(lens), T=sum(lens))
    for b, L in enumerate(lens):
        for which, got in ((0, got_k), (1, got_v)):
            ref = plain.val[which, b, :, :L].transpose(0, 1)
            diff = (got[cu[b]:cu[b + 1]].double() - ref).abs()
            step = plain.scale[which, b].repeat_interleave(block, dim=1)[:, :L].T[..., None]
            unit = step
            if fmt == "e4m3":
                unit = torch.exp2(torch.floor(torch.log2((ref / step).abs().clamp(min=2.0 ** -6)))
                                  - 3) * step
            if which == 1:
                assert (diff == 0).all()
            else:
                # a rounding the other way moves a code by one (two after a second
                # rounding of older rows); such borders are rare
                assert (diff <= 2 * unit * 1.001).all() and (diff > 0).double().mean() < 1e-3
    if cache.status is not None:
        assert tsa.workspace_status(cache.status) == 0


def test_append_flags_positions_out_of_range(tsa):
    g = gen(2)
    cache = make_cache(tsa, g, 1, 1, 128, 16, "int8", 16)
    table = tsa.RopeTable(128, 100, 1e4, sections=(32, 32))
    k = randn(g, 5, 1, D).bfloat16()
    pos = i32([[0, 1, 2, 3, 4], [0, 1, 100, 3, 4]])
    tsa.kv8_append(cache, k, k, i32([5]), rope=table, positions=pos)
    assert int(tsa.lib().tsa_workspace_status(cache.status.data_ptr(), 1, None)) != 0
    got, _ = tsa.kv8_read(cache, i32([5]), 5)
    assert (got[2, 0, 32:64] == 0).all() and (got[2, 0, 96:] == 0).all()   # NaN is code 0
    assert (got[2, 0, :32] != 0).any()
