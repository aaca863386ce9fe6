"""The cache-side operators against plain 64-bit forms of their definitions:
rotary positions, the 8-bit cache (written and read), attention over it, and
attention with a sliding window and sinks (one token and many).

Half a step of rounding, relative to the value: bf16 2^-8, e4m3 2^-4, fp32 2^-24.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
D = 128
DEV = "cuda"
HALF = 2.0 ** -8   # bf16


@pytest.fixture(scope="module")
def tsa():
    import top_retrieval_sparse_gb300 as t
    t.lib()
    return t


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------- rope
def rates(rot, theta, kind, f, orig):
    """(w_i, amplitude) by the definition, one pair at a time."""
    base = theta * f ** (rot / (rot - 2)) if kind == "ntk" else theta
    out, amp = [], 1.0
    for i in range(rot // 2):
        w = base ** (-2 * i / rot)
        if kind == "linear":
            w /= f
        if kind == "by_parts":
            turns = orig * w / (2 * math.pi)
            if turns < 1:
                w /= f
            elif turns <= 4:
                t = (turns - 1) / 3
                w = (1 - t) * w / f + t * w
        if kind == "yarn":
            at = [rot * math.log(orig / (2 * math.pi * b)) / (2 * math.log(theta))
                  for b in (32, 1)]
            lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
            r = min(max((i - lo) / max(hi - lo, 0.001), 0), 1)
            w = r * w / f + (1 - r) * w
            amp = 0.1 * math.log(f) + 1
        out.append(w)
    return torch.tensor(out, dtype=torch.float64, device=DEV), amp


def turn64(x, pos, rot, layout, w, amp, inverse=False):
    """Rotated rows and, per element, |a| + |b| of its pair."""
    x = x.double()
    ang = pos.double()[:, None] * w * (-1 if inverse else 1)
    c, s = ang.cos()[:, None] * amp, ang.sin()[:, None] * amp
    y, mag = x.clone(), torch.zeros_like(x)
    ia = torch.arange(rot // 2, device=DEV)
    ia, ib = (ia, ia + rot // 2) if layout == "half" else (2 * ia, 2 * ia + 1)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    mag[..., ia] = mag[..., ib] = (a.abs() + b.abs()) * amp
    return y, mag


def rope_close(got, ref, mag):
    # cos and sin are sums of two products of values rounded to 32 bits (2^-22
    # in all), the turn adds three roundings: under 2^-20 of |a| + |b|; then
    # half a step of bf16
    tol = ref.abs() * HALF + mag * 2.0 ** -20
    bad = (got.double() - ref).abs() > tol
    assert not bad.any(), float(((got.double() - ref).abs() - tol).max())


@pytest.mark.parametrize("T,Hq,Hkv,rot,layout,kind,theta,max_pos,inverse", [
    (1, 4, 1, 128, "half", "none", 1e4, 1 << 20, False),
    (7, 28, 4, 128, "interleaved", "yarn", 1e6, 131072, False),
    (33, 32, 8, 64, "half", "by_parts", 5e5, 131072, False),
    (130, 5, 5, 96, "half", "ntk", 1e4, 32768, True),
    (64, 3, 1, 16, "interleaved", "linear", 1e4, 4096, True),
    (2000, 32, 8, 112, "half", "yarn", 1e4, 1 << 22, False),
    (4097, 6, 2, 48, "interleaved", "by_parts", 5e5, 1 << 17, False)])
def test_rope(tsa, T, Hq, Hkv, rot, layout, kind, theta, max_pos, inverse):
    g = gen(T)
    q, k = randn(g, T, Hq, D).bfloat16(), randn(g, T, Hkv, D).bfloat16()
    pos = torch.randint(0, max_pos, (T,), generator=g, device=DEV).int()
    pos[0], pos[-1] = 0, max_pos - 1
    f, orig = 8.0, 4096
    table = tsa.RopeTable(rot, max_pos, theta, layout, kind, f, orig)
    qo, ko = tsa.rope(q, pos, table, k=k, inverse=inverse)
    w, amp = rates(rot, theta, kind, f, orig)
    for x, y in ((q, qo), (k, ko)):
        ref, mag = turn64(x, pos, rot, layout, w, amp, inverse)
        rope_close(y, ref, mag)
        assert torch.equal(y[..., rot:], x[..., rot:])
    q1, none = tsa.rope(q, pos, table, inverse=inverse)  # without keys: the same
    assert none is None and torch.equal(q1, qo)


def test_rope_in_place_on_a_fused_projection_and_positions_out_of_range(tsa):
    g = gen(3)
    T, Hq, Hkv = 50, 12, 4
    qkv = randn(g, T, (Hq + 2 * Hkv) * D).bfloat16()
    was = qkv.clone()
    heads = qkv.view(T, Hq + 2 * Hkv, D)
    q, k = heads[:, :Hq], heads[:, Hq:Hq + Hkv]
    pos = torch.arange(T, device=DEV).int()
    pos[7], pos[9] = -1, 4096
    table = tsa.RopeTable(64, 4096, 1e4)
    qo, ko = tsa.rope(was.view(T, -1, D)[:, :Hq], pos, table, k=was.view(T, -1, D)[:, Hq:Hq + Hkv])
    tsa.rope(q, pos, table, k=k, q_out=q, k_out=k)
    assert torch.equal(q.view(torch.int16), qo.view(torch.int16))
    assert torch.equal(k.view(torch.int16), ko.view(torch.int16))
    assert torch.equal(heads[:, Hq + Hkv:], was.view(T, -1, D)[:, Hq + Hkv:])
    nan = torch.isnan(qo)
    assert nan[[7, 9]][..., :64].all() and not nan[[7, 9]][..., 64:].any()
    nan[[7, 9]] = False
    assert not nan.any()


def test_rope_inverse_is_the_gradient(tsa):
    """<R x, y> = <x, R^T y>, and against differences: R is linear, so the
    difference quotient along any direction is R of it."""
    g = gen(4)
    T, H = 40, 3
    x, y = randn(g, T, H, D).bfloat16(), randn(g, T, H, D).bfloat16()
    pos = torch.randint(0, 9000, (T,), generator=g, device=DEV).int()
    for layout in ("half", "interleaved"):
        t = tsa.RopeTable(96, 9000, 1e4, layout, "yarn", 4.0, 2048)
        rx, _ = tsa.rope(x, pos, t)
        ry, _ = tsa.rope(y, pos, t, inverse=True)
        a = (rx.double() * y.double()).sum(-1)
        b = (x.double() * ry.double()).sum(-1)
        # each product's bf16 factor is within HALF of exact
        tol = HALF * 1.1 * ((rx.double() * y.double()).abs().sum(-1) +
                            (x.double() * ry.double()).abs().sum(-1))
        assert ((a - b).abs() <= tol).all()


# -------------------------------------------------------------- 8-bit cache
TOP = {"int8": 127.0, "e4m3": 448.0}


def grid8(y, fmt):
    """Nearest value of the 8-bit grid (ties to even)."""
    if fmt == "int8":
        return torch.round(y).clamp(-127, 127)
    unit = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(y / unit) * unit).clamp(-448, 448)


def scale64(amax, fmt):
    e = torch.ceil(torch.log2(amax.clamp(min=1e-300) / TOP[fmt]) - 1e-10).clamp(min=-60)
    return torch.exp2(e)


def values(cache):
    """Every stored value of a cache, fp64, and the codes."""
    out = []
    for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        x = c.double() - 128 if cache.fmt == "int8" else c.view(torch.float8_e4m3fn).double()
        out.append(x * s.double().repeat_interleave(cache.block, dim=2)[..., None])
    return out


def place(cache, b, pos):
    """(page or sequence, row) of position pos of sequence b."""
    if cache.page_table is None:
        return b, pos
    ps = cache.k.shape[2]
    return int(cache.page_table[b, pos // ps]), pos % ps


def make_cache(tsa, g, B, Hkv, l_cap, block, fmt, page, spare=2):
    if page == 0:
        return tsa.KV8.contiguous(B, Hkv, l_cap, block, fmt)
    per = l_cap // page
    pt = torch.randperm(B * per + spare, generator=g, device=DEV)[:B * per].view(B, per).int()
    return tsa.KV8.paged(B * per + spare, Hkv, page, pt.contiguous(), block, fmt)


class PlainCache:
    """Positions' values by the definition: one block at a time, 64 bits."""

    def __init__(self, B, Hkv, l_cap, block, fmt):
        self.val = torch.zeros((2, B, Hkv, l_cap, D), dtype=torch.float64, device=DEV)
        self.scale = torch.zeros((2, B, Hkv, l_cap // block), dtype=torch.float64, device=DEV)
        self.block, self.fmt = block, fmt

    def append(self, b, start, x):
        """x [2, n, Hkv, D] at positions start.. of sequence b."""
        n, blk = x.shape[1], self.block
        for j in range(start // blk, (start + n - 1) // blk + 1):
            lo, hi = max(start, j * blk), min(start + n, (j + 1) * blk)
            part = x[:, lo - start:hi - start].transpose(1, 2)        # [2, H, m, D]
            fin = torch.where(part.isfinite(), part.abs(), 0.0)
            s = scale64(fin.amax(dim=(2, 3)), self.fmt)
            if lo > j * blk:
                s = torch.maximum(s, self.scale[:, b, :, j])
                old = self.val[:, b, :, j * blk:lo]
                self.val[:, b, :, j * blk:lo] = grid8(old / s[..., None, None], self.fmt) * \
                    s[..., None, None]
            self.scale[:, b, :, j] = s
            self.val[:, b, :, lo:hi] = grid8(part / s[..., None, None], self.fmt) * \
                s[..., None, None]


def check_cache(cache, plain, lens):
    got = values(cache)
    for b, L in enumerate(lens):
        if L == 0:
            continue
        at = [place(cache, b, p) for p in range(L)]
        pi, ri = torch.tensor([x[0] for x in at]), torch.tensor([x[1] for x in at])
        for w in range(2):
            assert torch.equal(got[w][pi, :, ri].transpose(0, 1), plain.val[w, b, :, :L]), (b, w)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("Hkv,block,page", [(2, 16, 0), (1, 64, 0), (3, 128, 0), (2, 16, 16),
                                            (2, 32, 64), (1, 128, 256)])
def test_append_and_read_are_exact(tsa, fmt, Hkv, block, page):
    """Ragged appends of several calls, starting inside blocks, scales that
    grow by a little and by a lot: every stored value is the definition's."""
    g = gen(block + page)
    B, cap = 4, 768
    cache = make_cache(tsa, g, B, Hkv, cap, block, fmt, page)
    cache.k.fill_(77), cache.v.fill_(33)   # stale codes
    cache.k_scale.fill_(2.0 ** 40), cache.v_scale.fill_(float("nan"))
    plain = PlainCache(B, Hkv, cap, block, fmt)
    lens = [0] * B
    for step, news in enumerate([[5, 0, 130, 257], [1, 1, 1, 1], [0, 17, 64, 3], [1, 1, 1, 1],
                                 [300, 1, 0, 129]]):
        T = sum(news)
        x = randn(g, 2, T, Hkv, D).bfloat16() * float([1, 4, 0.25, 300, 1e-3][step])
        x[:, ::3] *= 0.01
        cu = [0]
        for n in news:
            cu.append(cu[-1] + n)
        lens = [a + n for a, n in zip(lens, news)]
        tsa.kv8_append(cache, x[0], x[1], i32(lens), cu_new=i32(cu), max_new=max(news))
        for b, n in enumerate(news):
            if n:
                plain.append(b, lens[b] - n, x[:, cu[b]:cu[b + 1]].double())
        check_cache(cache, plain, lens)
    # every row back: exact in bf16
    k, v = tsa.kv8_read(cache, i32(lens), n=max(lens), cu=i32([0, *torch.tensor(lens).cumsum(0)]),
                        T=sum(lens))
    at = 0
    for b, L in enumerate(lens):
        for w, o in enumerate((k, v)):
            assert torch.equal(o[at:at + L].double(), plain.val[w, b, :, :L].transpose(0, 1))
        at += L
    assert tsa.workspace_status(cache.status) == 0


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_append_leaves_everything_else_alone(tsa, fmt):
    g = gen(9)
    B, Hkv, cap, blk = 3, 2, 256, 32
    cache = make_cache(tsa, g, B, Hkv, cap, blk, fmt, 64)
    cache.k.copy_(torch.randint(1, 255, cache.k.shape, generator=g, device=DEV))
    cache.v.copy_(cache.k.flip(0))
    cache.k_scale.fill_(1.0), cache.v_scale.fill_(2.0)
    was = [t.clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    lens, news = [70, 33, 256], [3, 0, 10]
    x = randn(g, 2, 20, Hkv, D).bfloat16()   # rows past the last sequence's too
    tsa.kv8_append(cache, x[0], x[1], i32(lens), cu_new=i32([0, 3, 3, 13]), max_new=10)
    touched = torch.zeros(cache.k.shape[:3], dtype=torch.bool, device=DEV)
    tblock = torch.zeros(cache.k_scale.shape, dtype=torch.bool, device=DEV)
    for b, (L, n) in enumerate(zip(lens, news)):
        for p in range(L - n, L):
            pg, r = place(cache, b, p)
            touched[pg, :, r] = True
            tblock[pg, :, r // blk] = True
    # the scales were far above the new rows': nothing grows, old rows stay
    for now, old, m in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), was,
                           (touched, touched, tblock, tblock)):
        assert torch.equal(now[~m], old[~m])


@pytest.mark.parametrize("fmt,rot,layout,given", [("int8", 128, "half", False),
                                                  ("e4m3", 96, "interleaved", True),
                                                  ("int8", 32, "half", True)])
def test_append_rotates_keys(tsa, fmt, rot, layout, given):
    g = gen(rot)
    B, Hkv, cap, blk = 3, 4, 4096, 64
    cache = make_cache(tsa, g, B, Hkv, cap, blk, fmt, 128)
    lens, news = [1000, 4096, 333], [1000, 700, 1]
    cu = [0, 1000, 1700, 1701]
    fused = randn(g, cu[-1], 3 * Hkv, D).bfloat16()     # strided rows
    k, v = fused[:, Hkv:2 * Hkv], fused[:, 2 * Hkv:]
    pos = torch.cat([torch.arange(L - n, L) for L, n in zip(lens, news)]).to(DEV).int()
    if given:
        pos = (pos * 31 + 5) % 8000
    table = tsa.RopeTable(rot, 8000, 1e4, layout, "yarn", 4.0, 2048)
    tsa.kv8_append(cache, k, v, i32(lens), cu_new=i32(cu), max_new=1000, rope=table,
                   positions=pos if given else None)
    w, amp = rates(rot, 1e4, "yarn", 4.0, 2048)
    ref, mag = turn64(k, pos, rot, layout, w, amp)
    for b, (L, n) in enumerate(zip(lens, news)):
        at = [place(cache, b, p) for p in range(L - n, L)]
        pi, ri = torch.tensor([x[0] for x in at]), torch.tensor([x[1] for x in at])
        for codes, scale, r, m in ((cache.k, cache.k_scale, ref, mag),
                                   (cache.v, cache.v_scale, v.double(), None)):
            r = r[cu[b]:cu[b + 1]]
            s = scale.double()[pi, :, ri // blk][..., None]
            x = codes[pi, :, ri]
            x = (x.double() - 128 if fmt == "int8" else x.view(torch.float8_e4m3fn).double()) * s
            # half a step of the grid, and the rotation's own error
            step = s * 0.5 if fmt == "int8" else torch.maximum(r.abs() * 2.0 ** -4, s * 2.0 ** -10)
            tol = step * (1 + 1e-6) + (m[cu[b]:cu[b + 1]] * 2.0 ** -20 if m is not None else 0)
            assert ((x - r).abs() <= tol).all()
            # the scale is the smallest that holds the block's largest value
            start = L - n
            for j in range(start // blk, (L - 1) // blk + 1):
                lo, hi = max(start, j * blk), min(L, (j + 1) * blk)
                amax = r[lo - start:hi - start].abs().amax(dim=(0, 2))
                sc = s[lo - start, :, 0]
                if lo == j * blk:
                    assert (amax <= TOP[fmt] * sc * (1 + 1e-5)).all()
                    assert (amax > TOP[fmt] * sc / 2 * (1 - 1e-5)).all()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_append_of_zeros_infinities_and_nan(tsa, fmt):
    cache = tsa.KV8.contiguous(1, 1, 64, 32, fmt)
    x = torch.zeros((64, 1, D), dtype=torch.bfloat16, device=DEV)
    x[32, 0, 0], x[33, 0, 1], x[34, 0, 2], x[35, 0, 3] = 3.0, math.inf, -math.inf, math.nan
    tsa.kv8_append(cache, x, x, i32([64]))
    k, v = tsa.kv8_read(cache, i32([64]), n=64)
    assert torch.equal(k[:32], x[:32]) and (cache.k_scale[0, 0, 0] == 2.0 ** -60).all()
    s = float(cache.k_scale[0, 0, 1])
    assert s == 2.0 ** math.ceil(math.log2(3.0 / TOP[fmt]))
    assert float(k[32, 0, 0]) == 3.0
    assert float(k[33, 0, 1]) == TOP[fmt] * s and float(k[34, 0, 2]) == -TOP[fmt] * s
    assert float(k[35, 0, 3]) == 0.0 if fmt == "int8" else math.isnan(float(k[35, 0, 3]))


def test_bad_lengths_and_pages_are_flagged(tsa):
    pt = i32([[0, 1], [2, 9], [3, -1]])
    cache = tsa.KV8.paged(4, 1, 32, pt, 16)
    x = torch.ones((3, 1, D), dtype=torch.bfloat16, device=DEV)
    for lens in ([65, 1, 1], [0, 1, 1], [33, 33, 1], [33, 1, 33]):
        cache.k.zero_()
        tsa.kv8_append(cache, x, x, i32(lens))
        assert tsa.workspace_status(cache.status) == -5
        k, _ = tsa.kv8_read(cache, i32(lens), n=1)
        bad = torch.isnan(k.float()).view(3, -1).all(1).tolist()
        assert bad == [L > 64 or (b > 0 and L > 32) for b, L in enumerate(lens)]
        assert tsa.workspace_status(cache.status) == (-5 if any(bad) else 0)
    tsa.kv8_append(cache, x, x, i32([1, 1, 1]))
    assert tsa.workspace_status(cache.status) == 0
    # a sequence with more tokens than max_new is not written
    cache.k.zero_()
    tsa.kv8_append(cache, x, x, i32([5, 5, 5]), cu_new=i32([0, 2, 3, 3]), max_new=1)
    assert tsa.workspace_status(cache.status) == -5
    assert not cache.k[0].any() and cache.k[2].any()


def test_read_before_the_first_position_gives_zeros_and_keeps_the_rest(tsa):
    cache = tsa.KV8.contiguous(2, 3, 64, 16)
    x = torch.full((4, 3, D), 2.0, dtype=torch.bfloat16, device=DEV)
    tsa.kv8_append(cache, x, x, i32([2, 2]))
    out = torch.full((12, 3, D), 9.0, dtype=torch.bfloat16, device=DEV)
    k, v = tsa.kv8_read(cache, i32([2, 2]), n=5, cu=i32([0, 5, 7]), k_out=out, v_out=out.clone())
    for o in (k, v):
        assert (o[:3] == 0).all() and (o[3:7] == 2).all() and (o[7:] == 9).all()


# ---------------------------------------------------------------- attention
def attend64(q, k, v, seen, scale):
    """q [R, D], k, v [W, D], seen [R, W]: (out, lse, sum of p|v|, the largest
    sum over j of |q_j k_j| * scale of a visible row)."""
    q, k, v = q.double(), k.double(), v.double()
    k, v = (torch.where(seen.any(0)[:, None], x, 0.0) for x in (k, v))
    z = torch.where(seen, q @ k.T * scale, -math.inf)
    lse = torch.logsumexp(z, dim=1)
    p = torch.where(seen, torch.exp(z - torch.where(lse.isinf(), 0.0, lse)[:, None]), 0.0)
    zabs = torch.where(seen, q.abs() @ k.abs().T * abs(scale), 0.0).amax(dim=1) if k.shape[0] else \
        torch.zeros_like(lse)
    return p @ v, lse, p @ v.abs(), zabs


def seen_of(p, W, ni, nr):
    j = torch.arange(W, device=DEV)
    p = torch.as_tensor(p, device=DEV)[:, None]
    return (j <= p) & ((j < ni) | (j > p - nr))


def small_weights(q, k, v, seen, scale, steps):
    """What weights too small for fp16 can change: the 8-bit path's weights
    carry their row's value scale s_i, and are rounded to at least 2^-25 where
    the largest of them is at least 2^7 (each warp's own largest, at most the
    row's).  So out is off by at most 2^-32 max_j(p_j s_j) sum_i |v_i| / s_i."""
    z = torch.where(seen, q.double() @ k.double().T * scale, -math.inf)
    p = torch.softmax(z, dim=1).nan_to_num(0.0)
    return 2.0 ** -32 * (p * steps).amax(dim=1, keepdim=True) * \
        (seen.double() @ (v.double().abs() / steps[:, None]))


def decode_close(out, lse, ref, rlse, pv, zabs, n, extra=0.0):
    # Logit: 128 exact products added in 32 bits with truncating adds: within
    # 2^-20 of their magnitudes' sum (16 steps of 2^-23, and a factor 2 on top).
    # exp: 2^-21 with its argument's rounding (2^-24 of |z| log2 e, covered by
    # the zabs term).  Weights in two bf16 parts: 2^-17.  Sum over n rows in 32
    # bits, 16 a step, truncating: n/16 * 2^-23 at most.  Twice, for the
    # numerator and the denominator.
    eps = 2 * (zabs * 2.0 ** -19 + 2.0 ** -17 + 2.0 ** -20 + n * 2.0 ** -27)
    bad = (out.double() - ref).abs() > pv * eps[:, None] + extra + 1e-30
    assert not bad.any(), float(((out.double() - ref).abs() / pv.clamp(min=1e-30)).max())
    empty = rlse.isinf()
    assert torch.equal(lse.isinf(), empty) and (out[empty] == 0).all()
    assert ((lse.double() - rlse).abs()[~empty] <= (eps + rlse.abs() * 2.0 ** -22)[~empty]).all()


def bf16_cache(tsa, g, B, Hkv, cap, page, spare=2):
    """A bf16 cache and, per (sequence, head), a function to its rows."""
    if page == 0:
        k, v = randn(g, B, Hkv, cap, D).bfloat16(), randn(g, B, Hkv, cap, D).bfloat16()
        return tsa.kv_contiguous(k, v), lambda t, b, h: t[b, h]
    per = cap // page
    pt = torch.randperm(B * per + spare, generator=g, device=DEV)[:B * per].view(B, per).int()
    k = randn(g, B * per + spare, Hkv, page, D).bfloat16()
    v = randn(g, B * per + spare, Hkv, page, D).bfloat16()
    return tsa.kv_paged(k, v, pt.contiguous()), \
        lambda t, b, h: t[pt[b].long(), h].reshape(cap, D)


def quant_cache(tsa, g, B, Hkv, cap, block, fmt, page):
    cache = make_cache(tsa, g, B, Hkv, cap, block, fmt, page)
    amp = torch.exp(randn(g, B, cap // 16, 1, 1, 1)).expand(-1, -1, 16, 1, 1).reshape(B, cap, 1, 1)
    x = (randn(g, B, cap, Hkv, D) * amp).bfloat16().view(B * cap, Hkv, D)
    y = (randn(g, B, cap, Hkv, D) * amp.flip(1)).bfloat16().view(B * cap, Hkv, D)
    tsa.kv8_append(cache, x * 0.3, y, i32([cap] * B))
    val = values(cache)
    if page == 0:
        return cache, lambda w, b, h: val[w][b, h]
    return cache, lambda w, b, h: val[w][cache.page_table[b].long(), h].reshape(cap, D)


DECODE_CASES = [  # B, Hq, Hkv, cap, page, lens, n_init, n_recent
    (1, 4, 1, 64, 0, [1], 0, None), (1, 8, 1, 64, 16, [17], 0, None),
    (3, 6, 2, 640, 0, [640, 1, 0], 0, None), (2, 5, 5, 1024, 64, [1000, 999], 4, 100),
    (4, 28, 4, 4096, 16, [4096, 33, 2049, 130], 0, None),
    (2, 16, 2, 4096, 256, [4095, 3000], 130, 513), (2, 3, 1, 512, 32, [511, 300], 0, 1),
    (2, 14, 2, 512, 0, [512, 7], 5, 0), (2, 2, 2, 512, 0, [512, 7], 0, 0),
    (3, 32, 8, 2048, 128, [2048, 64, 65], 1, 63), (1, 32, 8, 70000, 0, [69999], 0, None),
    (40, 7, 1, 1024, 16, list(range(3, 1003, 25)), 0, None)]


@pytest.mark.parametrize("case", DECODE_CASES, ids=range(len(DECODE_CASES)))
def test_window_attn_decode(tsa, case):
    B, Hq, Hkv, cap, page, lens, ni, nr = case
    g = gen(cap + B)
    q = randn(g, B, Hq, D).bfloat16()
    kv, rows = bf16_cache(tsa, g, B, Hkv, cap, page)
    lse = torch.empty((B, Hq), device=DEV)
    ws = tsa.attn_decode_workspace(B, Hq, Hkv)
    out, _ = tsa.window_attn_decode(q, kv, i32(lens), ni, nr, lse_out=lse, workspace=ws)
    check_decode(q, lambda b, h: (rows(kv.k, b, h), rows(kv.v, b, h)), lens, Hkv, ni,
                 cap if nr is None else nr, out, lse)
    assert tsa.workspace_status(ws) == 0
    # the same call again on the same workspace, and without one: the same
    again, _ = tsa.window_attn_decode(q, kv, i32(lens), ni, nr, workspace=ws)
    assert torch.equal(out, again)
    assert torch.equal(out, tsa.window_attn_decode(q, kv, i32(lens), ni, nr)[0])


def value_steps(cache, b, h):
    """The value scale of every row of a sequence and KV head."""
    if cache.page_table is None:
        s = cache.v_scale[b, h]
    else:
        s = cache.v_scale[cache.page_table[b].long(), h].reshape(-1)
    return s.double().repeat_interleave(cache.block)


def check_decode(q, rows, lens, Hkv, ni, nr, out, lse, scale=1 / math.sqrt(D), steps=None):
    G = q.shape[1] // Hkv
    for b, L in enumerate(lens):
        seen = seen_of([L - 1], L, ni, nr)
        for h in range(Hkv):
            k, v = rows(b, h)
            at = slice(h * G, h * G + G)
            r = attend64(q[b, at], k[:L], v[:L], seen.expand(G, L), scale)
            extra = 0.0 if steps is None or L == 0 else small_weights(
                q[b, at], k[:L], v[:L], seen.expand(G, L), scale, steps(b, h)[:L])
            decode_close(out[b, at], lse[b, at], *r, n=L, extra=extra)


@pytest.mark.parametrize("fmt,block", [("int8", 16), ("int8", 128), ("e4m3", 64), ("e4m3", 32)])
@pytest.mark.parametrize("case", DECODE_CASES, ids=range(len(DECODE_CASES)))
def test_kv8_attn_decode(tsa, case, fmt, block):
    B, Hq, Hkv, cap, page, lens, ni, nr = case
    if page and block > page:
        block = page
    cap = -(-cap // 128) * 128 if page == 0 else cap
    g = gen(cap + B + block)
    q = randn(g, B, Hq, D).bfloat16()
    cache, rows = quant_cache(tsa, g, B, Hkv, cap, block, fmt, page)
    lse = torch.empty((B, Hq), device=DEV)
    ws = tsa.attn_decode_workspace(B, Hq, Hkv)
    out, _ = tsa.kv8_attn_decode(q, cache, i32(lens), ni, nr, lse_out=lse, workspace=ws)
    check_decode(q, lambda b, h: (rows(0, b, h), rows(1, b, h)), lens, Hkv, ni,
                 cap if nr is None else nr, out, lse,
                 steps=lambda b, h: value_steps(cache, b, h))
    assert tsa.workspace_status(ws) == 0
    again, _ = tsa.kv8_attn_decode(q, cache, i32(lens), ni, nr, workspace=ws)
    assert torch.equal(out, again)


def test_decode_of_the_largest_batches(tsa):
    """4096 sequences over one page each (empty ones among them), 1024 KV heads."""
    g = gen(50)
    B, ps = 4096, 16
    pt = torch.randperm(B, generator=g, device=DEV).view(B, 1).int()
    lens = torch.randint(0, ps + 1, (B,), generator=g, device=DEV).int()
    k, v = randn(g, B, 2, ps, D).bfloat16(), randn(g, B, 2, ps, D).bfloat16()
    cache = tsa.KV8.paged(B, 2, ps, pt.contiguous())
    x = k[pt[:, 0].long()].transpose(1, 2), v[pt[:, 0].long()].transpose(1, 2)
    tsa.kv8_append(cache, *(t.reshape(-1, 2, D) for t in x), i32([ps] * B))
    val = values(cache)
    q = randn(g, B, 8, D).bfloat16()
    for call, kk, vv in ((tsa.window_attn_decode, k, v), (tsa.kv8_attn_decode, *val)):
        kv = tsa.kv_paged(k, v, pt) if kk is k else cache
        lse = torch.empty((B, 8), device=DEV)
        out, _ = call(q, kv, lens, 0, None, lse_out=lse)
        kk, vv = (t[pt[:, 0].long()].double() for t in (kk, vv))       # [B, 2, ps, D]
        z = torch.einsum("bgid,bgjd->bgij", q.double().view(B, 2, 4, D), kk) / math.sqrt(D)
        on = torch.arange(ps, device=DEV) < lens[:, None, None, None]
        z = z.masked_fill(~on, -math.inf)
        p = torch.softmax(z, -1).nan_to_num(0.0)
        ref = (p @ vv).view(B, 8, D)
        # logits of order 5, 16 rows: 32-bit arithmetic is within 1e-5 of the values
        assert ((out - ref).abs() <= 1e-5 * vv.abs().max()).all()
        full = lens > 0
        want = torch.logsumexp(z, -1).view(B, 8)
        assert torch.equal(lse.isinf().all(1), ~full)
        assert ((lse - want).abs()[full] <= 1e-4).all()
    B, H = 1, 1024
    kv, rows = bf16_cache(tsa, g, B, H, 48, 0)
    q = randn(g, B, H, D).bfloat16()
    lse = torch.empty((B, H), device=DEV)
    out, _ = tsa.window_attn_decode(q, kv, i32([37]), 3, 20, lse_out=lse)
    check_decode(q, lambda b, h: (rows(kv.k, b, h), rows(kv.v, b, h)), [37], H, 3, 20, out, lse)


def test_two_streams_at_once(tsa):
    """Calls on two streams, a workspace each, give what each gives alone."""
    g = gen(51)
    kv, _ = bf16_cache(tsa, g, 4, 4, 8192, 16)
    cache, _ = quant_cache(tsa, g, 4, 4, 8192, 16, "e4m3", 16)
    q, qp = randn(g, 4, 28, D).bfloat16(), randn(g, 800, 28, D).bfloat16()
    lens = i32([8192, 5000, 77, 2500])
    want = [tsa.kv8_attn_decode(q, cache, lens)[0],
            tsa.window_attn_prefill(qp, kv, lens, 4, 1000)[0]]
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    got = [[], []]
    for _ in range(5):
        got[0].append(tsa.kv8_attn_decode(q, cache, lens, stream=a)[0])
        got[1].append(tsa.window_attn_prefill(qp, kv, lens, 4, 1000, stream=b)[0])
    torch.cuda.synchronize()
    for w, xs in zip(want, got):
        assert all(torch.equal(w, x) for x in xs)


def test_decode_logits_and_scales_over_a_wide_range(tsa):
    """Large logits of both signs (one row takes all the weight), blocks whose
    scales differ by 2^60, a block of zeros, and a scale of the logits below 0."""
    g = gen(77)
    B, Hq, Hkv, cap = 2, 8, 1, 512
    q = (randn(g, B, Hq, D) * 30).bfloat16()
    kv, rows = bf16_cache(tsa, g, B, Hkv, cap, 0)
    for scale in (1.0, -0.5, 0.0):
        lse = torch.empty((B, Hq), device=DEV)
        out, _ = tsa.window_attn_decode(q, kv, i32([500, 37]), 0, None, scale=scale, lse_out=lse)
        check_decode(q, lambda b, h: (rows(kv.k, b, h), rows(kv.v, b, h)), [500, 37], Hkv, 0, cap,
                     out, lse, scale)
    cache = tsa.KV8.contiguous(B, Hkv, cap, 64, "int8")
    x = randn(g, B, cap, Hkv, D)
    y = x * torch.exp2(torch.randint(-30, 31, (B, cap // 64, 1, 1, 1), generator=g, device=DEV)
                       .float()).expand(-1, -1, 64, 1, 1).reshape(B, cap, 1, 1)
    y[0, 64:128] = 0
    tsa.kv8_append(cache, x.bfloat16().view(-1, Hkv, D), y.bfloat16().view(-1, Hkv, D),
                   i32([cap] * B))
    val = values(cache)
    lse = torch.empty((B, Hq), device=DEV)
    q = (q / 30).bfloat16()
    for lens in ([512, 511], [64, 65], [128, 128]):
        out, _ = tsa.kv8_attn_decode(q, cache, i32(lens), lse_out=lse)
        check_decode(q, lambda b, h: (val[0][b, h], val[1][b, h]), lens, Hkv, 0, cap, out, lse,
                     steps=lambda b, h: value_steps(cache, b, h))
    # a window over the block of zeros alone
    out, _ = tsa.kv8_attn_decode(q, cache, i32([128, 128]), 0, 64, lse_out=lse)
    assert (out[0] == 0).all()
    check_decode(q, lambda b, h: (val[0][b, h], val[1][b, h]), [128, 128], Hkv, 0, 64, out, lse,
                 steps=lambda b, h: value_steps(cache, b, h))


def test_invisible_rows_and_pages_do_not_matter(tsa):
    """NaN and infinities in rows that nothing sees, page-table entries of
    evicted pages that point nowhere, windows that end inside pages."""
    g = gen(5)
    B, Hq, Hkv, cap, page = 2, 8, 2, 1024, 32
    lens, ni, nr = [1000, 517], 5, 300
    kv, rows = bf16_cache(tsa, g, B, Hkv, cap, page)
    cache, _ = quant_cache(tsa, g, B, Hkv, cap, 32, "e4m3", page)
    q = randn(g, B, Hq, D).bfloat16()
    qp = randn(g, 20, Hq, D).bfloat16()
    cu = i32([0, 13, 20])
    outs = []
    for poison in (False, True):
        if poison:
            for b, L in enumerate(lens):
                n = [13, 7][b]
                for p in range(cap):
                    if p >= L or ni <= p <= L - n - nr:   # no query of either call sees it
                        pg, r = place(cache, b, p)
                        cache.k[pg, :, r], cache.v[pg, :, r] = 0x7f, 0xff  # NaN
                        pg = int(kv.page_table[b, p // page])
                        kv.k[pg, :, p % page] = math.nan
                        kv.v[pg, :, p % page] = math.inf if p % 2 else math.nan
                gone = [j for j in range(cap // page) if j * page >= L or
                        (j * page >= ni and (j + 1) * page <= L - n - nr + 1)]
                kv.page_table[b, gone] = -7
                cache.page_table[b, gone] = 1 << 30
        ws = tsa.attn_decode_workspace(B, Hq, Hkv)
        wp = tsa.window_attn_prefill_workspace(B, Hq, Hkv, 13, cap, ni, nr)
        outs.append((tsa.window_attn_decode(q, kv, i32(lens), ni, nr, workspace=ws)[0],
                     tsa.kv8_attn_decode(q, cache, i32(lens), ni, nr, workspace=ws)[0],
                     tsa.window_attn_prefill(qp, kv, i32(lens), ni, nr, cu, 13, workspace=wp)[0]))
        assert tsa.workspace_status(ws) == 0 and tsa.workspace_status(wp) == 0
    for a, b in zip(*outs):
        assert torch.isfinite(a).all() and torch.equal(a, b)


def test_bad_visible_pages_and_lengths_are_reported(tsa):
    g = gen(6)
    B, Hq, Hkv, cap, page = 3, 4, 1, 256, 32
    kv, _ = bf16_cache(tsa, g, B, Hkv, cap, page)
    cache, _ = quant_cache(tsa, g, B, Hkv, cap, 32, "int8", page)
    q = randn(g, B, Hq, D).bfloat16()
    ws = tsa.attn_decode_workspace(B, Hq, Hkv)
    wp = tsa.window_attn_prefill_workspace(B, Hq, Hkv, 1, cap, 4, 64)
    kv.page_table[1, 7], cache.page_table[1, 7] = -1, cache.k.shape[0]
    lens = i32([256, 256, 200])
    for call in (lambda: tsa.window_attn_decode(q, kv, lens, 4, 64, workspace=ws)[0],
                 lambda: tsa.kv8_attn_decode(q, cache, lens, 4, 64, workspace=ws)[0],
                 lambda: tsa.window_attn_prefill(q, kv, lens, 4, 64, workspace=wp)[0]):
        w = wp if call().dtype == torch.bfloat16 else ws
        assert torch.isnan(call()).view(B, -1).all(1).tolist() == [False, True, False]
        assert not torch.isnan(call()[[0, 2]]).any()
        assert tsa.workspace_status(w) == -5 and tsa.workspace_status(w) == 0
    for L in (-3, 257):
        bad = i32([L, 30, 30])
        a = tsa.window_attn_decode(q, kv, bad, 4, 64, workspace=ws)[0]
        assert tsa.workspace_status(ws) == -5
        assert torch.equal(a, tsa.window_attn_decode(q, kv, i32([max(0, min(L, cap)), 30, 30]), 4,
                                                     64, workspace=ws)[0])
        assert tsa.workspace_status(ws) == 0


def test_far_rows_of_large_caches(tsa):
    """Row offsets past 2^32 bytes: the last head of a 4M-position cache."""
    Hkv, cap, L = 5, 1 << 22, (1 << 22) - 3
    q = randn(gen(8), 1, Hkv, D).bfloat16()
    k = torch.empty((1, Hkv, cap, D), dtype=torch.bfloat16, device=DEV)
    v = torch.empty_like(k)
    for t, s in ((k, 1), (v, 2)):
        t[:, :, :16] = randn(gen(s), 1, Hkv, 16, D)
        t[:, :, L - 400:] = randn(gen(s + 5), 1, Hkv, cap - L + 400, D)
    kv = tsa.kv_contiguous(k, v)
    lse = torch.empty((1, Hkv), device=DEV)
    out, _ = tsa.window_attn_decode(q, kv, i32([L]), 7, 300, lse_out=lse)
    idx = torch.cat([torch.arange(7), torch.arange(L - 300, L)]).to(DEV)
    one = torch.ones((1, 307), dtype=torch.bool, device=DEV)
    for h in range(Hkv):
        r = attend64(q[0, h:h + 1], k[0, h, idx], v[0, h, idx], one, 1 / math.sqrt(D))
        decode_close(out[0, h:h + 1], lse[0, h:h + 1], *r, n=307)
    qp = randn(gen(9), 40, Hkv, D).bfloat16()
    lp = torch.empty((40, Hkv), device=DEV)
    op, _ = tsa.window_attn_prefill(qp, kv, i32([L]), 7, 300, lse_out=lp)
    idx = torch.cat([torch.arange(7), torch.arange(L - 339, L)]).to(DEV)
    p = torch.arange(L - 40, L, device=DEV)[:, None]
    seen = (idx <= p) & ((idx < 7) | (idx > p - 300))
    for h in range(Hkv):
        r = attend64(qp[:, h], k[0, h, idx], v[0, h, idx], seen, 1 / math.sqrt(D))
        prefill_close(op[:, h], lp[:, h], *r, n=340)
    del k, v, kv
    cap = 1 << 23
    cache = tsa.KV8.contiguous(1, Hkv, cap, 64, "int8")
    x, y = (randn(gen(s), 5000, Hkv, D).bfloat16() for s in (1, 2))
    tsa.kv8_append(cache, x, y, i32([cap]))
    kr, vr = tsa.kv8_read(cache, i32([cap]), n=5000)
    assert ((kr.double() - x.double()).abs() <= 0.51 * cache.k_scale.max()).all()
    out, _ = tsa.kv8_attn_decode(q, cache, i32([cap]), 0, 4321, lse_out=lse)
    for h in range(Hkv):
        r = attend64(q[0, h:h + 1], kr[-4321:, h], vr[-4321:, h],
                     torch.ones((1, 4321), dtype=torch.bool, device=DEV), 1 / math.sqrt(D))
        decode_close(out[0, h:h + 1], lse[0, h:h + 1], *r, n=4321)


def prefill_close(out, lse, ref, rlse, pv, zabs, n):
    # as decode_close, with the weights in one bf16 part (HALF of each) and the
    # output rounded to bf16
    eps = 2 * (zabs * 2.0 ** -19 + 2.0 ** -20 + n * 2.0 ** -27)
    tol = pv * (eps[:, None] + HALF) + (ref.abs() + pv * HALF) * HALF + 1e-30
    bad = (out.double() - ref).abs() > tol
    assert not bad.any(), float(((out.double() - ref).abs() / tol).max())
    empty = rlse.isinf()
    assert torch.equal(lse.isinf(), empty) and (out[empty] == 0).all()
    assert ((lse.double() - rlse).abs()[~empty] <= (eps + rlse.abs() * 2.0 ** -22)[~empty]).all()


PREFILL_CASES = [  # Hq, Hkv, cap, page, lens, news, n_init, n_recent
    (4, 1, 64, 0, [1], [1], 0, None), (8, 2, 256, 16, [130], [130], 0, None),
    (6, 2, 1024, 0, [700, 300, 5], [700, 1, 0], 4, 64),
    (28, 4, 2048, 16, [2048, 1500, 77, 1024], [129, 64, 77, 500], 4, 256),
    (5, 5, 1024, 64, [1000, 999], [300, 257], 130, 100), (3, 1, 640, 32, [640], [600], 0, 1),
    (32, 8, 512, 256, [400, 512], [33, 200], 5, 0), (2, 2, 512, 0, [512, 64], [100, 64], 0, 0),
    (14, 2, 2048, 128, [2047, 1025], [1000, 1025], 1, 129), (12, 4, 1500, 0, [1499], [1499], 64, 512),
    (7, 1, 1024, 16, list(range(10, 1010, 100)), [10, 100, 3, 7, 200, 1, 64, 65, 128, 9], 2, 77),
    (4, 4, 256, 0, [3, 256], [5, 256], 2, 300),   # more tokens than positions
    (16, 2, 8192, 0, [8192], [17], 16, None),
    # few queries over many rows: their key tiles are split over CTAs
    (28, 4, 16384, 16, [16384, 9000], [1, 16], 4, None), (4, 1, 20000, 0, [19999], [40], 0, 9000),
    (32, 8, 8192, 64, [8000], [2], 130, 700), (1, 1, 30000, 0, [29999], [129], 300, None),
    (8, 1, 4096, 256, [4096, 5, 0], [3, 5, 1], 0, 600)]


@pytest.mark.parametrize("case", PREFILL_CASES, ids=range(len(PREFILL_CASES)))
def test_window_attn_prefill(tsa, case):
    Hq, Hkv, cap, page, lens, news, ni, nr = case
    B, G, T = len(lens), Hq // Hkv, sum(news)
    g = gen(cap + T)
    fused = randn(g, T + 9, Hq + 3, D).bfloat16()
    q = fused[:, 2:2 + Hq]                                   # strided, with rows to spare
    kv, rows = bf16_cache(tsa, g, B, Hkv, cap, page)
    cu = [0]
    for n in news:
        cu.append(cu[-1] + n)
    out = torch.full((T + 9, Hq, D), 9.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((T + 9, Hq), 9.0, device=DEV)
    ws = tsa.window_attn_prefill_workspace(B, Hq, Hkv, max(news), cap, ni, nr)
    tsa.window_attn_prefill(q, kv, i32(lens), ni, nr, i32(cu), max(news), out=out, lse_out=lse,
                            workspace=ws)
    assert (out[T:] == 9).all() and (lse[T:] == 9).all()
    w = cap if nr is None else nr
    for b, (L, n) in enumerate(zip(lens, news)):
        seen = seen_of(torch.arange(L - n, L), L, ni, w)
        for h in range(Hq):
            at = slice(cu[b], cu[b + 1])
            r = attend64(q[at, h], rows(kv.k, b, h // G)[:L], rows(kv.v, b, h // G)[:L], seen,
                         1 / math.sqrt(D))
            if n:
                prefill_close(out[at, h], lse[at, h], *r, n=L)
    assert tsa.workspace_status(ws) == 0
    again = torch.empty_like(out)
    tsa.window_attn_prefill(q, kv, i32(lens), ni, nr, i32(cu), max(news), out=again, workspace=ws)
    assert torch.equal(out[:T], again[:T])


def test_prefill_uniform_batch_and_too_many_tokens(tsa):
    g = gen(12)
    B, Hq, Hkv, cap = 3, 8, 2, 512
    kv, _ = bf16_cache(tsa, g, B, Hkv, cap, 0)
    q = randn(g, 3 * 40, Hq, D).bfloat16()
    lens = i32([500, 40, 77])
    a, _ = tsa.window_attn_prefill(q, kv, lens, 4, 64)
    b, _ = tsa.window_attn_prefill(q, kv, lens, 4, 64, i32([0, 40, 80, 120]), 40)
    assert torch.equal(a, b)
    ws = tsa.window_attn_prefill_workspace(B, Hq, Hkv, 40, cap, 4, 64)
    c, _ = tsa.window_attn_prefill(q, kv, lens, 4, 64, i32([0, 40, 81, 120]), 40, workspace=ws)
    assert tsa.workspace_status(ws) == -5
    assert torch.isnan(c[40:80]).all() and torch.equal(c[:40], a[:40])
    assert torch.isfinite(c[81:]).all()


def test_prefill_calls_of_all_sizes_share_a_workspace(tsa):
    """Split and whole calls by turns, eager and captured, on one workspace."""
    g = gen(14)
    kv, _ = bf16_cache(tsa, g, 2, 2, 8192, 32)
    q = randn(g, 700, 8, D).bfloat16()
    calls = [([8192, 8000], 1), ([8192, 100], 350), ([5000], 16), ([40, 8191], 33), ([8192], 700)]
    ws = torch.zeros(max(tsa.window_attn_prefill_workspace(len(ls), 8, 2, n, 8192, 4, 6000).numel()
                         for ls, n in calls), dtype=torch.uint8, device=DEV)
    want = [tsa.window_attn_prefill(q[:len(ls) * n], kv, i32(ls), 4, 6000)[0] for ls, n in calls]
    for _ in range(2):
        for (ls, n), w in zip(calls, want):
            got, _ = tsa.window_attn_prefill(q[:len(ls) * n], kv, i32(ls), 4, 6000, workspace=ws)
            assert torch.equal(got, w)
    lens, out, gr = i32(calls[0][0]), torch.empty_like(want[0]), torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        tsa.window_attn_prefill(q[:2], kv, lens, 4, 6000, out=out, workspace=ws)
    for _ in range(3):
        out.zero_()
        gr.replay()
        assert torch.equal(out, want[0])
        assert torch.equal(tsa.window_attn_prefill(q[:16], kv, i32(calls[2][0]), 4, 6000,
                                                   workspace=ws)[0], want[2])
    assert tsa.workspace_status(ws) == 0


def test_prefill_of_one_token_is_the_decode_step(tsa):
    g = gen(13)
    B, Hq, Hkv, cap = 4, 28, 4, 1024
    kv, _ = bf16_cache(tsa, g, B, Hkv, cap, 16)
    q = randn(g, B, Hq, D).bfloat16()
    lens = i32([1024, 1, 500, 77])
    la, lb = (torch.empty((B, Hq), device=DEV) for _ in range(2))
    a, _ = tsa.window_attn_decode(q, kv, lens, 4, 200, lse_out=la)
    b, _ = tsa.window_attn_prefill(q, kv, lens, 4, 200, lse_out=lb)
    assert ((a - b.float()).abs() <= a.abs() * HALF + 2.5 * HALF).all()
    assert torch.allclose(la, lb, rtol=1e-5, atol=1e-5)


def test_other_streams_graphs_and_shared_workspaces(tsa):
    """Captured and eager calls on one workspace in turn, a stream of its own,
    workspaces made by the call."""
    g = gen(21)
    B, Hq, Hkv, cap = 4, 32, 4, 4096
    kv, _ = bf16_cache(tsa, g, B, Hkv, cap, 16)
    cache, _ = quant_cache(tsa, g, B, Hkv, cap, 16, "int8", 16)
    q, q2 = randn(g, B, Hq, D).bfloat16(), randn(g, B, Hq, D).bfloat16()
    lens, lens2 = i32([4096, 1000, 33, 2000]), i32([17, 4000, 4096, 1])
    ws = tsa.attn_decode_workspace(B, Hq, Hkv)
    want = [tsa.kv8_attn_decode(q, cache, lens)[0], tsa.window_attn_decode(q, kv, lens, 4, 999)[0],
            tsa.kv8_attn_decode(q2, cache, lens2)[0]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = tsa.kv8_attn_decode(q, cache, lens, stream=side)[0]
    side.synchronize()
    assert torch.equal(got, want[0])
    graphs, outs = [], [torch.empty_like(want[0]) for _ in range(2)]
    qs, ls = q.clone(), lens.clone()
    for i in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            if i == 0:
                tsa.kv8_attn_decode(qs, cache, ls, out=outs[0], workspace=ws)
            else:
                tsa.window_attn_decode(qs, kv, ls, 4, 999, out=outs[1], workspace=ws)
        graphs.append(gr)
    for i in (0, 1, 1, 0):
        outs[i].zero_()
        graphs[i].replay()
        assert torch.equal(outs[i], want[i])
    # a smaller and a larger problem between, on the same workspace
    assert torch.equal(tsa.kv8_attn_decode(q2[:1], cache, lens2[:1], workspace=ws)[0], want[2][:1])
    qs.copy_(q2), ls.copy_(lens2)
    graphs[0].replay()
    assert torch.equal(outs[0], want[2])
    assert tsa.workspace_status(ws) == 0


def test_a_step_of_a_serving_program(tsa):
    """Prompt and decode steps as a program runs them: rotate, write, attend.
    The window's partial merged with the rest's is the whole, and the whole over
    the 8-bit cache is close to the whole over the bf16 one."""
    g = gen(31)
    B, Hq, Hkv, cap, ps = 2, 8, 2, 1024, 32
    pt = torch.randperm(B * cap // ps, generator=g, device=DEV).view(B, -1).int().contiguous()
    kp = torch.zeros((B * cap // ps, Hkv, ps, D), dtype=torch.bfloat16, device=DEV)
    vp = torch.zeros_like(kp)
    kv = tsa.kv_paged(kp, vp, pt)
    cache = tsa.KV8.paged(B * cap // ps, Hkv, ps, pt, 32, "int8")
    table = tsa.RopeTable(128, cap, 5e5, "half", "by_parts", 8.0, 512)
    ws = tsa.attn_decode_workspace(B, Hq, Hkv)
    lens = [0, 0]
    for news in ([600, 333], [1, 1], [1, 1], [31, 64], [1, 1]):
        T, cu = sum(news), [0, news[0], sum(news)]
        lens = [a + n for a, n in zip(lens, news)]
        qkv = randn(g, T, Hq + 2 * Hkv, D).bfloat16()
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        pos = torch.cat([torch.arange(L - n, L) for L, n in zip(lens, news)]).int().to(DEV)
        tsa.kv8_append(cache, k, v, i32(lens), cu_new=i32(cu), max_new=max(news), rope=table)
        qr, kr = tsa.rope(q, pos, table, k=k)
        for b in range(B):
            p = pos[cu[b]:cu[b + 1]].long()
            kp[pt[b].long()[p // ps], :, p % ps] = kr[cu[b]:cu[b + 1]]
            vp[pt[b].long()[p // ps], :, p % ps] = v[cu[b]:cu[b + 1]]
        if max(news) > 1:
            out, _ = tsa.window_attn_prefill(qr, kv, i32(lens), 4, 128, i32(cu), max(news))
            assert torch.isfinite(out).all()
            continue
        lse8, lse = (torch.empty((B, Hq), device=DEV) for _ in range(2))
        o8, _ = tsa.kv8_attn_decode(qr, cache, i32(lens), lse_out=lse8, workspace=ws)
        o, _ = tsa.window_attn_decode(qr, kv, i32(lens), 0, None, lse_out=lse, workspace=ws)
        # keys off by half a step of at most 5 sigma / 64: logits by about 0.02 s.d.
        assert (o8 - o).norm() <= 0.1 * o.norm() and (lse8 - lse).abs().max() < 0.05
        # window + sinks here, the other rows by attend_set, merged: the whole
        wo, wl = (torch.empty((B, Hq, D), device=DEV), torch.empty((B, Hq), device=DEV))
        tsa.window_attn_decode(qr, kv, i32(lens), 4, 128, out=wo, lse_out=wl, workspace=ws)
        M = cap
        rest = torch.zeros((B, Hq, M), dtype=torch.int32, device=DEV)
        cnt = torch.zeros((B, Hq), dtype=torch.int32, device=DEV)
        for b, L in enumerate(lens):
            m = torch.arange(4, L - 128, device=DEV).int()
            rest[b, :, :len(m)], cnt[b] = m, len(m)
        al = torch.empty((B, Hq), device=DEV)
        ao = tsa.attend_set(qr.contiguous(), kv, rest, cnt, lse_out=al)
        mo, ml = tsa.lse_merge(wo.view(-1, D), wl.view(-1), ao.view(-1, D), al.view(-1))
        assert torch.allclose(mo.view_as(o), o, rtol=0, atol=1e-4)
        assert torch.allclose(ml.view_as(lse), lse, rtol=0, atol=1e-4)
    assert tsa.workspace_status(cache.status) == 0 and tsa.workspace_status(ws) == 0
