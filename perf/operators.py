"""Cases for the cache-side operators: rotary positions, the 8-bit KV cache
(written, read back, attended) and sliding-window attention with sinks.

Every operator has a plain form here (elementary torch operations in 32 bits,
angles in 64) beside the call of the library's own kernel.  Four kinds:

  rope    q and k of T tokens rotated by their positions
  append  new tokens' K and V written into the 8-bit cache (a power-of-two
          scale per block of tokens and KV head), keys rotated on the way
          where the case says so, then the rows of the last `back` positions
          read back
  kv8     one decode step of attention over the 8-bit cache
  decode  one decode step over a bf16 cache, sliding window + sinks
  prompt  many new tokens per sequence over a bf16 cache, window + sinks

Geometries are the repository's: 32/8, 32/4, 28/4 and 4/1 query/KV heads,
head dimension 128, caches of 4K to 1M positions, pages of 16 to 256.
"""
import math

import torch

own = False

D = 128
_DEV = "cuda"
_MIN_EXP = -60          # smallest scale exponent of a block
_LAYOUTS = ("half", "interleaved")


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of a 16-sequence batch: launch latency decides
        dict(name="rope_step", op="rope", T=16, Hq=32, Hkv=4, rot=64, layout="interleaved",
             scaling="yarn", theta=10000.0, factor=16.0, orig=8192, max_pos=131072, inverse=False),
        # a whole 32K prompt, wavelength-banded scaling for a 128K context
        dict(name="rope_prompt", op="rope", T=32768, Hq=32, Hkv=8, rot=128, layout="half",
             scaling="by_parts", theta=500000.0, factor=8.0, orig=8192, max_pos=131072,
             inverse=False),
        # every decode step of a paged batch writes one token per sequence
        dict(name="append_step", op="append", B=16, Hkv=4, lo=8191, hi=32767, new_lo=1, new_hi=1,
             back=16, page=16, block=16, fmt="int8", l_cap=32768, rot=128, layout="half", mix=3),
        # chunked prompts of several sequences, ragged, starting inside blocks
        dict(name="append_chunks", op="append", B=8, Hkv=4, lo=4097, hi=16381, new_lo=1,
             new_hi=2047, back=128, page=256, block=128, fmt="int8", l_cap=16384, rot=96,
             layout="half", mix=5),
        # a 128K prompt written at once and read back whole
        dict(name="append_prompt", op="append", B=1, Hkv=8, lo=131071, hi=131071, new_lo=131071,
             new_hi=131071, back=131071, page=0, block=64, fmt="e4m3", l_cap=131072, rot=0,
             layout="half", mix=0),
        # the smallest step: one sequence, one KV head, 4K keys
        dict(name="kv8_small", op="kv8", B=1, Hq=4, Hkv=1, lo=4095, hi=4095, page=0, block=64,
             fmt="int8", l_cap=4096, n_init=0, n_recent=-1, mix=0),
        # the paged serving batch, 8K to 128K keys a sequence
        dict(name="kv8_batch", op="kv8", B=16, Hq=32, Hkv=4, lo=8192, hi=131072, page=16,
             block=16, fmt="int8", l_cap=131072, n_init=0, n_recent=-1, mix=11),
        # one sequence of a million keys
        dict(name="kv8_million", op="kv8", B=1, Hq=32, Hkv=8, lo=1048575, hi=1048575, page=0,
             block=64, fmt="e4m3", l_cap=1048576, n_init=0, n_recent=-1, mix=0),
        # the static window of a 128K decode step: 640 visible rows a head
        dict(name="decode_window", op="decode", B=1, Hq=32, Hkv=8, lo=131071, hi=131071, page=0,
             l_cap=131072, n_init=128, n_recent=512, mix=0),
        # a large paged batch with a wide window
        dict(name="decode_batch", op="decode", B=64, Hq=28, Hkv=4, lo=2001, hi=32768, page=64,
             l_cap=32768, n_init=64, n_recent=4096, mix=7),
        # chunked prefill: ragged chunks late in long paged caches, 7 heads a group
        dict(name="prompt_chunks", op="prompt", B=8, Hq=28, Hkv=4, lo=8191, hi=65536, q_lo=33,
             q_hi=512, page=16, l_cap=65536, n_init=4, n_recent=1024, mix=9),
        # a whole 32K prompt
        dict(name="prompt_32k", op="prompt", B=1, Hq=32, Hkv=8, lo=32768, hi=32768, q_lo=32768,
             q_hi=32768, page=0, l_cap=32768, n_init=128, n_recent=4096, mix=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "kv8", "decode", "prompt"])
    Hq, Hkv = rng.choice([(32, 8), (32, 4), (28, 4), (4, 1), (12, 4), (6, 2), (5, 5)])
    mix = rng.randrange(1, 1000)
    if op == "rope":
        return dict(op=op, T=_log(rng, 1, 24000), Hq=Hq, Hkv=Hkv,
                    rot=rng.choice([16, 32, 64, 96, 112, 128]), layout=rng.choice(_LAYOUTS),
                    scaling=rng.choice(["none", "linear", "ntk", "by_parts", "yarn"]),
                    theta=rng.choice([10000.0, 500000.0, 1000000.0]),
                    factor=rng.choice([2.0, 4.0, 8.0, 16.0]), orig=rng.choice([4096, 8192, 32768]),
                    max_pos=rng.choice([32768, 131072, 1048576]), inverse=rng.random() < 0.25)
    page = rng.choice([0, 0, 16, 32, 64, 128, 256])
    if op == "append":
        block = rng.choice([16, 32, 64, 128] if page == 0 else
                           [x for x in (16, 32, 64, 128) if x <= page])
        B = _log(rng, 1, 32)
        new = _log(rng, 1, 60000 // B)
        hi = new + _log(rng, 1, 8000)
        cap = -(-hi // 256) * 256
        return dict(op=op, B=B, Hkv=Hkv, lo=min(hi, new + 1), hi=hi, new_lo=(new + 1) // 2,
                    new_hi=new, back=min(block, (new + 1) // 2 + 1), page=page, block=block,
                    fmt=rng.choice(["int8", "e4m3"]), l_cap=cap, rot=rng.choice([0, 64, 96, 128]),
                    layout=rng.choice(_LAYOUTS), mix=mix)
    if op in ("kv8", "decode"):
        B = _log(rng, 1, 64)
        hi = _log(rng, 17, min(262144, 1600000 // (B * Hkv)))
        cap = -(-hi // 256) * 256
        windowed = op == "decode" or rng.random() < 0.3
        c = dict(op=op, B=B, Hq=Hq, Hkv=Hkv, lo=max(1, hi // rng.choice([1, 4, 16])), hi=hi,
                 page=page, l_cap=cap, n_init=rng.choice([0, 1, 4, 64, 130]) if windowed else 0,
                 n_recent=_log(rng, 1, 8192) if windowed else -1, mix=mix)
        if op == "kv8":
            c["block"] = rng.choice([16, 32, 64, 128] if page == 0 else
                                    [x for x in (16, 32, 64, 128) if x <= page])
            c["fmt"] = rng.choice(["int8", "e4m3"])
        return c
    B = _log(rng, 1, 8)
    q_hi = _log(rng, 2, 8192 // B)
    hi = q_hi + _log(rng, 1, 20000)
    return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, lo=(q_hi + hi) // 2, hi=hi, q_lo=(q_hi + 1) // 2,
                q_hi=q_hi, page=page, l_cap=-(-hi // 256) * 256,
                n_init=rng.choice([0, 1, 4, 64, 130]), n_recent=_log(rng, 1, 4096), mix=mix)


def _spread(case, lo, hi, salt):
    """B whole numbers in [lo, hi], the same for every seed."""
    return [lo + (b * 2654435761 + (case["mix"] + salt) * 40503 * 65537 + salt * 97) % (hi - lo + 1)
            for b in range(case["B"])]


def _lens(case):
    return _spread(case, case["lo"], case["hi"], 1)


def _news(case, a="new_lo", b="new_hi"):
    return _spread(case, case[a], case[b], 2)


def _visible(p, n_init, n_recent):
    """Positions that a query at position p sees."""
    rec = min(n_recent, p + 1) if n_recent >= 0 else p + 1
    return rec + max(0, min(n_init, p + 1 - rec))


def work(case):
    op = case["op"]
    if op == "rope":
        rows = case["T"] * (case["Hq"] + case["Hkv"])
        return {"bytes": rows * D * 2 * 2 + case["T"] * 4, "flops": rows * case["rot"] * 3}
    lens = _lens(case)
    if op == "append":
        rows = sum(_news(case)) * case["Hkv"]
        back = case["B"] * case["back"] * case["Hkv"]
        # new rows read (bf16) and written (one byte an element); rows read back, written as bf16
        return {"bytes": rows * D * 2 * 3 + back * D * 2 * 3,
                "flops": rows * D * 2 * 4 + back * D * 2}
    Hq, Hkv, ni, nr = case["Hq"], case["Hkv"], case["n_init"], case["n_recent"]
    if op in ("kv8", "decode"):
        vis = sum(_visible(L - 1, ni, nr) for L in lens)
        row = 2 * D * (1 if op == "kv8" else 2)
        scales = 8.0 / case["block"] if op == "kv8" else 0.0
        return {"bytes": vis * Hkv * (row + scales) + len(lens) * Hq * (D * 6 + 4),
                "flops": vis * Hq * 4 * D}
    rows, pairs, toks = 0, 0, 0
    for L, n in zip(lens, _news(case, "q_lo", "q_hi")):
        pairs += sum(_visible(p, ni, nr) for p in range(L - n, L))
        rows += min(L, min(ni, L) + min(L, n + nr - 1))
        toks += n
    return {"bytes": rows * Hkv * 4 * D + toks * Hq * (4 * D + 4), "flops": pairs * Hq * 4 * D}


# ----------------------------------------------------------------- inputs
def _gen(seed, salt=0):
    g = torch.Generator(device=_DEV)
    g.manual_seed(seed * 1000003 + salt)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=_DEV)


def _keys(g, *shape):
    """Keys off the origin, as the repository's workloads have them."""
    mu = _randn(g, D)
    mu *= 3.0 / mu.norm()
    return _randn(g, *shape, D) + mu


def _table(case, g):
    """Page table of a shuffled pool with some spare pages, or None."""
    if not case["page"]:
        return None, 0
    per = case["l_cap"] // case["page"]
    n = case["B"] * per + 3
    perm = torch.randperm(n, generator=g, device=_DEV)[: case["B"] * per]
    return perm.reshape(case["B"], per).to(torch.int32).contiguous(), n


def _rows(s, pos):
    """Flat row of position pos[b, ...] of every KV head: [B, Hkv, ...]."""
    B, Hkv = s["B"], s["Hkv"]
    view = (B,) + (1,) * (pos.dim() - 1)
    g = torch.arange(Hkv, device=pos.device).reshape((1, Hkv) + (1,) * (pos.dim() - 1))
    if s["table"] is None:
        b = torch.arange(B, device=pos.device).reshape(view).unsqueeze(1)
        return (b * Hkv + g) * s["l_cap"] + pos.unsqueeze(1)
    ps = s["page"]
    b = torch.arange(B, device=pos.device).reshape(view)
    page = s["table"].long()[b, pos // ps]
    return (page.unsqueeze(1) * Hkv + g) * ps + (pos % ps).unsqueeze(1)


def _exponent(amax, fmt):
    """Smallest e with top * 2^e >= amax (top: 127 or 448), not below -60."""
    m, e = torch.frexp(amax)
    cut, off = (127.0 / 128.0, 7) if fmt == "int8" else (448.0 / 512.0, 9)
    e = torch.where(m <= cut, e - off, e - off + 1)
    return torch.where(amax > 0, e.clamp(min=_MIN_EXP), torch.full_like(e, _MIN_EXP))


def _encode(y, fmt):
    """Codes of values already divided by their scale."""
    if fmt == "int8":
        return (torch.round(y).clamp(-127, 127) + 128).to(torch.uint8)
    return y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _decode(codes, fmt):
    if fmt == "int8":
        return codes.float() - 128.0
    return codes.view(torch.float8_e4m3fn).float()


def _cache_shape(case, n_pages):
    if case["page"]:
        return n_pages, case["Hkv"], case["page"]
    return case["B"], case["Hkv"], case["l_cap"]


def _make_cache8(case, g, n_pages):
    """A quantised cache: every row of it coded, whatever the lengths."""
    n, H, rows = _cache_shape(case, n_pages)
    blk, fmt, out = case["block"], case["fmt"], []
    for which in range(2):
        codes = torch.empty((n, H, rows, D), dtype=torch.uint8, device=_DEV)
        scale = torch.empty((n, H, rows // blk), dtype=torch.float32, device=_DEV)
        flat = codes.view(-1, blk, D)
        sflat = scale.view(-1)
        step = max(1, (1 << 27) // (blk * D))
        for i in range(0, flat.shape[0], step):
            m = min(step, flat.shape[0] - i)
            x = _keys(g, m, blk) if which == 0 else _randn(g, m, blk, D)
            e = _exponent(x.abs().amax(dim=(1, 2)), fmt)
            s = torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)
            flat[i:i + m] = _encode(x / s[:, None, None], fmt)
            sflat[i:i + m] = s
        out += [codes, scale]
    return out


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(case)
    s["seed"] = seed
    if op == "rope":
        T = case["T"]
        s["q"] = _randn(g, T, case["Hq"], D).bfloat16()
        s["k"] = _keys(g, T, case["Hkv"]).bfloat16()
        if T <= 64:  # a decode step: each token at its own sequence's position
            pos = torch.randint(0, case["max_pos"], (T,), generator=g, device=_DEV)
        else:        # a prompt, anywhere in the context
            start = int(torch.randint(0, max(1, case["max_pos"] - T), (1,), generator=g,
                                      device=_DEV))
            pos = start + torch.arange(T, device=_DEV) % case["max_pos"]
        s["pos"] = pos.clamp(max=case["max_pos"] - 1).to(torch.int32)
        return s
    s["lens_host"] = _lens(case)
    s["lens"] = torch.tensor(s["lens_host"], dtype=torch.int32, device=_DEV)
    s["table"], n_pages = _table(case, g)
    if op in ("append", "kv8"):
        s["k8"], s["ks"], s["v8"], s["vs"] = _make_cache8(case, g, n_pages)
    else:
        shape = _cache_shape(case, n_pages)
        s["k"], s["v"] = _keys(g, *shape).bfloat16(), _randn(g, *shape, D).bfloat16()
    if op in ("kv8", "decode"):
        q = _randn(g, 1, case["Hq"], D) + 0.3 * _randn(g, case["B"], case["Hq"], D)
        s["q"] = q.bfloat16()
        return s
    news = _news(case) if op == "append" else _news(case, "q_lo", "q_hi")
    cu = [0]
    for n in news:
        cu.append(cu[-1] + n)
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device=_DEV)
    s["max_new"], s["T"] = max(news), cu[-1]
    if op == "append":
        # twice the cached rows' spread in places, so that some scales grow
        amp = 1.0 + (torch.rand((s["T"], 1, 1), generator=g, device=_DEV) < 0.02)
        s["k_new"] = (_keys(g, s["T"], case["Hkv"]) * amp).bfloat16()
        s["v_new"] = (_randn(g, s["T"], case["Hkv"], D) * amp).bfloat16()
    else:
        s["q"] = (_randn(g, 1, case["Hq"], D) + 0.3 * _randn(g, s["T"], case["Hq"], D)).bfloat16()
    return s


# ------------------------------------------------------------ plain forms
def _freqs(c):
    """Rotation rates in 64 bits, [rot/2], and the amplitude."""
    rot, theta, f = c["rot"], c["theta"], c["factor"]
    i = torch.arange(rot // 2, dtype=torch.float64, device=_DEV)
    kind = c["scaling"]
    if kind == "ntk":
        theta = theta * f ** (rot / (rot - 2))
    w = theta ** (-2.0 * i / rot)
    if kind == "linear":
        return w / f, 1.0
    if kind == "by_parts":
        turns = c["orig"] * w / (2 * math.pi)
        t = ((turns - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        return (1 - t) * w / f + t * w, 1.0
    if kind == "yarn":
        lo = rot * math.log(c["orig"] / (2 * math.pi * 32.0)) / (2 * math.log(theta))
        hi = rot * math.log(c["orig"] / (2 * math.pi * 1.0)) / (2 * math.log(theta))
        lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), rot - 1)
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return w / f * ramp + w * (1 - ramp), 0.1 * math.log(f) + 1.0
    return w, 1.0


def _rotate(x, pos, c, inverse=False):
    """x fp32 [T, H, D] rotated; pos [T]."""
    rot = c["rot"]
    w, amp = _freqs(c)
    ang = pos.double()[:, None] * w
    cos, sin = (ang.cos() * amp).float()[:, None], (ang.sin() * amp).float()[:, None]
    if inverse:
        sin = -sin
    y = x.clone()
    if c["layout"] == "half":
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        y[..., : rot // 2], y[..., rot // 2: rot] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    return y


def _spec(s):
    """The rotation of an append case."""
    return dict(rot=s["rot"], layout=s["layout"], scaling="none", theta=500000.0, factor=1.0,
                orig=8192)


def _plain_append(s):
    B, H, blk, fmt = s["B"], s["Hkv"], s["block"], s["fmt"]
    lens, cu = s["lens"].long(), s["cu"].long()
    n = cu[1:] - cu[:-1]
    start = lens - n
    nb = (s["max_new"] + blk - 2) // blk + 1
    # positions of every block that can be touched: [B, nb, blk]
    first = start // blk * blk
    pos = first[:, None, None] + torch.arange(nb * blk, device=_DEV).reshape(1, nb, blk)
    new = (pos >= start[:, None, None]) & (pos < lens[:, None, None])
    old = pos < start[:, None, None]
    at = (cu[:-1, None, None] + (pos - start[:, None, None])).clamp(0, s["T"] - 1)
    rows = _rows(s, pos.clamp(max=s["l_cap"] - 1))                 # [B, H, nb, blk]
    brow = rows[..., 0] // blk
    out = []
    tok = torch.repeat_interleave(torch.arange(B, device=_DEV), n, output_size=s["T"])
    tpos = start[tok] + torch.arange(s["T"], device=_DEV) - cu[tok]
    for x, codes, scale in ((s["k_new"], s["k8"], s["ks"]), (s["v_new"], s["v8"], s["vs"])):
        x = x.float()
        if codes is s["k8"] and s["rot"]:
            x = _rotate(x, tpos, _spec(s))
        x = x[at].permute(0, 3, 1, 2, 4)                           # [B, H, nb, blk, D]
        m = new[:, None, :, :, None]
        fresh = torch.where(m, x, torch.zeros_like(x))
        e = _exponent(fresh.abs().amax(dim=(3, 4)), fmt)
        need = torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)
        flat, sflat = codes.view(-1, D), scale.view(-1)
        had = sflat[brow]
        keep = old.any(dim=2)[:, None]
        sc = torch.where(keep, torch.maximum(had, need), need)
        was = _decode(flat[rows], fmt) * had[..., None, None]
        y = torch.where(m, x, was) / sc[..., None, None]
        c = _encode(y, fmt)
        some = new.any(dim=2)[:, None].expand_as(brow)
        put = ((new | old) & new.any(dim=2, keepdim=True))[:, None].expand_as(rows)
        flat[rows[put]] = c[put]
        sflat[brow[some]] = sc[some]
        out.append(_plain_read(s, codes, scale))
    return out + [s["ks"], s["vs"]]


def _plain_read(s, codes, scale):
    """The last `back` rows of every sequence, [B * back, H, D] bf16."""
    pos = s["lens"].long()[:, None] - s["back"] + torch.arange(s["back"], device=_DEV)
    rows = _rows(s, pos)
    x = _decode(codes.view(-1, D)[rows], s["fmt"]) * scale.view(-1)[rows // s["block"]][..., None]
    return x.permute(0, 2, 1, 3).reshape(-1, s["Hkv"], D).bfloat16()


def _attend(q, k, v, seen, scale):
    """q [N, Hkv, R, D], k and v [N, Hkv, W, D], seen [N, 1 or Hkv, R, W]."""
    z = torch.matmul(q, k.transpose(-1, -2)) * scale
    z.masked_fill_(~seen, -math.inf)
    m = z.amax(dim=-1, keepdim=True)
    z.sub_(torch.where(m.isinf(), torch.zeros_like(m), m)).exp_()
    l = z.sum(dim=-1, keepdim=True)
    o = torch.matmul(z, v) / torch.where(l > 0, l, torch.ones_like(l))
    return o, (m + l.log()).squeeze(-1)


def _plain_step(s):
    B, Hq, H = s["B"], s["Hq"], s["Hkv"]
    ni, nr = s["n_init"], s["n_recent"]
    W = max(s["lens_host"])
    lens = s["lens"].long()[:, None]
    if 0 <= nr and ni + nr < W:  # the visible rows alone
        j = torch.arange(ni + nr, device=_DEV)[None]
        pos = torch.where(j < ni, j, lens - nr + (j - ni))
        ok = (pos < lens) & (pos >= 0) & ((j < ni) | (pos >= ni))
    else:
        pos = torch.arange(W, device=_DEV)[None].expand(B, W)
        ok = pos < lens
        if nr >= 0:
            ok = ok & ((pos >= lens - nr) | (pos < ni))
    pos = pos.clamp(0, s["l_cap"] - 1)
    rows = _rows(s, torch.where(ok, pos, torch.zeros_like(pos)))
    if s["op"] == "kv8":
        k = _decode(s["k8"].view(-1, D)[rows], s["fmt"])
        k *= s["ks"].view(-1)[rows // s["block"]][..., None]
        v = _decode(s["v8"].view(-1, D)[rows], s["fmt"])
        v *= s["vs"].view(-1)[rows // s["block"]][..., None]
    else:
        k, v = s["k"].view(-1, D)[rows].float(), s["v"].view(-1, D)[rows].float()
    o, lse = _attend(s["q"].float().view(B, H, Hq // H, D), k, v, ok[:, None, None],
                     1.0 / math.sqrt(D))
    return [o.reshape(B, Hq, D), lse.reshape(B, Hq)]


def _chunk_positions(s, C):
    """Query positions [B * n, C], their tokens and the key positions that a
    chunk of C queries can see [B * n, W], with what of them counts."""
    n = -(-s["max_new"] // C)
    cu, lens = s["cu"].long(), s["lens"].long()
    j = torch.arange(n * C, device=_DEV).reshape(1, n, C)
    have = (cu[1:] - cu[:-1])[:, None, None]
    tok = cu[:-1, None, None] + j
    p = (lens[:, None, None] - have + j).reshape(-1, C)
    live = (j < have).reshape(-1, C)
    ni, nr = s["n_init"], s["n_recent"]
    top = max(s["lens_host"])
    if ni + nr + C - 1 >= top:
        kp = torch.arange(top, device=_DEV)[None].expand(p.shape[0], top)
        ok = torch.ones_like(kp, dtype=torch.bool)
    else:
        i = torch.arange(ni + nr + C - 1, device=_DEV)[None]
        kp = torch.where(i < ni, i, p[:, :1] - nr + 1 + (i - ni))
        ok = (kp >= 0) & ((i < ni) | (kp >= ni))
    return p, live, tok.reshape(-1, C).clamp(max=s["T"] - 1), kp, ok, n


def _plain_prompt(s):
    B, Hq, H, T = s["B"], s["Hq"], s["Hkv"], s["T"]
    G = Hq // H
    C = min(s["max_new"], 1024)
    p, live, tok, kp, ok, n = _chunk_positions(s, C)
    N, W = kp.shape
    kc = kp.clamp(0, s["l_cap"] - 1)
    rows = _rows(s, kc.reshape(B, n * W)).reshape(B, H, n, W).transpose(1, 2).reshape(N, H, W)
    k, v = s["k"].view(-1, D)[rows].float(), s["v"].view(-1, D)[rows].float()
    q = s["q"].float()[tok]                                        # [N, C, Hq, D]
    q = q.view(N, C, H, G, D).permute(0, 2, 3, 1, 4).reshape(N, H, G * C, D)
    kq, pq = kp[:, None, :], p[:, :, None]
    seen = ok[:, None] & (kq <= pq) & ((kq > pq - s["n_recent"]) | (kq < s["n_init"]))
    seen = seen[:, None].expand(N, G, C, W).reshape(N, 1, G * C, W)
    o, lse = _attend(q, k, v, seen, 1.0 / math.sqrt(D))
    o = o.view(N, H, G, C, D).permute(0, 3, 1, 2, 4).reshape(N, C, Hq, D)
    lse = lse.view(N, H, G, C).permute(0, 3, 1, 2).reshape(N, C, Hq)
    out = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=_DEV)
    lo = torch.empty((T, Hq), dtype=torch.float32, device=_DEV)
    out[tok[live]] = o[live].bfloat16()
    lo[tok[live]] = lse[live]
    return [out, lo]


# ------------------------------------------------------- the library's own
def _kept(s, key, make):
    """What a program makes once and keeps beside its buffers."""
    if key not in s:
        s[key] = make()
    return s[key]


def _rope_table(tsa, s, c):
    return _kept(s, "rope", lambda: tsa.RopeTable(
        c["rot"], s.get("max_pos", s.get("l_cap")), theta=c["theta"], layout=c["layout"],
        scaling=c["scaling"], factor=c["factor"], orig_len=c["orig"], device=_DEV))


def _own_run(s):
    import top_retrieval_sparse_gb300 as tsa
    op = s["op"]
    if op == "rope":
        return tsa.rope(s["q"], s["pos"], _rope_table(tsa, s, s), k=s["k"], inverse=s["inverse"])
    if op in ("append", "kv8"):
        cache = _kept(s, "cache", lambda: tsa.KV8(s["k8"], s["v8"], s["ks"], s["vs"],
                                                  fmt=s["fmt"], page_table=s["table"]))
    if op == "append":
        rope = _rope_table(tsa, s, _spec(s)) if s["rot"] else None
        tsa.kv8_append(cache, s["k_new"], s["v_new"], s["lens"], cu_new=s["cu"],
                       max_new=s["max_new"], rope=rope)
        k, v = tsa.kv8_read(cache, s["lens"], s["back"])
        return [k, v, s["ks"], s["vs"]]
    if op != "kv8":
        cache = _kept(s, "cache", lambda: tsa.KV(s["k"], s["v"], s["table"], s["page"]))
    T = s["q"].shape[0]
    lse = _kept(s, "lse", lambda: torch.empty((T, s["Hq"]), dtype=torch.float32, device=_DEV))
    nr = None if s["n_recent"] < 0 else s["n_recent"]
    if op == "prompt":
        ws = _kept(s, "ws", lambda: tsa.window_attn_prefill_workspace(
            s["B"], s["Hq"], s["Hkv"], s["max_new"], s["l_cap"], s["n_init"], nr, device=_DEV))
        return tsa.window_attn_prefill(s["q"], cache, s["lens"], s["n_init"], nr, cu_q=s["cu"],
                                       max_q=s["max_new"], lse_out=lse, workspace=ws)
    ws = _kept(s, "ws", lambda: tsa.attn_decode_workspace(s["B"], s["Hq"], s["Hkv"], device=_DEV))
    call = tsa.kv8_attn_decode if op == "kv8" else tsa.window_attn_decode
    return call(s["q"], cache, s["lens"], s["n_init"], nr, lse_out=lse, workspace=ws)


def run(state):
    if own:
        return list(_own_run(state))
    op = state["op"]
    if op == "rope":
        q = _rotate(state["q"].float(), state["pos"], state, state["inverse"])
        k = _rotate(state["k"].float(), state["pos"], state, state["inverse"])
        return [q.bfloat16(), k.bfloat16()]
    if op == "append":
        return _plain_append(state)
    return _plain_prompt(state) if op == "prompt" else _plain_step(state)


# ------------------------------------------------------------------ exact
def _turn64(x, pos, c, inverse=False):
    """The rotation as a product of complex numbers, 64 bits."""
    rot = c["rot"]
    w, amp = _freqs(c)
    ang = pos.double()[:, None] * w
    unit = torch.polar(torch.full_like(ang, amp), -ang if inverse else ang)[:, None]
    r = x[..., :rot]
    if c["layout"] == "half":
        z = torch.complex(*(t.contiguous() for t in r.chunk(2, dim=-1))) * unit
        r = torch.cat([z.real, z.imag], dim=-1)
    else:
        r = torch.view_as_real(torch.view_as_complex(r.reshape(*r.shape[:-1], -1, 2)) * unit)
        r = r.flatten(-2)
    return torch.cat([r, x[..., rot:]], dim=-1)


def _step64(y, fmt):
    """Values of the 8-bit grid nearest to y (ties to even), 64 bits."""
    if fmt == "int8":
        return torch.round(y).clamp(-127, 127)
    unit = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(y / unit) * unit).clamp(-448, 448)


def _seq_rows(s, b, h, n):
    """Flat rows of positions 0..n-1 of one sequence and KV head."""
    pos = torch.arange(n, device=_DEV)
    if s["table"] is None:
        return (b * s["Hkv"] + h) * s["l_cap"] + pos
    page = s["table"][b].long()[pos // s["page"]]
    return (page * s["Hkv"] + h) * s["page"] + pos % s["page"]


def _exact_append(s):
    top = 127.0 if s["fmt"] == "int8" else 448.0
    blk, H, back = s["block"], s["Hkv"], s["back"]
    got, scales = [], []
    cu = s["cu"].tolist()
    for x, codes, scale in ((s["k_new"], s["k8"], s["ks"]), (s["v_new"], s["v8"], s["vs"])):
        x, sc = x.double(), scale.double().clone().view(-1)
        out = torch.empty((s["B"], back, H, D), dtype=torch.float64, device=_DEV)
        for b, L in enumerate(s["lens_host"]):
            n = cu[b + 1] - cu[b]
            L0, part = L - n, x[cu[b]:cu[b + 1]]
            if codes is s["k8"] and s["rot"]:
                part = _turn64(part, torch.arange(L0, L, device=_DEV), _spec(s))
            lo = min(L0 // blk, (L - back) // blk) * blk       # from a block's start
            for h in range(H):
                rows = _seq_rows(s, b, h, L)[lo:]
                val = _decode(codes.view(-1, D)[rows], s["fmt"]).double()
                val *= sc[rows // blk][:, None]
                val[L0 - lo:] = part[:, h]
                pad = -len(rows) % blk
                full = torch.cat([val, val.new_zeros((pad, D))]).view(-1, blk, D)
                place = torch.arange(lo, lo + len(rows) + pad, device=_DEV).view(-1, blk)
                is_new = (place >= L0) & (place < L)
                amax = (full.abs().amax(dim=2) * is_new).amax(dim=1)
                # the logarithm of a power of two may come out a hair above it
                e = torch.ceil(torch.log2(amax.clamp(min=1e-300) / top) - 1e-10)
                e = e.clamp(min=_MIN_EXP)
                need = torch.exp2(e)
                at = rows[::blk] // blk
                has_old, touched = place[:, 0] < L0, is_new.any(dim=1)
                fin = torch.where(touched, torch.where(has_old, torch.maximum(sc[at], need),
                                                       need), sc[at])
                sc[at] = fin
                val = _step64(full / fin[:, None, None], s["fmt"]) * fin[:, None, None]
                out[b, :, h] = val.view(-1, D)[L - back - lo: L - lo]
        got.append(out.view(-1, H, D))
        scales.append(sc.view(scale.shape))
    return got + scales


def _soft64(q, k, v, seen):
    """Attention of rows q over k, v by logsumexp, 64 bits."""
    z = (q @ k.T) / math.sqrt(D)
    z = torch.where(seen, z, torch.full_like(z, -math.inf))
    lse = torch.logsumexp(z, dim=-1)
    w = torch.where(seen, torch.exp(z - torch.where(lse.isinf(), 0.0, lse)[..., None]), 0.0)
    return w @ v, lse


def _exact_attention(s):
    prompt = s["op"] == "prompt"
    T, Hq, H = s["q"].shape[0], s["Hq"], s["Hkv"]
    G = Hq // H
    out = torch.empty((T, Hq, D), dtype=torch.float64, device=_DEV)
    lse = torch.empty((T, Hq), dtype=torch.float64, device=_DEV)
    cu = s["cu"].tolist() if prompt else list(range(T + 1))
    for b, L in enumerate(s["lens_host"]):
        for t0 in range(cu[b], cu[b + 1], 2048):
            t1 = min(t0 + 2048, cu[b + 1])
            p = L - cu[b + 1] + torch.arange(t0, t1, device=_DEV)
            first, last = L - cu[b + 1] + t0, L - cu[b + 1] + t1
            nr = s["n_recent"] if s["n_recent"] >= 0 else L
            j = torch.arange(last, device=_DEV)
            j = j[(j < s["n_init"]) | (j > first - nr)]
            seen = (j <= p[:, None]) & ((j > p[:, None] - nr) | (j < s["n_init"]))
            for h in range(H):
                rows = _seq_rows(s, b, h, L)[j]
                if s["op"] == "kv8":
                    at = rows // s["block"]
                    k = _decode(s["k8"].view(-1, D)[rows], s["fmt"]).double()
                    k *= s["ks"].view(-1)[at].double()[:, None]
                    v = _decode(s["v8"].view(-1, D)[rows], s["fmt"]).double()
                    v *= s["vs"].view(-1)[at].double()[:, None]
                else:
                    k, v = s["k"].view(-1, D)[rows].double(), s["v"].view(-1, D)[rows].double()
                for i in range(h * G, (h + 1) * G):
                    o, l = _soft64(s["q"][t0:t1, i].double(), k, v, seen)
                    out[t0:t1, i], lse[t0:t1, i] = o, l
    return [out, lse]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return [_turn64(s[x].double(), s["pos"], s, s["inverse"]) for x in ("q", "k")]
    return _exact_append(s) if case["op"] == "append" else _exact_attention(s)
