"""Cases for the operators of shared caches: pages that sequences take, share, move
and give back, attention of a batch that shares long prefixes, and rotary
positions with several axes.

Every operator has a plain form here (elementary torch operations in 32 bits,
angles in 64) beside the call of the library's own kernel.  Six kinds:

  step     the pages of one decode step: taken for the new tokens, given back
           where they fell out of the window
  fork     sequences forked (whole pages shared, the last partial one copied),
           every layer's rows copied; 8-bit caches are read back
  compact  sequences leave, the pool's live pages move to its front
  shared   one decode step of attention over groups of sequences that share
           their first rows
  axes     q and k rotated by positions of two to four axes
  append   new tokens written into the 8-bit cache, keys rotated by such
           positions, and read back

Geometries are the repository's: 32/8, 32/4, 28/4 and 4/1 query/KV heads,
head dimension 128, caches of 4K to 128K positions, pages of 16 to 256.
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
        # the page bookkeeping of every decode step: one token a sequence, a window behind it
        dict(name="pages_step", op="step", B=16, page=16, lo=4097, hi=32767, l_cap=32768, new=1,
             n_init=64, n_recent=1024, mix=3),
        # four samples of one prompt, two layers of an 8-bit cache
        dict(name="fork_samples", op="fork", N=1, C=4, page=16, lo=4001, hi=4001, l_cap=8192,
             Hkv=4, layers=2, fmt="int8", block=16, back=16, mix=5),
        # beams of a batch: 16 sequences of up to 32K tokens, each forked four times, eight layers
        dict(name="fork_beams", op="fork", N=16, C=4, page=64, lo=8191, hi=32767, l_cap=32768,
             Hkv=4, layers=8, fmt="bf16", block=0, back=0, mix=7),
        # a third of the requests has ended: the pool of two layers becomes dense again
        dict(name="compact_pool", op="compact", B=48, page=64, lo=1025, hi=16381, l_cap=16384,
             Hkv=4, layers=2, spare=40, mix=11),
        # the smallest step: four sequences of one prompt, one KV head
        dict(name="shared_small", op="shared", N=1, s_lo=4, s_hi=4, p_lo=4001, p_hi=4001, o_lo=1,
             o_hi=95, Hq=4, Hkv=1, page=0, fmt="bf16", block=0, out="fp32", mix=1),
        # a serving batch under one long system prompt
        dict(name="shared_batch", op="shared", N=1, s_lo=64, s_hi=64, p_lo=32767, p_hi=32767,
             o_lo=1, o_hi=1023, Hq=32, Hkv=8, page=16, fmt="bf16", block=0, out="fp32", mix=2),
        # several prompts of very different lengths in one batch, 8-bit pages
        dict(name="shared_groups", op="shared", N=6, s_lo=1, s_hi=15, p_lo=2001, p_hi=131001,
             o_lo=0, o_hi=2047, Hq=32, Hkv=4, page=64, fmt="int8", block=64, out="fp32", mix=9),
        # a million keys' worth of documents, eight questions on each (e4m3)
        dict(name="shared_documents", op="shared", N=8, s_lo=8, s_hi=8, p_lo=98304, p_hi=131072,
             o_lo=33, o_hi=512, Hq=32, Hkv=8, page=256, fmt="e4m3", block=128, out="bf16", mix=4),
        # 256 samples of one 128K prompt: the matrix products bound it
        dict(name="shared_samples", op="shared", N=1, s_lo=256, s_hi=256, p_lo=131071,
             p_hi=131071, o_lo=1, o_hi=511, Hq=28, Hkv=4, page=256, fmt="bf16", block=0,
             out="bf16", mix=6),
        # a decode step of 64 sequences behind images
        dict(name="axes_step", op="axes", T=64, Hq=28, Hkv=4, rot=128, sections="16,24,24",
             order="blocks", rates="joint", layout="half", theta=1000000.0, max_pos=131072,
             inverse=False),
        # a prompt of text, images and video frames
        dict(name="axes_prompt", op="axes", T=32767, Hq=32, Hkv=8, rot=128, sections="24,20,20",
             order="turns", rates="joint", layout="half", theta=500000.0, max_pos=131072,
             inverse=False),
        # chunks of such prompts on their way into the 8-bit cache
        dict(name="append_axes", op="append", B=8, Hkv=4, new_lo=257, new_hi=4095, off_hi=8,
             back=128, page=64, block=64, fmt="e4m3", rot=128, sections="16,24,24",
             order="blocks", rates="joint", layout="half", theta=1000000.0, mix=13),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


_SECTIONS = [(16, "4,4"), (32, "5,5,6"), (64, "16,16"), (64, "8,12,12"), (96, "16,16,16"),
             (128, "16,24,24"), (128, "24,20,20"), (128, "22,21,21"), (128, "33,31"),
             (128, "16,16,16,16")]


def draw(rng):
    op = rng.choice(["step", "fork", "compact", "shared", "shared", "shared", "axes", "append"])
    Hq, Hkv = rng.choice([(32, 8), (32, 4), (28, 4), (4, 1), (12, 4), (6, 2), (5, 5)])
    mix = rng.randrange(1, 1000)
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "step":
        hi = _log(rng, 64, 65536)
        return dict(op=op, B=_log(rng, 1, 256), page=page, lo=max(1, hi // 8), hi=hi,
                    l_cap=-(-hi // page) * page, new=rng.choice([1, 1, 2, 5, 33]),
                    n_init=rng.choice([0, 4, 64, 130]), n_recent=_log(rng, 1, 8192), mix=mix)
    if op == "fork":
        N, C = _log(rng, 1, 16), rng.choice([1, 2, 3, 4, 8])
        hi = _log(rng, 2 * page, 32768 // N + 2 * page)
        fmt = rng.choice(["bf16", "bf16", "int8", "e4m3"])
        return dict(op=op, N=N, C=C, page=page, lo=max(page, hi // 4), hi=hi,
                    l_cap=-(-hi // page) * page, Hkv=Hkv, layers=rng.choice([1, 2, 3]), fmt=fmt,
                    block=0 if fmt == "bf16" else rng.choice([16, page]) if page <= 128 else 128,
                    back=0 if fmt == "bf16" else rng.choice([1, 16]), mix=mix)
    if op == "compact":
        B = _log(rng, 2, 64)
        hi = _log(rng, page, 100000 // B)
        return dict(op=op, B=B, page=page, lo=max(1, hi // 16), hi=hi, l_cap=-(-hi // page) * page,
                    Hkv=Hkv, layers=rng.choice([1, 2]), spare=rng.choice([0, 1, 40]), mix=mix)
    if op == "shared":
        N, s_hi = _log(rng, 1, 12), _log(rng, 1, 96)
        p_hi = _log(rng, 1, max(2, min(131072, 3000000 // (N * s_hi), 1500000 // (N * Hkv))))
        fmt = rng.choice(["bf16", "bf16", "int8", "e4m3"])
        own_hi = _log(rng, 1, max(2, min(2048, 600000 // (N * s_hi * Hkv))))
        page = rng.choice([0, page]) if N * s_hi * Hkv * (p_hi + own_hi) < 8000000 else page
        return dict(op=op, N=N, s_lo=max(1, s_hi // rng.choice([1, 4])), s_hi=s_hi,
                    p_lo=p_hi // rng.choice([1, 4, 64]), p_hi=p_hi, o_lo=rng.choice([0, 1]),
                    o_hi=own_hi, Hq=Hq, Hkv=Hkv, page=page, fmt=fmt,
                    block=0 if fmt == "bf16" else
                    rng.choice([x for x in (16, 32, 64, 128) if not page or x <= page]),
                    out=rng.choice(["fp32", "fp32", "bf16"]), mix=mix)
    rot, sections = rng.choice(_SECTIONS)
    c = dict(op=op, Hkv=Hkv, rot=rot, sections=sections, order=rng.choice(["blocks", "turns"]),
             rates=rng.choice(["joint", "joint", "own"]), layout=rng.choice(_LAYOUTS),
             theta=rng.choice([10000.0, 500000.0, 1000000.0]))
    if op == "axes":
        c.update(T=_log(rng, 1, 24000), Hq=Hq, max_pos=rng.choice([32768, 131072, 1048576]),
                 inverse=rng.random() < 0.25)
        return c
    B = _log(rng, 1, 16)
    new = _log(rng, 2, 30000 // B)
    c.update(B=B, new_lo=(new + 1) // 2, new_hi=new, off_hi=rng.choice([0, 3, 20]),
             back=rng.choice([1, (new + 1) // 2]), page=page,
             block=rng.choice([x for x in (16, 32, 64, 128) if x <= page]),
             fmt=rng.choice(["int8", "e4m3"]), mix=mix)
    return c


def _spread(case, n, lo, hi, salt):
    """n whole numbers in [lo, hi], the same for every seed."""
    return [lo + (b * 2654435761 + (case["mix"] + salt) * 40503 * 65537 + salt * 97) % (hi - lo + 1)
            for b in range(n)]


def _groups(case):
    """Sizes and shared lengths of the groups, own rows of every sequence."""
    sizes = _spread(case, case["N"], case["s_lo"], case["s_hi"], 1)
    shared = _spread(case, case["N"], case["p_lo"], case["p_hi"], 2)
    rest = _spread(case, sum(sizes), case["o_lo"], case["o_hi"], 3)
    return sizes, shared, rest


def _sections(case):
    """Pairs of every axis."""
    return [int(n) for n in case["sections"].split(",")]


def _row_bytes(case):
    """A K and a V row of one head with its part of the scales."""
    return 4 * D if case["fmt"] == "bf16" else 2 * D + 8.0 / case["block"]


def work(case):
    op = case["op"]
    if op == "axes":
        rows = case["T"] * (case["Hq"] + case["Hkv"])
        return {"bytes": rows * D * 2 * 2 + case["T"] * 4 * len(_sections(case)),
                "flops": rows * case["rot"] * 3}
    if op == "append":
        toks = sum(_spread(case, case["B"], case["new_lo"], case["new_hi"], 2))
        rows, back = toks * case["Hkv"], case["B"] * case["back"] * case["Hkv"]
        return {"bytes": rows * D * 2 * 3 + back * D * 2 * 3 + toks * 4 * len(_sections(case)),
                "flops": rows * D * 2 * 4 + back * D * 2}
    if op == "step":
        # what changes: a table entry and a count for each page taken or given back
        pages = case["B"] * (case["new"] // case["page"] + 2)
        return {"bytes": pages * 16 + case["B"] * 16, "flops": pages * 2}
    if op == "fork":
        lens = _spread(case, case["N"], case["lo"], case["hi"], 1)
        part = sum(x % case["page"] > 0 for x in lens) * case["C"]
        rows = part * case["page"] * case["Hkv"] * case["layers"]
        entries = sum(-(-x // case["page"]) for x in lens) * (1 + 3 * case["C"])
        back = case["N"] * (1 + case["C"]) * case["back"] * case["Hkv"] * case["layers"] * 6 * D
        return {"bytes": rows * _row_bytes(case) * 2 + entries * 4 + back, "flops": entries}
    if op == "compact":
        lens = _spread(case, case["B"], case["lo"], case["hi"], 1)
        pages = [-(-x // case["page"]) for x in lens]
        live = sum(n for b, n in enumerate(pages) if b % 3)
        total = sum(pages) + case["spare"]
        moves = live * (total - live) // total           # expected of a shuffled pool
        rows = moves * case["page"] * case["Hkv"] * case["layers"]
        return {"bytes": rows * 4 * D * 2 + sum(pages) * 8 + total * 4, "flops": total}
    sizes, shared, rest = _groups(case)
    rows = sum(shared) + sum(rest)
    pairs = sum(s * p for s, p in zip(sizes, shared)) + sum(rest)
    out = 4 if case["out"] == "fp32" else 2
    return {"bytes": rows * case["Hkv"] * _row_bytes(case) +
            sum(sizes) * case["Hq"] * (D * (2 + out) + 4),
            "flops": pairs * case["Hq"] * 4 * D}


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


def _int(x):
    return torch.tensor(x, dtype=torch.int32, device=_DEV)


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


def _pool(case, g, n, rows):
    """K and V of one layer, [n][Hkv][rows][128]: bf16, or codes and scales."""
    H, out = case["Hkv"], {}
    step = max(1, (1 << 27) // (H * rows * D))
    for which in ("k", "v"):
        make = (lambda m: _keys(g, m, H, rows)) if which == "k" else \
            (lambda m: _randn(g, m, H, rows, D))
        if case["fmt"] == "bf16":
            x = torch.empty((n, H, rows, D), dtype=torch.bfloat16, device=_DEV)
            for i in range(0, n, step):
                x[i:i + step] = make(min(step, n - i))
            out[which] = x
            continue
        blk, fmt = case["block"], case["fmt"]
        codes = torch.empty((n, H, rows, D), dtype=torch.uint8, device=_DEV)
        scale = torch.empty((n, H, rows // blk), dtype=torch.float32, device=_DEV)
        for i in range(0, n, step):
            x = make(min(step, n - i)).view(-1, H, rows // blk, blk, D)
            e = _exponent(x.abs().amax(dim=(3, 4)), fmt)
            s = torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)
            codes[i:i + step] = _encode(x / s[..., None, None], fmt).view(-1, H, rows, D)
            scale[i:i + step] = s
        out[which], out[which + "s"] = codes, scale
    return out


def _full_tables(counts, per, n, g):
    """Tables whose row b holds counts[b] pages of a shuffled pool of n."""
    perm = torch.randperm(n, generator=g, device=_DEV).to(torch.int32)
    table = torch.full((len(counts), per), -1, dtype=torch.int32, device=_DEV)
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = perm[at:at + c]
        at += c
    return table


def _count_refs(table, n):
    refs = torch.zeros(n, dtype=torch.int32, device=_DEV)
    used = table[table >= 0].long()
    return refs.index_add_(0, used, torch.ones_like(used, dtype=torch.int32))


def _prepare_pages(case, s, g):
    ps, per = case["page"], case["l_cap"] // case["page"]
    if case["op"] == "fork":
        lens = _spread(case, case["N"], case["lo"], case["hi"], 1)
        B = case["N"] * (1 + case["C"])
        counts = [-(-x // ps) for x in lens] + [0] * (B - case["N"])
        n = sum(counts) + case["N"] * case["C"] + 3
        s["parents"] = _int([i for i in range(case["N"]) for _ in range(case["C"])])
        s["children"] = _int(list(range(case["N"], B)))
        s["take"] = _int([x for x in lens for _ in range(case["C"])])
        s["lens"] = _int(lens + [x for x in lens for _ in range(case["C"])])
    else:
        B = case["B"]
        lens = _spread(case, B, case["lo"], case["hi"], 1)
        s["lens"] = _int(lens)
        if case["op"] == "step":
            had = [max(0, x - case["new"]) for x in lens]
            counts = [-(-x // ps) for x in had]
            n = sum(-(-x // ps) for x in lens) + 3
            s["lo"] = _int(had)
            s["seen_lo"] = torch.full_like(s["lens"], case["n_init"])
            s["seen_hi"] = (s["lens"] - case["n_recent"]).clamp(min=0)
        else:
            counts = [-(-x // ps) for x in lens]
            n = sum(counts) + case["spare"]
            s["zero"] = torch.zeros_like(s["lens"])
            s["leave"] = _int([case["l_cap"] if b % 3 == 0 else 0 for b in range(B)])
    s["n_pages"], s["per"], s["B"] = n, per, B
    table = _full_tables(counts, per, n, g)
    if case["op"] == "step":  # what an earlier step has given back
        j = torch.arange(per, device=_DEV)
        gone = (j * ps >= case["n_init"]) & ((j + 1) * ps <= (s["lo"][:, None] - case["n_recent"]))
        table[gone & (table >= 0)] = -1
    s["table0"], s["refs0"] = table, _count_refs(table, n)
    s["table"], s["refs"] = table.clone(), s["refs0"].clone()
    s["caches"] = [_pool(s, g, n, ps) for _ in range(case.get("layers", 0))]


def _prepare_shared(case, s, g):
    sizes, shared, rest = _groups(case)
    cu, lens, start = [0], [], []
    for n, size in enumerate(sizes):
        cu.append(cu[-1] + size)
        for b in range(cu[-2], cu[-1]):
            lens.append(shared[n] + rest[b])
            start.append(shared[n])
    B, page = cu[-1], case["page"]
    s["B"], s["cu_host"], s["shared_host"], s["lens_host"] = B, cu, shared, lens
    s["start_host"] = start
    s["lens"], s["cu"], s["shared"] = _int(lens), _int(cu), _int(shared)
    s["l_cap"] = -(-max(max(lens), 1) // 256) * 256
    if page:
        # whole pages of the shared rows are the first sequence's, the others have their own
        per = s["l_cap"] // page
        counts = [max(0, -(-lens[b] // page) - (0 if b in cu[:-1] else start[b] // page))
                  for b in range(B)]
        n = sum(counts) + 3
        perm = torch.randperm(n, generator=g, device=_DEV).to(torch.int32).cpu()
        table = torch.full((B, per), -1, dtype=torch.int32)
        at, first = 0, 0
        for b in range(B):
            skip = 0
            if b in cu[:-1]:
                first = b
            else:
                skip = start[b] // page
                table[b, :skip] = table[first, :skip]
            table[b, skip:skip + counts[b]] = perm[at:at + counts[b]]
            at += counts[b]
        s["table"] = table.to(_DEV)
        s["cache"] = _pool(case, g, n, page)
    else:
        s["table"] = None
        s["cache"] = _pool(case, g, B, s["l_cap"])
    q = _randn(g, 1, case["Hq"], D) + 0.3 * _randn(g, B, case["Hq"], D)
    s["q"] = q.bfloat16()


def _axis_positions(g, T, n_axes, start, most):
    """Text tokens count all axes together; every image or frame counts rows and
    columns from where it starts, and the text goes on behind it."""
    i = torch.arange(T, device=_DEV)
    w = int(torch.randint(3, 40, (1,), generator=g, device=_DEV))
    h = int(torch.randint(3, 40, (1,), generator=g, device=_DEV))
    run = 32 + h * w                                  # 32 tokens of text, then a frame
    part, at = i // run, i % run
    base = start + part * (32 + max(h, w))
    pic = at >= 32
    y, x = (at - 32) // w, (at - 32) % w
    text = base + at
    rows = [torch.where(pic, base + 32, text), torch.where(pic, base + 32 + y, text),
            torch.where(pic, base + 32 + x, text), text]
    pos = torch.stack(rows[:n_axes] if n_axes != 2 else rows[1:3])
    return pos.clamp(0, most - 1).to(torch.int32).contiguous()


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(case)
    s.setdefault("fmt", "bf16")
    if op in ("step", "fork", "compact"):
        _prepare_pages(case, s, g)
    elif op == "shared":
        _prepare_shared(case, s, g)
    elif op == "axes":
        T, A = case["T"], len(_sections(case))
        s["q"] = _randn(g, T, case["Hq"], D).bfloat16()
        s["k"] = _keys(g, T, case["Hkv"]).bfloat16()
        if T <= 64:  # a decode step: each token at its own sequence's positions
            s["pos"] = torch.randint(0, case["max_pos"], (A, T), generator=g,
                                     device=_DEV).to(torch.int32)
        else:
            start = int(torch.randint(0, case["max_pos"] // 2, (1,), generator=g, device=_DEV))
            s["pos"] = _axis_positions(g, T, A, start, case["max_pos"])
    else:
        B, ps, blk = case["B"], case["page"], case["block"]
        news = _spread(case, B, case["new_lo"], case["new_hi"], 2)
        offs = [x * blk for x in _spread(case, B, 0, case["off_hi"], 4)]
        lens = [a + b for a, b in zip(news, offs)]
        per = -(-max(lens) // ps)
        s["l_cap"], s["max_pos"], s["news"], s["offs"] = per * ps, per * ps, news, offs
        n = B * per + 3
        s["table"] = _full_tables([per] * B, per, n, g)
        s["cache"] = _pool(case, g, n, ps)
        cu = [0]
        for x in news:
            cu.append(cu[-1] + x)
        s["cu_host"], s["T"], s["max_new"] = cu, cu[-1], max(news)
        s["cu"], s["lens"] = _int(cu), _int(lens)
        s["pos"] = torch.cat([_axis_positions(g, x, len(_sections(case)), o, s["max_pos"])
                              for x, o in zip(news, offs)], dim=1).contiguous()
        s["k_new"] = _keys(g, s["T"], case["Hkv"]).bfloat16()
        s["v_new"] = _randn(g, s["T"], case["Hkv"], D).bfloat16()
    return s


# ------------------------------------------------- plain forms: the pages
def _plain_alloc(s, lo, hi):
    j = torch.arange(s["per"], device=_DEV)
    ps = s["page"]
    need = ((j + 1) * ps > lo[:, None]) & (j * ps < hi[:, None]) & (hi > lo)[:, None]
    need &= s["table"] < 0
    free = (s["refs"] == 0).nonzero().flatten()[: int(need.sum())]
    s["table"][need] = free.to(torch.int32)           # sequence by sequence, lowest pages first
    s["refs"][free] = 1


def _plain_free(s, lo, hi):
    j = torch.arange(s["per"], device=_DEV)
    ps = s["page"]
    gone = (j * ps >= lo[:, None]) & ((j + 1) * ps <= hi[:, None]) & (s["table"] >= 0)
    used = s["table"][gone].long()
    s["refs"].index_add_(0, used, torch.full_like(used, -1, dtype=torch.int32))
    s["table"][gone] = -1


def _plain_fork(s):
    ps, j = s["page"], torch.arange(s["per"], device=_DEV)
    n, par, kid = s["take"].long(), s["parents"].long(), s["children"].long()
    free = (s["refs"] == 0).nonzero().flatten()
    rows = s["table"][par]
    full, part = n // ps, n % ps > 0
    row = torch.where(j < full[:, None], rows, torch.full_like(rows, -1))
    src = torch.full_like(s["take"], -1)
    dst = src.clone()
    src[part] = rows[part, full[part]]
    dst[part] = free[: int(part.sum())].to(torch.int32)
    row[part, full[part]] = dst[part]
    used = row[row >= 0].long()
    s["refs"].index_add_(0, used, torch.ones_like(used, dtype=torch.int32))
    s["table"][kid] = row
    return src, dst


def _plain_compact(s):
    refs, n = s["refs"], s["n_pages"]
    live = int((refs > 0).sum())
    holes = (refs[:live] == 0).nonzero().flatten()
    high = (refs[live:] > 0).nonzero().flatten() + live
    m = len(holes)
    src = torch.full((n // 2,), -1, dtype=torch.int32, device=_DEV)
    dst = src.clone()
    src[:m], dst[:m] = high.to(torch.int32), holes.to(torch.int32)
    to = torch.arange(n, device=_DEV, dtype=torch.int32)
    to[high] = holes.to(torch.int32)
    s["table"].copy_(torch.where(s["table"] >= 0, to[s["table"].clamp(min=0).long()], s["table"]))
    refs[holes] = refs[high]
    refs[high] = 0
    return src, dst, torch.tensor([m], dtype=torch.int32, device=_DEV)


def _plain_copy(s, src, dst):
    on = src >= 0
    a, b = src[on].long(), dst[on].long()
    for c in s["caches"]:
        for x in c.values():
            x[b] = x[a]


def _read_back(s, c):
    """The last `back` rows of every sequence of one layer, values."""
    pos = s["lens"].long()[:, None] - s["back"] + torch.arange(s["back"], device=_DEV)
    page = s["table"].gather(1, pos // s["page"]).long()
    out = []
    for which in ("k", "v"):
        x = _decode(c[which][page, :, pos % s["page"]], s["fmt"])       # [B, back, H, D]
        x = x * c[which + "s"][page, :, pos % s["page"] // s["block"]][..., None]
        out.append(x.reshape(-1, s["Hkv"], D).bfloat16())
    return out


def _pages_back(s):
    s["table"].copy_(s["table0"])
    s["refs"].copy_(s["refs0"])


def _plain_pages(s):
    _pages_back(s)
    out = [s["table"], s["refs"]]
    if s["op"] == "step":
        _plain_alloc(s, s["lo"], s["lens"])
        _plain_free(s, s["seen_lo"], s["seen_hi"])
        return out
    if s["op"] == "compact":
        _plain_free(s, s["zero"], s["leave"])
        moves = _plain_compact(s)
    else:
        moves = _plain_fork(s)
    _plain_copy(s, *moves[:2])
    out += moves
    for c in s["caches"]:
        out += _read_back(s, c) + [c["ks"], c["vs"]] if "ks" in c else [c["k"], c["v"]]
    return out


# ----------------------------------------------- plain forms: shared rows
def _at(s, pos, seq):
    """Pool index and row in it of positions pos (any shape) of sequences seq."""
    if s["table"] is None:
        return seq.expand_as(pos), pos
    return s["table"][seq, pos // s["page"]].long(), pos % s["page"]


def _values(s, which, entry, row):
    """fp32 rows [..., Hkv, D]."""
    c = s["cache"]
    x = c[which][entry, :, row]
    if s["fmt"] == "bf16":
        return x.float()
    return _decode(x, s["fmt"]) * c[which + "s"][entry, :, row // s["block"]][..., None]


def _soft(z, v):
    """Maximum, sum and sums of values of e^z, z [..., R, W], v [..., W, D]."""
    m = z.amax(dim=-1, keepdim=True)
    z.sub_(torch.where(m.isinf(), torch.zeros_like(m), m)).exp_()
    return m, z.sum(dim=-1, keepdim=True), torch.matmul(z, v)


def _plain_shared(s):
    B, Hq, H = s["B"], s["Hq"], s["Hkv"]
    G, scale = Hq // H, 1.0 / math.sqrt(D)
    q = s["q"].float().view(B, H, G, D)
    cu = s["cu_host"]
    m1 = torch.full((B, H, G, 1), -math.inf, device=_DEV)
    l1, o1 = torch.zeros_like(m1), torch.zeros((B, H, G, D), device=_DEV)
    for n, P in enumerate(s["shared_host"]):
        b0, b1 = cu[n], cu[n + 1]
        if P == 0 or b0 == b1:
            continue
        pos = torch.arange(P, device=_DEV)
        at = _at(s, pos, torch.full_like(pos, b0))
        k, v = (_values(s, w, *at).transpose(0, 1) for w in ("k", "v"))      # [H, P, D]
        x = q[b0:b1].permute(1, 0, 2, 3).reshape(H, (b1 - b0) * G, D)
        m, l, o = _soft(torch.matmul(x, k.transpose(-1, -2)) * scale, v)
        for t, u in ((m1, m), (l1, l), (o1, o)):
            t[b0:b1] = u.view(H, b1 - b0, G, -1).transpose(0, 1)
    start = _kept(s, "start", lambda: torch.tensor(s["start_host"], device=_DEV))
    W = max(1, max(a - b for a, b in zip(s["lens_host"], s["start_host"])))
    pos = start[:, None] + torch.arange(W, device=_DEV)
    ok = pos < s["lens"].long()[:, None]
    pos = torch.where(ok, pos, torch.zeros_like(pos))
    at = _at(s, pos, torch.arange(B, device=_DEV)[:, None])
    if s["table"] is not None:
        at = at[0].clamp(min=0), at[1]
    k, v = (_values(s, w, *at).transpose(1, 2) for w in ("k", "v"))          # [B, H, W, D]
    z = torch.matmul(q, k.transpose(-1, -2)) * scale
    z.masked_fill_(~ok[:, None, None], -math.inf)
    m2, l2, o2 = _soft(z, v)
    m = torch.maximum(m1, m2)
    c = torch.where(m.isinf(), torch.zeros_like(m), m)
    f1, f2 = (m1 - c).exp(), (m2 - c).exp()
    l = l1 * f1 + l2 * f2
    out = (o1 * f1 + o2 * f2) / torch.where(l > 0, l, torch.ones_like(l))
    out = out.reshape(B, Hq, D)
    return [out if s["out"] == "fp32" else out.bfloat16(), (m + l.log()).reshape(B, Hq)]


# ---------------------------------------------- plain forms: several axes
def _axis_of(c):
    """Axis of every pair: in blocks, or dealt by turns to the axes not yet full."""
    if c["order"] == "blocks":
        return [a for a, n in enumerate(_sections(c)) for _ in range(n)]
    left, out = _sections(c), []
    while any(left):
        for a in range(len(left)):
            if left[a]:
                left[a] -= 1
                out.append(a)
    return out


def _freqs(c):
    """Rotation rates in 64 bits, [rot/2]: of the pair's number among all pairs, or among
    its axis' own."""
    axis, seen, e = _axis_of(c), [0] * len(_sections(c)), []
    for i, a in enumerate(axis):
        e.append(-2.0 * i / c["rot"] if c["rates"] == "joint" else -seen[a] / _sections(c)[a])
        seen[a] += 1
    return c["theta"] ** torch.tensor(e, dtype=torch.float64, device=_DEV)


def _angles(c, pos):
    return pos.double()[torch.tensor(_axis_of(c), device=_DEV)].T * _freqs(c)


def _rotate(x, pos, c, inverse=False):
    """x fp32 [T, H, D] rotated; pos [axes, T]."""
    rot = c["rot"]
    ang = _angles(c, pos)
    cos, sin = ang.cos().float()[:, None], ang.sin().float()[:, None]
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


def _plain_append(s):
    """The new rows start at a block's start, so that a block's rows are all new."""
    blk, fmt, H = s["block"], s["fmt"], s["Hkv"]
    nb = -(-s["max_new"] // blk)
    cu = s["cu"].long()
    n = cu[1:] - cu[:-1]
    start = s["lens"].long() - n
    j = torch.arange(nb * blk, device=_DEV).view(1, nb, blk)
    new = j < n[:, None, None]
    tok = (cu[:-1, None, None] + j).clamp(max=s["T"] - 1)
    pos = (start[:, None, None] + j).clamp(max=s["l_cap"] - 1)
    page = s["table"].long().gather(1, (pos // s["page"]).flatten(1)).view_as(pos)
    row, c = pos % s["page"], s["cache"]
    some = new[:, :, 0]
    for which, x in (("k", _rotate(s["k_new"].float(), s["pos"], s)), ("v", s["v_new"].float())):
        x = torch.where(new[..., None, None], x[tok], torch.zeros((), device=_DEV))
        e = _exponent(x.abs().amax(dim=(2, 4)), fmt)                         # [B, nb, H]
        sc = torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)
        code = _encode(x / sc[:, :, None, :, None], fmt)
        c[which][page[new], :, row[new]] = code[new]
        c[which + "s"][page[..., 0][some], :, row[..., 0][some] // blk] = sc[some]
    return _read_back(s, c) + [c["ks"], c["vs"]]


# ------------------------------------------------------- the library's own
def _kept(s, key, make):
    """What a program makes once and keeps beside its buffers."""
    if key not in s:
        s[key] = make()
    return s[key]


def _cache(tsa, s, c, table):
    if s["fmt"] == "bf16":
        return tsa.KV(c["k"], c["v"], table, s["page"])
    return tsa.KV8(c["k"], c["v"], c["ks"], c["vs"], fmt=s["fmt"], page_table=table)


def _own_pages(tsa, s):
    pages = _kept(s, "pages", lambda: tsa.Pages(s["table"], s["refs"], s["page"]))
    caches = _kept(s, "own_caches", lambda: [_cache(tsa, s, c, s["table"]) for c in s["caches"]])
    _pages_back(s)
    out = [s["table"], s["refs"]]
    if s["op"] == "step":
        tsa.pages_alloc(pages, s["lo"], s["lens"])
        tsa.pages_free(pages, s["seen_lo"], s["seen_hi"])
        return out
    if s["op"] == "compact":
        tsa.pages_free(pages, s["zero"], s["leave"])
        moves = tsa.pages_compact(pages)
        tsa.pages_copy(caches, *moves)
    else:
        moves = tsa.pages_fork(pages, s["parents"], s["children"], s["take"])
        tsa.pages_copy(caches, *moves)
    out += moves
    for cache, c in zip(caches, s["caches"]):
        if "ks" in c:
            out += [*tsa.kv8_read(cache, s["lens"], s["back"]), c["ks"], c["vs"]]
        else:
            out += [c["k"], c["v"]]
    return out


def _own_run(s):
    import top_retrieval_sparse_gb300 as tsa
    if s["op"] in ("step", "fork", "compact"):
        return _own_pages(tsa, s)
    if s["op"] == "shared":
        cache = _kept(s, "own_cache", lambda: _cache(tsa, s, s["cache"], s["table"]))
        ws = _kept(s, "ws", lambda: tsa.shared_attn_decode_workspace(
            s["B"], s["N"], s["Hq"], s["Hkv"], device=_DEV))
        lse = _kept(s, "lse", lambda: torch.empty((s["B"], s["Hq"]), dtype=torch.float32,
                                                  device=_DEV))
        out = torch.empty_like(s["q"], dtype=torch.float32 if s["out"] == "fp32" else
                               torch.bfloat16)
        return tsa.shared_attn_decode(s["q"], cache, s["lens"], s["cu"], s["shared"], out=out,
                                      lse_out=lse, workspace=ws)
    table = _kept(s, "rope", lambda: tsa.RopeTable(
        s["rot"], s["max_pos"], theta=s["theta"], layout=s["layout"], sections=_sections(s),
        order=s["order"], rates=s["rates"], device=_DEV))
    if s["op"] == "axes":
        return tsa.rope(s["q"], s["pos"], table, k=s["k"], inverse=s["inverse"])
    cache = _kept(s, "own_cache", lambda: _cache(tsa, s, s["cache"], s["table"]))
    tsa.kv8_append(cache, s["k_new"], s["v_new"], s["lens"], cu_new=s["cu"],
                   max_new=s["max_new"], rope=table, positions=s["pos"])
    return [*tsa.kv8_read(cache, s["lens"], s["back"]), s["cache"]["ks"], s["cache"]["vs"]]


def run(state):
    if own:
        return list(_own_run(state))
    op = state["op"]
    if op in ("step", "fork", "compact"):
        return _plain_pages(state)
    if op == "shared":
        return _plain_shared(state)
    if op == "axes":
        return [_rotate(state[x].float(), state["pos"], state, state["inverse"]).bfloat16()
                for x in ("q", "k")]
    return _plain_append(state)


# ------------------------------------------------------------------ exact
def _exact_pages(s):
    """Lists and loops on the host; the moved pages one after another."""
    table, refs, ps = s["table0"].tolist(), s["refs0"].tolist(), s["page"]

    def release(b, lo, hi):
        for j, page in enumerate(table[b]):
            if page >= 0 and j * ps >= lo and (j + 1) * ps <= hi:
                refs[page] -= 1
                table[b][j] = -1

    src, dst, count = [], [], None
    lens = s["lens"].tolist()
    if s["op"] == "step":
        free = iter([p for p, r in enumerate(refs) if r == 0])
        for b, had in enumerate(s["lo"].tolist()):
            for j in range(had // ps, -(-lens[b] // ps)):
                if table[b][j] < 0:
                    table[b][j] = page = next(free)
                    refs[page] = 1
        for b, (lo, hi) in enumerate(zip(s["seen_lo"].tolist(), s["seen_hi"].tolist())):
            release(b, lo, hi)
    elif s["op"] == "fork":
        free = iter([p for p, r in enumerate(refs) if r == 0])
        for p, c, n in zip(s["parents"].tolist(), s["children"].tolist(), s["take"].tolist()):
            for j in range(n // ps):
                table[c][j] = table[p][j]
                refs[table[p][j]] += 1
            if n % ps:
                table[c][n // ps] = page = next(free)
                refs[page] = 1
            src.append(table[p][n // ps] if n % ps else -1)
            dst.append(page if n % ps else -1)
    else:
        for b, hi in enumerate(s["leave"].tolist()):
            release(b, 0, hi)
        left = sum(r > 0 for r in refs)
        move, hole = {}, 0
        for page in range(left, len(refs)):
            if refs[page] > 0:
                while refs[hole] > 0:
                    hole += 1
                move[page] = hole
                refs[hole], refs[page] = refs[page], 0
        table = [[move.get(p, p) for p in row] for row in table]
        pad = [-1] * (len(refs) // 2 - len(move))
        src, dst, count = list(move) + pad, list(move.values()) + pad, [len(move)]
    out = [_int(table), _int(refs)]
    if s["op"] == "step":
        return out
    out += [_int(src), _int(dst)] + ([_int(count)] if count else [])
    for c in s["caches"]:
        for x in c.values():
            for a, b in zip(src, dst):
                if a >= 0:
                    x[b].copy_(x[a])
        if "ks" not in c:
            out += [c["k"], c["v"]]
            continue
        got = []
        for which in ("k", "v"):
            val = _decode(c[which], s["fmt"]).double().unflatten(2, (-1, s["block"]))
            val = (val * c[which + "s"].double()[..., None, None]).flatten(2, 3)
            got.append(torch.stack([val[table[b][p // ps], :, p % ps]
                                    for b in range(s["B"])
                                    for p in range(lens[b] - s["back"], lens[b])]))
        out += got + [c["ks"], c["vs"]]
    return out


def _exact_shared(s):
    """Every sequence by itself over all its rows."""
    B, Hq, H = s["B"], s["Hq"], s["Hkv"]
    G = Hq // H
    out = torch.zeros((B, Hq, D), dtype=torch.float64, device=_DEV)
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device=_DEV)
    cu = s["cu_host"]
    for n, P in enumerate(s["shared_host"]):
        for b in range(cu[n], cu[n + 1]):
            L = s["lens_host"][b]
            if L == 0:
                continue
            pos = torch.arange(L, device=_DEV)
            owner = torch.where(pos < P, cu[n], b)
            if s["table"] is None:
                entry, row = owner, pos
            else:
                entry, row = s["table"][owner, pos // s["page"]].long(), pos % s["page"]
            for h in range(H):
                k, v = s["cache"]["k"][entry, h, row], s["cache"]["v"][entry, h, row]
                if s["fmt"] != "bf16":
                    at = row // s["block"]
                    k = _decode(k, s["fmt"]).double() * s["cache"]["ks"][entry, h, at][:, None]
                    v = _decode(v, s["fmt"]).double() * s["cache"]["vs"][entry, h, at][:, None]
                x = s["q"][b, h * G:(h + 1) * G].double()
                z = x @ k.double().T / math.sqrt(D)
                top = torch.logsumexp(z, dim=-1)
                out[b, h * G:(h + 1) * G] = torch.exp(z - top[:, None]) @ v.double()
                lse[b, h * G:(h + 1) * G] = top
    return [out, lse]


def _turn64(x, pos, c, inverse=False):
    """The rotation as a product of complex numbers, 64 bits."""
    rot = c["rot"]
    ang = _angles(c, pos)
    unit = torch.polar(torch.ones_like(ang), -ang if inverse else ang)[:, None]
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


def _exact_append(s):
    top, blk = (127.0 if s["fmt"] == "int8" else 448.0), s["block"]
    cu, got, scales = s["cu_host"], [], []
    for which in ("k", "v"):
        x = s[which + "_new"].double()
        if which == "k":
            x = _turn64(x, s["pos"], s)
        sc = s["cache"][which + "s"].double().clone()
        rows = []
        for b, (new, off) in enumerate(zip(s["news"], s["offs"])):
            vals = []
            for i in range(0, new, blk):
                part = x[cu[b] + i: min(cu[b] + i + blk, cu[b + 1])]          # [n, H, D]
                amax = part.abs().amax(dim=(0, 2))
                # the logarithm of a power of two may come out a hair above it
                e = torch.ceil(torch.log2(amax.clamp(min=1e-300) / top) - 1e-10)
                unit = torch.exp2(e.clamp(min=_MIN_EXP))
                page = int(s["table"][b, (off + i) // s["page"]])
                sc[page, :, (off + i) % s["page"] // blk] = unit
                vals.append(_step64(part / unit[:, None], s["fmt"]) * unit[:, None])
            rows.append(torch.cat(vals)[new - s["back"]:])
        got.append(torch.cat(rows))
        scales.append(sc)
    return got + scales


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("step", "fork", "compact"):
        return _exact_pages(s)
    if case["op"] == "shared":
        return _exact_shared(s)
    if case["op"] == "axes":
        return [_turn64(s[x].double(), s["pos"], s, s["inverse"]) for x in ("q", "k")]
    return _exact_append(s)
