"""The step over shared rows where a share of the work has units of a single key tile, which one
of the kernel's two streams passes by, in front of longer ones: against 64-bit attention of every
sequence by itself.  What such lists do to the rings is modelled in test_shared_ring_host.py."""
import pytest
import torch

from test_parity_cache_ops import D, DEV, gen, i32, randn, values
from test_parity_shared_attn import check, members, roomy
from test_shared_ring_host import SHORT_BEFORE_LONG

pytestmark = pytest.mark.gpu
PS = 64


@pytest.fixture(scope="module")
def tsa():
    import top_retrieval_sparse_gb300 as t
    t.lib()
    return t


def pool_of(g, cu, shared, lens, Hkv, row_bytes):
    """A page table that names the first sequences' pages and the others' own rows' alone, for a
    cache past the size at which shared rows are read for every sequence; every page's keys and
    values.  A column of the values stands out in every key tile, another one in the next, so
    that a tile taken for another shows."""
    B = len(lens)
    cap = roomy(B, Hkv, -(-max(lens) // PS) * PS, PS, row_bytes)
    want = []                                        # (sequence, entry)
    for b, (n, first) in enumerate(members(B, cu)):
        begin = 0 if b == first or n < 0 else shared[n]
        want += [(b, j) for j in range(begin // PS, -(-lens[b] // PS))]
    n_pages = len(want) + 3
    ids = torch.randperm(n_pages, generator=g, device=DEV)[: len(want)].int()
    at = torch.tensor(want, device=DEV)
    table = torch.full((B, cap // PS), -1, dtype=torch.int32, device=DEV)
    table[at[:, 0], at[:, 1]] = ids
    k, v = (randn(g, n_pages, Hkv, PS, D) for _ in range(2))
    v[ids.long(), :, :, (at[:, 1] * PS // 128 + 5 * at[:, 0]) % D] += 16.0
    return table, k.bfloat16(), v.bfloat16()


@pytest.mark.parametrize("fmt", ["bf16", "int8", "e4m3"])
@pytest.mark.parametrize("name", SHORT_BEFORE_LONG)
def test_short_units_before_long_ones(tsa, name, fmt):
    sizes, shared, G, Hkv = SHORT_BEFORE_LONG[name]
    cu = [sum(sizes[:i]) for i in range(len(sizes) + 1)]
    lens = [shared[n] + b % 4 for n, s in enumerate(sizes) for b in range(s)]
    B, Hq = len(lens), G * Hkv
    g = gen(len(name))
    table, k, v = pool_of(g, cu, shared, lens, Hkv, 512 if fmt == "bf16" else 256)
    if fmt == "bf16":
        cache, steps = tsa.kv_paged(k, v, table), None
        pool = (k, v)
    else:
        n = k.shape[0]
        cache = tsa.KV8.paged(n, Hkv, PS, table, 32, fmt)
        for i in range(0, n, 4096):                  # every page a sequence of its own
            j = min(n, i + 4096)
            one = tsa.KV8(cache.k, cache.v, cache.k_scale, cache.v_scale, fmt,
                          torch.arange(i, j, device=DEV).int().view(-1, 1))
            tsa.kv8_append(one, *(x[i:j].transpose(1, 2).reshape(-1, Hkv, D) for x in (k, v)),
                           i32([PS] * (j - i)))
        pool = values(cache)

        def steps(b, h):
            s = cache.v_scale[table[b].long().clamp(min=0), h].reshape(-1)
            return s.double().repeat_interleave(32)

    def rows(b, h):
        used = table[b, : -(-lens[b] // PS)].long().clamp(min=0)
        return tuple(x[used, h].reshape(-1, D) for x in pool)

    q = randn(g, B, Hq, D).bfloat16()
    ws = tsa.shared_attn_decode_workspace(B, len(shared), Hq, Hkv)
    args = (q, cache, i32(lens), i32(cu), i32(shared))
    for dtype in (torch.float32, torch.bfloat16):
        out = torch.empty((B, Hq, D), dtype=dtype, device=DEV)
        lse = torch.empty((B, Hq), device=DEV)
        tsa.shared_attn_decode(*args, out=out, lse_out=lse, workspace=ws)
        assert tsa.workspace_status(ws) == 0
        check(q, rows, lens, cu, shared, Hkv, out, lse, steps=steps)
        for _ in range(3):                           # the same however the roles run
            again = torch.empty_like(out)
            tsa.shared_attn_decode(*args, out=again, workspace=ws)
            assert torch.equal(out, again)
    assert tsa.workspace_status(ws) == 0


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
def test_many_short_units_and_a_long_one_in_random_order(tsa, fmt):
    """Groups of 1 to 300 shared rows around long ones, against the decode step of every sequence
    by itself over its own table."""
    rng = __import__("random").Random(7)
    g = gen(30)
    Hq, Hkv = 16, 4
    for turn in range(6):
        shared = [rng.randint(1, 128) for _ in range(rng.choice([5, 30, 60]))]
        for _ in range(3):
            shared.insert(rng.randrange(len(shared) + 1), rng.choice([250, 6000, 20000]))
        sizes = [rng.choice([1, 2, 5]) for _ in shared]
        cu = [sum(sizes[:i]) for i in range(len(sizes) + 1)]
        lens = [shared[n] + b % 3 for n, s in enumerate(sizes) for b in range(s)]
        B = len(lens)
        table, k, v = pool_of(g, cu, shared, lens, Hkv, 512 if fmt == "bf16" else 256)
        whole = table.clone()                        # what every sequence reads by itself
        for b, (n, first) in enumerate(members(B, cu)):
            j = shared[n] // PS
            whole[b, :j] = table[first, :j]
            if b != first and shared[n] % PS and lens[b] > shared[n]:
                a, z = table[first, j].long(), table[b, j].long()
                k[z, :, : shared[n] % PS], v[z, :, : shared[n] % PS] = (
                    x[a, :, : shared[n] % PS] for x in (k, v))
            elif shared[n] % PS:
                whole[b, j] = table[first, j]
        if fmt == "bf16":
            cache, plain = tsa.kv_paged(k, v, table), tsa.kv_paged(k, v, whole)
        else:
            # one scale, so that a block of shared and own rows has the first sequence's too
            cache = tsa.KV8.paged(k.shape[0], Hkv, PS, table, 64, fmt)
            for x, scale, codes in ((k, cache.k_scale, cache.k), (v, cache.v_scale, cache.v)):
                scale.fill_(2.0 ** -2)
                codes.copy_((x.float() * 4).round().clamp(-127, 127) + 128)
            plain = tsa.KV8(cache.k, cache.v, cache.k_scale, cache.v_scale, fmt, whole)
        q = randn(g, B, Hq, D).bfloat16()
        lse, lse1 = (torch.empty((B, Hq), device=DEV) for _ in range(2))
        ws = tsa.shared_attn_decode_workspace(B, len(shared), Hq, Hkv)
        out, _ = tsa.shared_attn_decode(q, cache, i32(lens), i32(cu), i32(shared), lse_out=lse,
                                        workspace=ws)
        step = tsa.window_attn_decode if fmt == "bf16" else tsa.kv8_attn_decode
        want, _ = step(q, plain, i32(lens), 0, None, lse_out=lse1)
        assert tsa.workspace_status(ws) == 0
        # each within 2 (20 2^-19 + 2^-17 + 2^-20 + 2e4 2^-27) of 64 bits where logits' terms add
        # up to 20, relative to values of at most 22 and sums of weights: 4e-4
        assert ((lse - lse1).abs() <= 8e-4).all(), turn
        assert ((out - want).abs() <= 8e-4 * 22).all(), turn


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_many_calls_over_codes_in_the_second_level_cache(tsa, fmt):
    """Codes that are copied as fast as their slots are given back: hundreds of calls give what
    the first gave, and that is right."""
    rng = __import__("random").Random(8)
    g = gen(31)
    for G, Hkv in ((5, 2), (7, 4), (8, 8)):
        shared = [rng.choice([rng.randint(1, 128), rng.randint(129, 3000), rng.randint(300, 9000)])
                  for _ in range(40)]
        sizes = [rng.choice([1, 2, 5, 16]) for _ in shared]
        cu = [sum(sizes[:i]) for i in range(len(sizes) + 1)]
        lens = [shared[n] + b % 4 for n, s in enumerate(sizes) for b in range(s)]
        B, Hq = len(lens), G * Hkv
        table, k, v = pool_of(g, cu, shared, lens, Hkv, 256)
        cache = tsa.KV8.paged(k.shape[0], Hkv, PS, table, 64, fmt)
        for x, scale, codes in ((k, cache.k_scale, cache.k), (v, cache.v_scale, cache.v)):
            scale.fill_(2.0 ** -2)
            codes.copy_((x.float() * 4).round().clamp(-127, 127) + 128 if fmt == "int8" else
                        (x.float() * 4).to(torch.float8_e4m3fn).view(torch.uint8))
        pool = values(cache)

        def rows(b, h):
            used = table[b, : -(-lens[b] // PS)].long().clamp(min=0)
            return tuple(x[used, h].reshape(-1, D) for x in pool)

        def steps(b, h):
            return torch.full((-(-lens[b] // PS) * PS,), 0.25, dtype=torch.float64, device=DEV)

        q = randn(g, B, Hq, D).bfloat16()
        lse = torch.empty((B, Hq), device=DEV)
        ws = tsa.shared_attn_decode_workspace(B, len(shared), Hq, Hkv)
        args = (q, cache, i32(lens), i32(cu), i32(shared))
        for dtype in (torch.bfloat16, torch.float32):
            out, again = (torch.empty((B, Hq, D), dtype=dtype, device=DEV) for _ in range(2))
            tsa.shared_attn_decode(*args, out=out, lse_out=lse, workspace=ws)
            check(q, rows, lens, cu, shared, Hkv, out, lse, steps=steps,
                  only=[b for b in range(B) if b % 5 == 0])
            wrong = torch.zeros((), dtype=torch.int64, device=DEV)
            for _ in range(250):
                tsa.shared_attn_decode(*args, out=again, workspace=ws)
                wrong += (again != out).any()
            assert int(wrong) == 0
        assert tsa.workspace_status(ws) == 0
