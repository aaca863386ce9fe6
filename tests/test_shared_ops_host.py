"""Refusals and sizes of the operators of shared caches (pages, rotation by several axes, the
step over shared rows): nothing here launches, so no GPU is needed."""
import ctypes as C

import pytest
import torch

from test_cache_ops_host import FAKE, _cache, _refused, _spec


@pytest.fixture(scope="module")
def tsa():
    import top_retrieval_sparse_gb300 as t
    t.lib()
    return t


# ------------------------------------------------------------------ pages
def _pages(tsa, **kw):
    a = dict(table=FAKE, refs=FAKE * 2, B=4, max_pages=32, n_pages=100, page_size=16)
    a.update(kw)
    return C.byref(tsa._PagesStruct(**a))


def _call(tsa, name, pages, **kw):
    a = dict(lo=FAKE, hi=FAKE, parents=FAKE, children=FAKE, lens=FAKE, n=3, src=FAKE, dst=FAKE,
             count=FAKE, ws=FAKE * 9, wb=1 << 40)
    a.update(kw)
    keys = {"pages_alloc": "lo hi", "pages_free": "lo hi",
            "pages_fork": "parents children lens n src dst", "pages_compact": "src dst count"}[name]
    return getattr(tsa.lib(), name)(pages, *(a[k] for k in keys.split()), a["ws"], a["wb"], None)


ALL = ["pages_alloc", "pages_free", "pages_fork", "pages_compact"]


@pytest.mark.parametrize("name", ALL)
def test_page_states_that_are_refused(tsa, name):
    for kw in (dict(table=None), dict(refs=None), dict(table=FAKE + 2), dict(B=-1), dict(B=4097),
               dict(max_pages=0), dict(n_pages=0), dict(n_pages=(1 << 23) + 1), dict(page_size=8),
               dict(page_size=48), dict(page_size=512), dict(B=4096, max_pages=1 << 19),
               dict(page_size=256, max_pages=1 << 23)):
        _refused(tsa, _call(tsa, name, _pages(tsa, **kw)))
    _refused(tsa, _call(tsa, name, None))
    need = tsa.lib().tsa_pages_workspace_size(4, 32, 100)
    assert need > 0 and need % 256 == 0
    for kw in (dict(ws=None), dict(ws=FAKE + 64), dict(wb=need - 1)):
        _refused(tsa, _call(tsa, name, _pages(tsa), **kw), -2)


@pytest.mark.parametrize("name,kw", [
    ("pages_alloc", dict(lo=None)), ("pages_alloc", dict(hi=None)), ("pages_free", dict(lo=None)),
    ("pages_free", dict(hi=None)), ("pages_fork", dict(parents=None)),
    ("pages_fork", dict(children=None)), ("pages_fork", dict(lens=None)),
    ("pages_fork", dict(src=None)), ("pages_fork", dict(dst=None)), ("pages_fork", dict(n=-1)),
    ("pages_fork", dict(n=5)), ("pages_compact", dict(src=None)), ("pages_compact", dict(dst=None)),
    ("pages_compact", dict(count=None))])
def test_page_calls_that_are_refused(tsa, name, kw):
    _refused(tsa, _call(tsa, name, _pages(tsa), **kw))


def test_page_calls_with_nothing_to_do(tsa):
    for name in ALL[:2]:
        assert _call(tsa, name, _pages(tsa, B=0), lo=None, hi=None) == 0
    assert _call(tsa, "pages_fork", _pages(tsa), n=0, parents=None, src=None) == 0
    assert tsa.lib().tsa_pages_workspace_size(1, 0, 5) == 0
    assert tsa.lib().tsa_pages_workspace_size(4097, 1, 5) == 0


def _copy(tsa, bufs=((FAKE, 4096),), **kw):
    a = dict(n_pages=10, src=FAKE, dst=FAKE, count=None, n=3, status=None)
    a.update(kw)
    arr = (tsa._PageBuf * max(1, len(bufs)))(*bufs)
    return tsa.lib().pages_copy(arr, len(bufs), a["n_pages"], a["src"], a["dst"], a["count"],
                                a["n"], a["status"], None)


def test_copies_that_are_refused(tsa):
    for bufs in (((None, 4096),), ((FAKE + 2, 4096),), ((FAKE, 0),), ((FAKE, -4),), ((FAKE, 6),),
                 ((FAKE, (1 << 32) + 4),), ((FAKE, 64), (FAKE, 2))):
        _refused(tsa, _copy(tsa, bufs))
    for kw in (dict(n_pages=0), dict(src=None), dict(dst=None), dict(n=-1), dict(status=FAKE + 8)):
        _refused(tsa, _copy(tsa, **kw))
    _refused(tsa, tsa.lib().pages_copy(None, 1, 10, FAKE, FAKE, None, 3, None, None))
    assert _copy(tsa, n=0, src=None) == 0 and _copy(tsa, ()) == 0


# ---------------------------------------------------- several axes
def _axes(tsa, n=3, order=0, rates=0, pairs=(16, 24, 24, 0)):
    return tsa._RopeAxes(n, order, rates, (C.c_int32 * 4)(*pairs))


BAD_AXES = [dict(n=0), dict(n=5), dict(order=2), dict(order=-1), dict(rates=2), dict(n=2),
            dict(pairs=(16, 24, 23, 0)), dict(pairs=(40, 24, 0, 0)), dict(pairs=(-16, 40, 40, 0)),
            dict(pairs=(1 << 30, 1 << 30, 64, 0))]


@pytest.mark.parametrize("kw", BAD_AXES)
def test_axes_that_are_refused(tsa, kw):
    L, r = tsa.lib(), tsa._RopeStruct()
    x = C.byref(_axes(tsa, **kw))
    _refused(tsa, L.tsa_rope_table_axes(C.byref(_spec(tsa)), x, FAKE, 1 << 40, C.byref(r), None))
    rows = C.byref(tsa._RowsStruct(FAKE, 4096, 128))
    rope = C.byref(tsa._RopeStruct(FAKE, 4096, 128, 0))
    _refused(tsa, L.rope_apply_axes(rows, rows, 4, None, None, 0, 7, 128, FAKE, 7, rope, x, 0, None))
    _refused(tsa, L.kv8_append_axes(C.byref(_cache(tsa)), rows, rows, None, 10, 5, FAKE, 2, 2, 128,
                                    rope, x, FAKE, 10, None))


def test_calls_with_axes_that_are_refused(tsa):
    L, r = tsa.lib(), tsa._RopeStruct()
    x, spec = C.byref(_axes(tsa)), C.byref(_spec(tsa))
    rows = C.byref(tsa._RowsStruct(FAKE, 4096, 128))
    rope = C.byref(tsa._RopeStruct(FAKE, 4096, 128, 0))
    _refused(tsa, L.tsa_rope_table_axes(spec, None, FAKE, 1 << 40, C.byref(r), None))
    _refused(tsa, L.tsa_rope_table_axes(None, x, FAKE, 1 << 40, C.byref(r), None))
    _refused(tsa, L.tsa_rope_table_axes(spec, x, FAKE, 1 << 40, None, None))
    _refused(tsa, L.tsa_rope_table_axes(C.byref(_spec(tsa, rot_dim=24)), x, FAKE, 1 << 40,
                                        C.byref(r), None))
    ntk = C.byref(_spec(tsa, scaling=2, factor=2.0))
    one = C.byref(_axes(tsa, 2, 0, 1, (1, 63, 0, 0)))
    _refused(tsa, L.tsa_rope_table_axes(ntk, one, FAKE, 1 << 40, C.byref(r), None))
    apply = lambda rope=rope, x=x, pos=FAKE, stride=7: L.rope_apply_axes(  # noqa: E731
        rows, rows, 4, None, None, 0, 7, 128, pos, stride, rope, x, 0, None)
    for kw in (dict(rope=None), dict(x=None), dict(pos=None), dict(stride=-1),
               dict(stride=1 << 40)):
        _refused(tsa, apply(**kw))
    append = lambda rope=rope, x=x, pos=FAKE, stride=10: L.kv8_append_axes(  # noqa: E731
        C.byref(_cache(tsa)), rows, rows, None, 10, 5, FAKE, 2, 2, 128, rope, x, pos, stride, None)
    for kw in (dict(rope=None), dict(x=None), dict(pos=None), dict(stride=-1)):
        _refused(tsa, append(**kw))


def test_what_the_binding_refuses_about_axes(tsa):
    for kw in (dict(sections=()), dict(sections=(10,) * 5), dict(order="rows"),
               dict(rates="all"), dict(sections=(-1, 65)), dict(sections=(1 << 31, 3))):
        with pytest.raises(ValueError):
            tsa.RopeTable(128, 10, **{"sections": (64,), "device": "cpu", **kw})
    pos = torch.zeros((3, 5), dtype=torch.int32)

    class Table:
        sections = (16, 24, 24)

    class Plain:
        sections = None

    assert tsa._axis_positions(pos, Table, 5) == 5 and tsa._axis_positions(pos[0], Plain, 5) == -1
    assert tsa._axis_positions(pos[:, :4], Table, 4) == 5
    for p, t, T in ((pos, Plain, 5), (pos, None, 5), (pos[:2], Table, 5), (pos, Table, 4),
                    (pos.T.contiguous().T, Table, 5), (pos[0], Table, 4), (pos[None], Table, 5)):
        with pytest.raises(ValueError):
            tsa._axis_positions(p, t, T)
    with pytest.raises(TypeError):
        tsa._axis_positions(pos.long(), Table, 5)


# ---------------------------------------------------- shared rows
def _step(tsa, cache, kv8=True, **kw):
    a = dict(q=FAKE * 6, lens=FAKE * 7, B=4, cu=FAKE * 5, shared=FAKE * 4, N=2, Hq=8, Hkv=2, d=128,
             scale=0.1, out=FAKE * 8, out16=0, lse=None, ws=FAKE * 9, wb=1 << 40)
    a.update(kw)
    fn = tsa.lib().kv8_shared_attn_decode if kv8 else tsa.lib().shared_attn_decode
    return fn(a["q"], cache, a["lens"], a["B"], a["cu"], a["shared"], a["N"], a["Hq"], a["Hkv"],
              a["d"], a["scale"], a["out"], a["out16"], a["lse"], a["ws"], a["wb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(d=64), -1), (dict(B=-1), -1), (dict(B=4097), -1), (dict(Hkv=0), -1), (dict(Hq=18), -1),
    (dict(Hq=7), -1), (dict(B=4096, Hq=16), -1), (dict(N=-1), -1), (dict(N=4097), -1),
    (dict(q=None), -1), (dict(lens=None), -1), (dict(out=None), -1), (dict(cu=None), -1),
    (dict(shared=None), -1), (dict(q=FAKE + 2), -1), (dict(out=FAKE + 4), -1),
    (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1), (dict(ws=None), -2),
    (dict(ws=FAKE + 64), -2), (dict(wb=100), -2)])
def test_shared_step_refusals(tsa, kw, code):
    _refused(tsa, _step(tsa, C.byref(_cache(tsa)), **kw), code)
    kv = C.byref(tsa._KvStruct(FAKE, FAKE * 2, None, 0, 0, 1024))
    _refused(tsa, _step(tsa, kv, kv8=False, **kw), code)
    _refused(tsa, _step(tsa, None, **kw), -1)


def test_shared_step_caches_and_sizes(tsa):
    L = tsa.lib()
    _refused(tsa, _step(tsa, C.byref(_cache(tsa, format=2))))
    _refused(tsa, _step(tsa, C.byref(tsa._KvStruct(FAKE, None, None, 0, 0, 1024)), kv8=False))
    assert _step(tsa, C.byref(_cache(tsa)), B=0, q=None, out=None, lens=None, ws=None) == 0
    assert L.tsa_shared_attn_workspace_size(4, 2, 8, 2, 128) >= 256
    assert L.tsa_shared_attn_workspace_size(4, 2, 8, 2, 64) == 0
    assert L.tsa_shared_attn_workspace_size(0, 2, 8, 2, 128) == 0
    need = L.tsa_shared_attn_workspace_size(4, 2, 8, 2, 128)
    _refused(tsa, _step(tsa, C.byref(_cache(tsa)), wb=need - 1), -2)


def test_what_the_binding_refuses_about_pages_and_groups(tsa):
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError, match="CUDA tensor"):
        tsa.Pages(i(2, 4), i(9), 16)
    with pytest.raises(ValueError):
        tsa.Pages(i(8), i(9), 16)
    with pytest.raises(TypeError):
        tsa.Pages(i(2, 4).long(), i(9), 16)
    k = torch.zeros((4, 2, 32, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="paged"):
        tsa.pages_copy(tsa.kv_contiguous(k, k), i(3), i(3))
    kv = tsa.kv_paged(k, k, i(2, 4))
    with pytest.raises(ValueError):
        tsa.pages_copy([kv, tsa.kv_paged(k[:3].contiguous(), k[:3].contiguous(), i(2, 4))], i(3),
                       i(3))
    with pytest.raises(ValueError):
        tsa.pages_copy(kv, i(3), i(4))
    with pytest.raises(TypeError):
        tsa.pages_copy(kv, i(3), i(3).long())
    q = torch.zeros((2, 4, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="cu_group"):
        tsa.shared_attn_decode(q, kv, i(2), i(2), i(2))
    with pytest.raises(ValueError, match="sequences"):
        tsa.shared_attn_decode(q[:1], kv, i(2), i(2), i(1))
    with pytest.raises(ValueError, match="CUDA"):
        tsa.shared_attn_decode(q, kv, i(2), i(2), i(1))


def test_a_pool_without_sequences_needs_no_table(tsa):
    for name in ALL[:2]:
        assert _call(tsa, name, _pages(tsa, B=0, table=None), lo=None, hi=None) == 0
    assert _call(tsa, "pages_fork", _pages(tsa, B=0, table=None), n=0) == 0
    for name in ALL:
        _refused(tsa, _call(tsa, name, _pages(tsa, B=1, table=None)))
        _refused(tsa, _call(tsa, name, _pages(tsa, B=0, refs=None)))
