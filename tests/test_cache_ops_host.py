"""Refusals and sizes of the cache-side entry points (rotary positions, the
8-bit cache, window attention): nothing here launches, so no GPU is needed."""
import ctypes as C

import pytest
import torch

FAKE = 1 << 20  # aligned, never dereferenced: validation fails first


@pytest.fixture(scope="module")
def tsa():
    import top_retrieval_sparse_gb300 as t
    t.lib()
    return t


def _refused(tsa, rc, code=-1):
    assert rc == code, (rc, tsa.lib().tsa_last_error().decode())
    assert tsa.lib().tsa_last_error().decode() != ""


def _spec(tsa, **kw):
    a = dict(theta=1e4, factor=1.0, low=0.0, high=0.0, amplitude=0.0, orig_len=0, max_pos=4096,
             rot_dim=128, layout=0, scaling=0)
    a.update(kw)
    return tsa._RopeSpec(**a)


@pytest.mark.parametrize("kw", [
    dict(rot_dim=0), dict(rot_dim=24), dict(rot_dim=144), dict(max_pos=0),
    dict(max_pos=(1 << 26) + 1), dict(layout=2), dict(scaling=5), dict(scaling=-1),
    dict(theta=1.0), dict(theta=float("inf")), dict(scaling=1, factor=0.5),
    dict(scaling=2, factor=float("nan")), dict(scaling=3, factor=2.0, orig_len=0),
    dict(scaling=4, factor=2.0, orig_len=4096, low=4.0, high=1.0),
    dict(scaling=3, factor=2.0, orig_len=4096, low=0.0, high=2.0),
    dict(amplitude=-1.0), dict(amplitude=float("nan"))])
def test_rope_table_refusals(tsa, kw):
    r = tsa._RopeStruct()
    _refused(tsa, tsa.lib().tsa_rope_table(C.byref(_spec(tsa, **kw)), FAKE, 1 << 40, C.byref(r),
                                           None))


def test_rope_table_size_and_memory(tsa):
    L = tsa.lib()
    assert L.tsa_rope_table_size(128, 1) == (2048 + 1) * 64 * 8
    assert L.tsa_rope_table_size(32, 2049) == (2048 + 2) * 16 * 8
    assert L.tsa_rope_table_size(24, 100) == 0 and L.tsa_rope_table_size(64, 0) == 0
    r = tsa._RopeStruct()
    need = L.tsa_rope_table_size(128, 4096)
    _refused(tsa, L.tsa_rope_table(C.byref(_spec(tsa)), FAKE, need - 1, C.byref(r), None))
    _refused(tsa, L.tsa_rope_table(C.byref(_spec(tsa)), FAKE + 8, need, C.byref(r), None))
    _refused(tsa, L.tsa_rope_table(C.byref(_spec(tsa)), None, need, C.byref(r), None))


def _rope_call(tsa, **kw):
    a = dict(q=(FAKE, 4096, 128), qo=(FAKE * 2, 4096, 128), Hq=4, k=(FAKE * 3, 4096, 128),
             ko=(FAKE * 4, 4096, 128), Hkv=2, T=7, d=128, pos=FAKE,
             rope=(FAKE, 4096, 128, 0))
    a.update(kw)
    rows = [C.byref(tsa._RowsStruct(*a[n])) if a[n] else None for n in ("q", "qo", "k", "ko")]
    rope = C.byref(tsa._RopeStruct(*a["rope"])) if a["rope"] else None
    return tsa.lib().rope_apply(rows[0], rows[1], a["Hq"], rows[2], rows[3], a["Hkv"], a["T"],
                                a["d"], a["pos"], rope, 0, None)


@pytest.mark.parametrize("kw", [
    dict(d=64), dict(Hq=0), dict(Hkv=-1), dict(T=-1), dict(T=1 << 31), dict(q=None),
    dict(qo=None), dict(k=None), dict(ko=None), dict(pos=None), dict(rope=None),
    dict(q=(FAKE + 8, 4096, 128)), dict(q=(FAKE, 4100, 128)), dict(q=(FAKE, -8, 128)),
    dict(qo=(FAKE * 2, 4096, 120)), dict(qo=(FAKE * 2, 504, 128)), dict(qo=(FAKE * 2, 0, 128)),
    dict(qo=(FAKE, 2048, 128)),  # over q with other strides
    dict(rope=(None, 4096, 128, 0)), dict(rope=(FAKE, 0, 128, 0)), dict(rope=(FAKE, 4096, 20, 0)),
    dict(rope=(FAKE, 4096, 128, 3))])
def test_rope_apply_refusals(tsa, kw):
    _refused(tsa, _rope_call(tsa, **kw))


def test_rope_apply_without_tokens_is_ok(tsa):
    assert _rope_call(tsa, T=0, q=None, qo=None, k=None, ko=None, pos=None) == 0


def _cache(tsa, **kw):
    a = dict(k=FAKE, v=FAKE * 2, k_scale=FAKE * 3, v_scale=FAKE * 4, page_table=None, status=None,
             l_cap=1024, page_size=0, max_pages=0, n_pages=0, block=64, format=0)
    a.update(kw)
    return tsa._Kv8Struct(**a)


PAGED = dict(page_table=FAKE * 5, page_size=32, max_pages=32, n_pages=100, block=32)
BAD_CACHES = [
    dict(k=None), dict(v_scale=None), dict(k=FAKE + 8), dict(k_scale=FAKE + 2),
    dict(status=FAKE + 4), dict(format=2), dict(block=48), dict(block=8), dict(block=256),
    dict(l_cap=0), dict(l_cap=1 << 31), dict(l_cap=1000), {**PAGED, "page_size": 24},
    {**PAGED, "block": 64}, {**PAGED, "max_pages": 31}, {**PAGED, "n_pages": 0}]


def _append(tsa, cache, **kw):
    a = dict(k=(FAKE * 6, 256, 128), v=(FAKE * 7, 256, 128), cu=FAKE * 8, T=10, max_new=5,
             lens=FAKE * 9, B=2, Hkv=2, d=128, rope=None, pos=None)
    a.update(kw)
    rows = [C.byref(tsa._RowsStruct(*a[n])) if a[n] else None for n in ("k", "v")]
    rope = C.byref(tsa._RopeStruct(*a["rope"])) if a["rope"] else None
    return tsa.lib().kv8_append(cache, rows[0], rows[1], a["cu"], a["T"], a["max_new"],
                                a["lens"], a["B"], a["Hkv"], a["d"], rope, a["pos"], None)


def _read(tsa, cache, **kw):
    a = dict(k=(FAKE * 6, 256, 128), v=(FAKE * 7, 256, 128), cu=FAKE * 8, T=10, max_new=5,
             lens=FAKE * 9, B=2, Hkv=2, d=128)
    a.update(kw)
    rows = [C.byref(tsa._RowsStruct(*a[n])) if a[n] else None for n in ("k", "v")]
    return tsa.lib().kv8_read(cache, rows[0], rows[1], a["cu"], a["T"], a["max_new"], a["lens"],
                              a["B"], a["Hkv"], a["d"], None)


def _decode(tsa, cache, kv8=True, **kw):
    a = dict(q=FAKE * 6, lens=FAKE * 7, B=2, Hq=8, Hkv=2, d=128, ni=4, nr=8, scale=0.1,
             out=FAKE * 8, lse=None, ws=FAKE * 9, wb=1 << 40)
    a.update(kw)
    fn = tsa.lib().kv8_attn_decode if kv8 else tsa.lib().window_attn_decode
    return fn(a["q"], cache, a["lens"], a["B"], a["Hq"], a["Hkv"], a["d"], a["ni"], a["nr"],
              a["scale"], a["out"], a["lse"], a["ws"], a["wb"], None)


@pytest.mark.parametrize("kw", BAD_CACHES)
def test_bad_caches_are_refused(tsa, kw):
    c = C.byref(_cache(tsa, **kw))
    _refused(tsa, _append(tsa, c))
    _refused(tsa, _read(tsa, c))
    _refused(tsa, _decode(tsa, c))


@pytest.mark.parametrize("call", [_append, _read])
@pytest.mark.parametrize("kw", [
    dict(d=64), dict(B=-1), dict(B=4097), dict(Hkv=0), dict(Hkv=1025), dict(k=None),
    dict(v=None), dict(lens=None), dict(T=-1), dict(max_new=-1), dict(cu=None),  # 10 != 2 * 5 is ok
    dict(k=(FAKE * 6 + 2, 256, 128)), dict(v=(FAKE * 7, 252, 128))])
def test_append_and_read_refusals(tsa, call, kw):
    if kw == dict(cu=None):
        kw = dict(cu=None, T=11)
    _refused(tsa, call(tsa, C.byref(_cache(tsa)), **kw))


def test_read_refuses_overlapping_rows(tsa):
    _refused(tsa, _read(tsa, C.byref(_cache(tsa)), k=(FAKE * 6, 128, 128)))
    _refused(tsa, _append(tsa, C.byref(_cache(tsa)), rope=(FAKE, 100, 24, 0)))


def test_nothing_to_do_is_ok(tsa):
    c = C.byref(_cache(tsa))
    for call in (_append, _read):
        assert call(tsa, c, T=0, k=None, v=None, lens=None) == 0
        assert call(tsa, c, B=0, T=0, k=None, v=None, lens=None) == 0
    assert _decode(tsa, c, B=0, q=None, out=None, lens=None, ws=None) == 0


DECODE = [(dict(d=64), -1), (dict(B=-1), -1), (dict(B=4097), -1), (dict(Hkv=0), -1),
          (dict(Hq=18), -1), (dict(Hq=7), -1), (dict(B=4096, Hq=16), -1), (dict(q=None), -1),
          (dict(lens=None), -1), (dict(out=None), -1), (dict(q=FAKE + 2), -1),
          (dict(out=FAKE + 4), -1), (dict(ni=-1), -1), (dict(nr=-1), -1),
          (dict(scale=float("nan")), -1), (dict(ws=None), -2), (dict(ws=FAKE + 64), -2),
          (dict(wb=100), -2)]


@pytest.mark.parametrize("kw,code", DECODE)
def test_decode_refusals(tsa, kw, code):
    _refused(tsa, _decode(tsa, C.byref(_cache(tsa)), **kw), code)
    kv = C.byref(tsa._KvStruct(FAKE, FAKE * 2, None, 0, 0, 1024))
    _refused(tsa, _decode(tsa, kv, kv8=False, **kw), code)


def _prefill(tsa, kv, **kw):
    a = dict(q=(FAKE * 6, 1024, 128), cu=FAKE * 5, T=10, max_q=6, lens=FAKE * 7, B=2, Hq=8, Hkv=2,
             d=128, ni=4, nr=8, scale=0.1, out=FAKE * 8, lse=None, ws=FAKE * 9, wb=1 << 40)
    a.update(kw)
    rows = C.byref(tsa._RowsStruct(*a["q"])) if a["q"] else None
    return tsa.lib().window_attn_prefill(
        rows, kv, a["cu"], a["T"], a["max_q"], a["lens"], a["B"], a["Hq"], a["Hkv"], a["d"],
        a["ni"], a["nr"], a["scale"], a["out"], a["lse"], a["ws"], a["wb"], None)


@pytest.mark.parametrize("kw,code", [x for x in DECODE if x[0] not in (
    dict(B=4096, Hq=16), dict(q=FAKE + 2))] + [
    (dict(q=(FAKE + 2, 1024, 128)), -1), (dict(q=(FAKE, 1020, 128)), -1), (dict(T=-1), -1),
    (dict(max_q=-1), -1), (dict(cu=None), -1), (dict(B=4096, Hkv=16, Hq=16), -1)])
def test_prefill_refusals(tsa, kw, code):
    kv = C.byref(tsa._KvStruct(FAKE, FAKE * 2, None, 0, 0, 1024))
    _refused(tsa, _prefill(tsa, kv, **kw), code)


def test_workspace_sizes(tsa):
    L = tsa.lib()
    assert L.tsa_attn_decode_workspace_size(1, 8, 2, 128) >= 256
    assert L.tsa_attn_decode_workspace_size(1, 8, 2, 64) == 0
    assert L.window_attn_prefill_workspace_size(1, 8, 2, 128, 5, 100, 4, 8) >= 256
    assert L.window_attn_prefill_workspace_size(1, 8, 2, 128, 5, 0, 4, 8) == 0


def test_binding_refuses_host_tensors_and_types(tsa):
    q = torch.zeros((3, 4, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        tsa.KV8(*(torch.zeros((1, 2, 64, 128), dtype=torch.uint8),) * 2,
                *(torch.zeros((1, 2, 1)),) * 2)
    with pytest.raises(TypeError):
        tsa.KV8(q, q, q, q)
    with pytest.raises(ValueError, match="fmt"):
        tsa.KV8(q, q, q, q, fmt="int4")
    with pytest.raises(ValueError, match="layout"):
        tsa.RopeTable(128, 10, layout="quarter")
    with pytest.raises(ValueError, match="scaling"):
        tsa.RopeTable(128, 10, scaling="more")
    with pytest.raises(tsa.TsaError):
        tsa.RopeTable(100, 10)
