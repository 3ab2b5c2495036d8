"""Host-side validation of the KV cache's C entry points (nothing is launched)."""
import ctypes

import pytest

import bit_quantized_decode_unpack_gb300 as bqd
from bit_quantized_decode_unpack_gb300 import _build
from bit_quantized_decode_unpack_gb300.kv_cache import CacheStruct

INV, ALIGN = 1, 3


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return bqd.load()


def _cache(**kw):
    a = dict(k_codes=0x10000, v_codes=0x20000, k_scales=0x30000, v_scales=0x40000, table=0x50000, lens=0x60000,
             refs=0x70000, pages=8, layers=2, kv_heads=2, head_dim=128, page_tokens=64, rows=3, row_pages=4, format=1,
             reserved=0)
    a.update(kw)
    return CacheStruct(**a)


def _attend(lib, c=None, layer=0, q=0x1000, ts=512, hs=128, dt=1, heads=4, starts=None, tokens=3, max_new=1, max_len=0,
            scale=0.1, window=0, out=0x2000, lse=None, work=None, work_bytes=0):
    c = c or _cache()
    return lib.bqd_kv_attend(ctypes.byref(c), layer, q, ts, hs, dt, heads, starts, tokens, max_new, max_len, scale,
                             window, out, lse, work, work_bytes, None)


def test_struct_layout_matches_the_header():
    # seven pointers, one int64, eight int32, in the header's order
    assert ctypes.sizeof(CacheStruct) == 7 * 8 + 8 + 8 * 4
    assert CacheStruct.pages.offset == 56 and CacheStruct.format.offset == 88


@pytest.mark.parametrize("kw,want", [
    (dict(format=0), INV), (dict(format=3), INV), (dict(head_dim=96), INV), (dict(page_tokens=48), INV),
    (dict(page_tokens=8), INV), (dict(layers=0), INV), (dict(kv_heads=0), INV), (dict(pages=0), INV),
    (dict(pages=1 << 30), INV), (dict(rows=-1), INV), (dict(rows=65536), INV), (dict(row_pages=0), INV),
    (dict(row_pages=1 << 25), INV), (dict(k_codes=None), INV), (dict(v_scales=None), INV), (dict(table=None), INV),
    (dict(lens=None), INV), (dict(refs=None), INV), (dict(k_codes=0x10008), ALIGN), (dict(v_scales=0x40002), ALIGN),
    (dict(table=0x50001), ALIGN),
])
def test_every_entry_point_checks_the_cache(lib, kw, want):
    c = _cache(**kw)
    r = ctypes.byref(c)
    assert _attend(lib, c) == want
    assert lib.bqd_kv_append(r, 0, 0x1000, 256, 128, 0x2000, 256, 128, 1, 0x3000, None, 3, 1, None) == want
    assert lib.bqd_kv_reserve(r, None, 0x1000, 0x2000, 0x3000, None) == want
    assert lib.bqd_kv_fork(r, r, 0x1000, None, None) == want
    assert lib.bqd_kv_compact(r, r, 0x1000, 0x2000, None) == want
    assert lib.bqd_kv_copy_pages(r, 0x1000, 0x2000, 1, None) == want


def test_null_cache(lib):
    assert lib.bqd_kv_reserve(None, None, 0x1000, 0x2000, 0x3000, None) == INV


@pytest.mark.parametrize("kw,want", [
    (dict(layer=-1), INV), (dict(layer=2), INV), (dict(dt=2), INV), (dict(heads=3), INV), (dict(heads=0), INV),
    (dict(tokens=2), INV), (dict(tokens=-1), INV), (dict(starts=0x4000, max_new=-1), INV), (dict(q=None), INV),
    (dict(out=None), INV), (dict(scale=float("inf")), INV), (dict(scale=float("nan")), INV), (dict(window=-1), INV),
    (dict(max_len=-1), INV), (dict(ts=-1), INV), (dict(hs=1 << 41), INV), (dict(q=0x1001), ALIGN),
    (dict(out=0x2008), ALIGN), (dict(lse=0x2002), ALIGN), (dict(starts=0x4002), ALIGN),
    (dict(work_bytes=-1), INV), (dict(work_bytes=16), INV), (dict(work=0x9008, work_bytes=16), ALIGN),
    (dict(starts=0x4000, tokens=0, q=None, out=None), 0), (dict(starts=0x4000, max_new=0, q=None), 0),
])
def test_attend(lib, kw, want):
    assert _attend(lib, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(layer=2), INV), (dict(k=None), INV), (dict(v=None), INV), (dict(base=None), INV), (dict(dt=2), INV),
    (dict(tokens=4), INV), (dict(ts=-8), INV), (dict(k=0x1001), ALIGN), (dict(base=0x3002), ALIGN),
    (dict(starts=0x4000, tokens=0, k=None, v=None), 0),
])
def test_append(lib, kw, want):
    a = dict(layer=0, k=0x1000, v=0x2000, ts=256, hs=128, dt=1, base=0x3000, starts=None, tokens=3, max_new=1)
    a.update(kw)
    c = _cache()
    assert lib.bqd_kv_append(ctypes.byref(c), a["layer"], a["k"], a["ts"], a["hs"], a["v"], a["ts"], a["hs"], a["dt"],
                             a["base"], a["starts"], a["tokens"], a["max_new"], None) == want


def test_workspace(lib):
    r = ctypes.byref(_cache())
    w = lambda *x: lib.bqd_kv_attend_workspace(*x, 0)
    assert w(r, 4, 3, 1, 0) == 0                                       # few queries and keys need none
    assert w(r, 4, 9000, 4096, 200) >= 3 * 2 * 200 * 2 * 128 * 2       # fp16 K and V of every row and head
    assert w(r, 4, 9000, 4096, 100) < w(r, 4, 9000, 4096, 256) == w(r, 4, 9000, 4096, 0) == w(r, 4, 9000, 4096, 10 ** 9)
    assert w(r, 4, 4096, 10 ** 6, 0) == w(r, 4, 4096, 4096, 0)
    for bad in ((r, 3, 9000, 4096, 0), (r, 0, 9000, 4096, 0), (r, 4, 9000, 0, 0), (r, 4, 0, 4096, 0), (r, 4, 9000, 4096, -1),
                (r, 4, 1 << 40, 1 << 40, 0), (ctypes.byref(_cache(pages=0)), 4, 9000, 4096, 0), (None, 4, 9000, 4096, 0)):
        assert w(*bad) == 0
    assert lib.bqd_kv_attend_workspace(r, 4, 9000, 4096, 0, -1) == 0


def test_pages(lib):
    c, other = _cache(), _cache(table=0x51000, lens=0x61000, refs=0x71000)
    r, o = ctypes.byref(c), ctypes.byref(other)
    assert lib.bqd_kv_reserve(r, None, None, 0x2000, 0x3000, None) == INV
    assert lib.bqd_kv_reserve(r, None, 0x1000, 0x2000, None, None) == INV
    assert lib.bqd_kv_reserve(r, 0x1002, 0x1000, 0x2000, 0x3000, None) == ALIGN
    many = _cache(rows=4097)
    assert lib.bqd_kv_reserve(ctypes.byref(many), None, 0x1000, 0x2000, 0x3000, None) == INV
    # `to` must be another state of the same pools
    assert lib.bqd_kv_fork(r, r, 0x1000, None, None) == INV
    assert lib.bqd_kv_fork(r, o, None, None, None) == INV
    assert lib.bqd_kv_fork(r, o, 0x1002, None, None) == ALIGN
    for kw in (dict(k_codes=0x90000), dict(pages=7), dict(layers=1), dict(row_pages=5), dict(refs=0x70000), dict(table=0x50000),
               dict(lens=0x60000), dict(page_tokens=32), dict(format=2)):
        bad = _cache(**dict(dict(table=0x51000, lens=0x61000, refs=0x71000), **kw))
        assert lib.bqd_kv_fork(r, ctypes.byref(bad), 0x1000, None, None) == INV
        assert lib.bqd_kv_compact(r, ctypes.byref(bad), 0x1000, 0x2000, None) == INV
    rows = _cache(table=0x51000, lens=0x61000, refs=0x71000, rows=5)
    assert lib.bqd_kv_compact(r, ctypes.byref(rows), 0x1000, 0x2000, None) == INV
    assert lib.bqd_kv_compact(r, o, None, 0x2000, None) == INV
    assert lib.bqd_kv_compact(r, o, 0x1000, None, None) == INV
    assert lib.bqd_kv_copy_pages(r, 0x1000, 0x2000, -1, None) == INV
    assert lib.bqd_kv_copy_pages(r, 0x1000, 0x2000, 9, None) == INV
    assert lib.bqd_kv_copy_pages(r, None, 0x2000, 1, None) == INV
    assert lib.bqd_kv_copy_pages(r, 0x1000, 0x2002, 1, None) == ALIGN
    assert lib.bqd_kv_copy_pages(r, None, None, 0, None) == 0


def test_tensors_on_the_host_are_refused():
    import torch
    z = torch.zeros
    with pytest.raises(ValueError):
        bqd.KVCache(z((1, 4, 1, 16, 64), dtype=torch.int8), z((1, 4, 1, 16, 64), dtype=torch.int8), z((1, 4, 1, 1)),
                    z((1, 4, 1, 1)), z((2, 2), dtype=torch.int32), z(2, dtype=torch.int32), z(4, dtype=torch.int32))
