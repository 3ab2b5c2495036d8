"""Which kernel a masked call is planned for (host only), by its scratch: that of the tile kernel is over 16 MB.
Each case takes 1.4 to 6.7 times as long with the other one, measured."""
import ctypes

import pytest

import bit_quantized_decode_unpack_gb300 as bqd
from bit_quantized_decode_unpack_gb300 import _build
from bit_quantized_decode_unpack_gb300.kv_cache import CacheStruct


@pytest.fixture(scope="module")
def tiles():
    _build.build()
    lib = bqd.load()

    def f(d, heads, group, nodes, rows, live, keys):
        c = CacheStruct(k_codes=0x10000, v_codes=0x20000, k_scales=0x30000, v_scales=0x40000, table=0x50000, lens=0x60000,
                        refs=0x70000, pages=8, layers=1, kv_heads=heads, head_dim=d, page_tokens=64, rows=rows,
                        row_pages=1024, format=1, reserved=0)
        return lib.bqd_kv_attend_masked_workspace(ctypes.byref(c), heads * group, live * nodes, nodes, keys, 0) > 1 << 24
    return f


@pytest.mark.parametrize("case", [
    # head_dim, KV heads, group, nodes of a row, rows, rows with nodes, keys
    (256, 4, 6, 4, 1024, 8, 500), (128, 8, 6, 8, 1024, 8, 4000), (128, 8, 6, 21, 1024, 8, 500), (64, 8, 6, 8, 256, 8, 500),
    (128, 2, 16, 21, 256, 8, 500), (64, 8, 6, 21, 1024, 8, 4000), (128, 8, 6, 4, 1024, 1024, 500), (128, 8, 6, 8, 256, 256, 200),
    (64, 8, 6, 8, 1024, 1024, 200)])
def test_few_queries(tiles, case):
    assert not tiles(*case)


@pytest.mark.parametrize("case", [
    (128, 8, 6, 21, 1024, 1024, 500), (128, 8, 6, 8, 256, 256, 4000), (128, 8, 6, 21, 64, 8, 4000), (128, 8, 6, 21, 4, 4, 65001),
    (256, 4, 6, 21, 1024, 1024, 4000), (64, 8, 6, 21, 256, 256, 500), (128, 2, 16, 21, 64, 64, 4000), (64, 8, 6, 21, 64, 8, 4000)])
def test_tiles(tiles, case):
    assert tiles(*case)
