"""Scratch of bqd_kv_attend for many queries (host only): it follows the keys that a call can see,
and a plan too large to convert the codes ahead still shares the keys of a query tile."""
import ctypes

import pytest

import bit_quantized_decode_unpack_gb300 as bqd
from bit_quantized_decode_unpack_gb300 import _build
from bit_quantized_decode_unpack_gb300.kv_cache import CacheStruct

MOST = 2 << 30  # bytes that a call may ask for


@pytest.fixture(scope="module")
def need():
    _build.build()
    lib = bqd.load()

    def f(rows, heads, d, capacity, group, max_new, max_len=0, window=0):
        c = CacheStruct(k_codes=0x10000, v_codes=0x20000, k_scales=0x30000, v_scales=0x40000, table=0x50000, lens=0x60000,
                        refs=0x70000, pages=8, layers=1, kv_heads=heads, head_dim=d, page_tokens=64, rows=rows,
                        row_pages=capacity // 64, format=1, reserved=0)
        return lib.bqd_kv_attend_workspace(ctypes.byref(c), heads * group, rows * max_new, max_new, max_len, window)
    return f


def tiles(rows, heads, d, keys):
    """fp16 K and V of the steps that `keys` keys of each row and head can touch, with their scales."""
    step = 64 if d == 256 else 128
    return rows * heads * (keys // step + 2) * (2 * step * d * 2 + step // 16 * 8)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("window", [100, 4096])
def test_a_window_bounds_the_scratch(need, d, window):
    rows, heads, max_new = 8, 8, 2048
    want = tiles(rows, heads, d, window + max_new)
    for max_len in (0, 131072, 100000, window + max_new):
        assert need(rows, heads, d, 131072, 6, max_new, max_len, window) == want
    # rows shorter than the window and its queries
    assert need(rows, heads, d, 131072, 6, max_new, 1000, window) == tiles(rows, heads, d, min(1000, window + max_new))
    # a window that hides nothing
    assert need(rows, heads, d, 8192, 6, max_new, 0, 1 << 40) == need(rows, heads, d, 8192, 6, max_new)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_a_plan_too_large_to_convert_ahead_keeps_the_shares(need, d):
    rows, heads, group, max_new, capacity = 2, 64, 3, 200, 1 << 19
    assert tiles(rows, heads, d, capacity) > MOST
    # few query tiles, very many keys: O, m and l of every CTA that shares them
    bytes_ = need(rows, heads, d, capacity, group, max_new)
    a_share = rows * max_new * heads * group * (d * 4 + 8)
    assert bytes_ >= 2 * a_share and bytes_ % a_share == 0 and bytes_ <= MOST


@pytest.mark.parametrize("rows,max_new,capacity,window", [
    (1, 5000, 1 << 20, 0), (64, 300, 65536, 0), (4096, 64, 1 << 20, 777), (64, 300, 1 << 20, 50000), (3, 64, 1 << 20, 0)])
def test_never_more_than_the_most(need, rows, max_new, capacity, window):
    assert 0 <= need(rows, 8, 128, capacity, 6, max_new, 0, window) <= MOST
