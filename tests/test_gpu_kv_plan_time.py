"""Time of masked attention over the number of a cache's rows, most of them idle."""
import pytest

from _kv_util import i32

pytestmark = pytest.mark.gpu


def _ms(rows, live=64, length=2000, nodes=21, heads=8, group=6, d=128, pt=64):
    import torch
    from bit_quantized_decode_unpack_gb300.kv_cache import KVCache
    each = -(-length // pt)
    codes = torch.randint(-127, 128, (2, 1, live * each, heads, pt, d), dtype=torch.int8, device="cuda")
    scales = torch.full((2, 1, live * each, heads, pt // 16), 1 / 60, device="cuda")
    table = torch.full((rows, each), -1, dtype=torch.int32, device="cuda")
    table[:live] = torch.arange(live * each, dtype=torch.int32, device="cuda").view(live, each)
    lens = i32([length] * live + [0] * (rows - live))
    cache = KVCache(codes[0], codes[1], scales[0], scales[1], table, lens, i32([1] * (live * each)))
    starts = i32([min(r, live) * nodes for r in range(rows + 1)])
    q = torch.randn((live * nodes, heads * group, d), device="cuda").half()
    mask = torch.full((live * nodes, 1), -1, dtype=torch.int64, device="cuda")
    assert cache.attend_workspace(heads * group, live * nodes, nodes, masked=True) > 1 << 24  # the tile kernel
    out, lse = cache.attend(q, starts, mask=mask, max_new=nodes)
    best = []
    for _ in range(7):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(5):
            cache.attend(q, starts, mask=mask, max_new=nodes, out=out, lse=lse)
        b.record()
        b.synchronize()
        best.append(a.elapsed_time(b) / 5)
    return min(best)


def test_idle_rows_do_not_multiply_the_time():
    """Sixteen times the rows with the same work: with a plan that every CTA makes of all rows, twenty times as long."""
    few, many = _ms(64), _ms(1000)
    assert many < 8 * few, (few, many)
