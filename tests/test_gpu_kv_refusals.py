"""What the KV cache's Python calls refuse before a kernel sees an address."""
import numpy as np
import pytest

from _kv_util import i32, random_cache, to_library

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    return to_library(random_cache(np.random.default_rng(0), [20, 5], heads=2, d=64, pt=16))


def _q(n=2, heads=4, d=64, **kw):
    import torch
    return torch.zeros((n, heads, d), dtype=kw.get("dtype", torch.float16), device=kw.get("device", "cuda"))


def test_cache_tensors(lib):
    import torch
    from bit_quantized_decode_unpack_gb300.kv_cache import KVCache
    good = [lib.k, lib.v, lib.k_scales, lib.v_scales, lib.table, lib.lens, lib.refs]
    KVCache(*good)
    bad = {0: [lib.k.cpu(), lib.k.half(), lib.k[0], lib.k[:, :, :, :8], lib.k[:, :, :, :, :32]],
           1: [lib.v.cpu(), lib.v[:, :-1], lib.v.view(torch.uint8), lib.v.transpose(1, 2)],
           2: [lib.k_scales.half(), lib.k_scales[:, :-1]],
           3: [lib.v_scales.cpu(), lib.v_scales.double()],
           4: [lib.table.long(), lib.table.flatten(), lib.table.t(), lib.table.cpu(), lib.table[:, :0]],
           5: [lib.lens.long(), lib.lens[:1]],
           6: [lib.refs[:-1], lib.refs.cpu()]}
    for i, values in bad.items():
        for value in values:
            with pytest.raises(ValueError):
                KVCache(*good[:i], value, *good[i + 1:])
    with pytest.raises(ValueError):
        KVCache.empty(1, 4, 1, 64, 1, 1, format="int4")
    with pytest.raises(ValueError):
        KVCache.empty(1, 4, 1, 96, 1, 1)
    with pytest.raises(ValueError):
        KVCache.empty(0, 4, 1, 64, 1, 1)


def test_attend_arguments(lib):
    import torch
    lib.attend(_q())
    starts = i32([0, 1, 2])
    for args, kw in [((_q(dtype=torch.float32),), {}), ((_q(device="cpu"),), {}), ((_q(heads=3),), {}),
                     ((_q(heads=0),), {}), ((_q(d=128),), {}), ((_q(n=3),), {}), ((_q()[0],), {}),
                     ((_q().transpose(1, 2).contiguous().transpose(1, 2),), {}),
                     ((_q(), starts.long()), {}), ((_q(), starts[:2]), {}), ((_q(), starts.cpu()), {}),
                     ((_q(), starts), {"max_new": -1}), ((_q(),), {"window": -1}), ((_q(),), {"max_len": -1}),
                     ((_q(),), {"layer": 1}), ((_q(),), {"layer": -1}),
                     ((_q(),), {"out": _q(n=3)}), ((_q(),), {"out": _q(dtype=torch.bfloat16)}),
                     ((_q(),), {"lse": torch.zeros((2, 3), device="cuda")})]:
        with pytest.raises(ValueError):
            lib.attend(*args, **kw)
    from bit_quantized_decode_unpack_gb300 import BqdError
    with pytest.raises(BqdError):
        lib.attend(_q(), scale=float("nan"))
    empty, lse = lib.attend(_q(n=0), i32([0, 0, 0]))
    assert empty.shape == (0, 4, 64) and lse.shape == (0, 4)


def test_append_arguments(lib):
    import torch
    k, base = _q(heads=2), i32([0, 0])
    lib.append(k, k, base)
    for args, kw in [((k, k.bfloat16(), base), {}), ((k, k[:1], base), {}), ((k, _q(heads=1), base), {}),
                     ((k, k, base.long()), {}), ((k, k, base[:1]), {}), ((k, k, None), {}), ((k.float(), k.float(), base), {}),
                     ((k, k, base, i32([0, 2])), {}), ((k, k, base), {"layer": 7}),
                     ((k, k, base, i32([0, 1, 2])), {"max_new": -3})]:
        with pytest.raises(ValueError):
            lib.append(*args, **kw)
    assert torch.cuda.current_device() == 0


def test_page_arguments(lib):
    with pytest.raises(ValueError):
        lib.reserve(i32([1]))
    with pytest.raises(ValueError):
        lib.reserve(i32([1, 1]).long())
    with pytest.raises(ValueError):
        lib.fork(i32([[0]]))
    with pytest.raises(ValueError):
        lib.fork(i32([0, 1]), i32([1]))
    with pytest.raises(ValueError):
        lib.fork(i32([0, 1]).cpu())
    with pytest.raises(ValueError):
        lib.truncate(i32([1]))
    with pytest.raises(ValueError):
        lib.copy_pages(i32([1]), i32([1, 2]))
