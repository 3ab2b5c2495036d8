"""Random caches for the KV cache's tests, as NumPy arrays (for the oracle) and
as device tensors (for the library)."""
import numpy as np

import oracle.kv_cache as okv

BF16_HALF, F16_HALF = 2.0 ** -8, 2.0 ** -11  # half a unit in the last place, relative


def rounded(x, dtype):
    """x as the values of fp16 or bf16 (a torch tensor) and as float64."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(getattr(torch, dtype))
    return t, t.double().numpy()


def random_cache(rng, lens, *, heads=2, d=128, pt=64, fmt="int8", layers=1, spare=3, row_pages=None, spread=0.25):
    """Rows of these lengths over a randomly ordered pool; every page holds random codes."""
    need = [-(-n // pt) for n in lens]
    pages = sum(need) + spare
    width = row_pages or max([1] + need) + 1
    perm = rng.permutation(pages)
    table = np.full((len(lens), width), -1, np.int64)
    refs = np.zeros(pages, np.int64)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = perm[at:at + n]
        refs[table[r, :n]] = 1
        at += n
    shape = (layers, pages, heads, pt, d)
    cache = {"table": table, "lens": np.array(lens, np.int64), "refs": refs, "fmt": fmt}
    for name in ("k", "v"):
        x = rng.standard_normal(shape) * (34 if fmt == "int8" else 110)
        cache[name] = okv.encode(x, fmt)
        mean = 1 / 34 if fmt == "int8" else 1 / 110
        cache[name + "s"] = (mean * np.exp(spread * rng.standard_normal(shape[:3] + (pt // 16,)))).astype(np.float32)
    return cache


def code_bytes(values, fmt):
    """Code values to stored bytes."""
    if fmt == "int8":
        return values.astype(np.int8).view(np.uint8)
    mag = np.searchsorted(okv.E4M3[:127], np.abs(values)).astype(np.uint8)
    return mag | (np.signbit(values).astype(np.uint8) << 7)


def to_library(cache, dev="cuda"):
    import torch
    from bit_quantized_decode_unpack_gb300.kv_cache import KVCache
    kind = torch.int8 if cache["fmt"] == "int8" else torch.float8_e4m3fn
    t = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(dev)
    i32 = lambda x: t(np.asarray(x, np.int32))
    return KVCache(t(code_bytes(cache["k"], cache["fmt"])).view(kind), t(code_bytes(cache["v"], cache["fmt"])).view(kind),
                   t(cache["ks"]), t(cache["vs"]), i32(cache["table"]), i32(cache["lens"]), i32(cache["refs"]))


def raw(t):
    import torch
    return t.view(torch.uint8).cpu().numpy()


def assert_same(lib, cache, pools=True):
    """The library's state is the oracle's, bit for bit (a zero's sign apart)."""
    np.testing.assert_array_equal(lib.table.cpu().numpy(), cache["table"])
    np.testing.assert_array_equal(lib.lens.cpu().numpy(), cache["lens"])
    np.testing.assert_array_equal(lib.refs.cpu().numpy(), cache["refs"])
    if pools:
        for name in ("k", "v"):
            np.testing.assert_array_equal(okv.decode_bytes(raw(getattr(lib, name)), cache["fmt"]), cache[name])
            np.testing.assert_array_equal(getattr(lib, name + "_scales").cpu().numpy(), cache[name + "s"])


def i32(x, dev="cuda"):
    import torch
    return torch.tensor(np.asarray(x, np.int32), device=dev)


def starts_of(news):
    return np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
