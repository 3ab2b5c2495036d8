"""Host-side validation of the tree step's C entry points and Python calls (nothing is launched)."""
import ctypes

import pytest

import bit_quantized_decode_unpack_gb300 as bqd
from bit_quantized_decode_unpack_gb300 import _build
from bit_quantized_decode_unpack_gb300.rope import RopeStruct
from test_kv_abi_cpu import _cache

INV, ALIGN = 1, 3


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return bqd.load()


def _rope(lib, plan=None, q=0x1000, qts=512, qhs=128, qh=4, k=0x9000, kts=256, khs=128, kh=2, dt=1, pos=0x2000, tokens=3,
          qo=0x3000, qots=512, qohs=128, ko=0x5000, kots=256, kohs=128, **kw):
    p = dict(q_weight=0x6000, k_weight=None, freqs=0x7000, head_dim=128, rotary_dim=64, weight_dtype=1, interleaved=0, norm=1,
             reserved=0, eps=1e-6, amplitude=1.0)
    p.update(kw)
    c = RopeStruct(**p)
    return lib.bqd_qk_norm_rope(ctypes.byref(c), q, qts, qhs, qh, k, kts, khs, kh, dt, pos, tokens, qo, qots, qohs, ko, kots,
                                kohs, None)


def test_struct_layout_matches_the_header():
    assert ctypes.sizeof(RopeStruct) == 3 * 8 + 6 * 4 + 2 * 4 and RopeStruct.eps.offset == 48


@pytest.mark.parametrize("kw,want", [
    (dict(head_dim=96), INV), (dict(rotary_dim=24), INV), (dict(rotary_dim=256), INV), (dict(rotary_dim=-16), INV),
    (dict(freqs=None), INV), (dict(dt=2), INV), (dict(weight_dtype=3), INV), (dict(weight_dtype=0), INV),
    (dict(eps=0.0), INV), (dict(eps=float("nan")), INV), (dict(eps=float("inf")), INV), (dict(amplitude=float("inf")), INV),
    (dict(tokens=-1), INV), (dict(qh=-1), INV), (dict(q=None), INV), (dict(ko=None), INV), (dict(pos=None), INV),
    (dict(qts=-1), INV), (dict(qots=100), INV), (dict(qohs=64), INV), (dict(qots=256, qohs=128), INV), (dict(kts=1 << 41), INV),
    (dict(q=0x1001), ALIGN), (dict(qo=0x3001), ALIGN), (dict(pos=0x2002), ALIGN), (dict(freqs=0x7004), ALIGN),
    (dict(q_weight=0x6001), ALIGN), (dict(q_weight=0x6002, weight_dtype=2), ALIGN),
    (dict(tokens=0, q=None, qo=None, k=None, ko=None, pos=None), 0), (dict(qh=0, kh=0, q=None, k=None), 0),
    (dict(tokens=0, eps=0.0, norm=0), 0),
])
def test_qk_norm_rope(lib, kw, want):
    assert _rope(lib, **kw) == want


def test_qk_norm_rope_without_a_plan(lib):
    assert lib.bqd_qk_norm_rope(None, 0x1000, 1, 1, 1, None, 0, 0, 0, 1, None, 1, 0x1000, 1, 1, None, 0, 0, None) == INV


def test_tree_mask(lib):
    f = lambda parents=0x1000, starts=0x2000, rows=2, tokens=9, words=1, base=0x3000, mask=0x4000, depth=0x5000, pos=0x6000: \
        lib.bqd_tree_mask(parents, starts, rows, tokens, words, base, mask, depth, pos, None)  # noqa: E731
    for kw in (dict(rows=-1), dict(tokens=-1), dict(tokens=1 << 31), dict(words=0), dict(words=17), dict(base=None),
               dict(parents=None), dict(starts=None)):
        assert f(**kw) == INV, kw
    for kw in (dict(parents=0x1002), dict(starts=0x2001), dict(base=0x3002), dict(mask=0x4004), dict(depth=0x5002), dict(pos=0x6002)):
        assert f(**kw) == ALIGN, kw
    assert f(rows=0, parents=None) == 0 and f(tokens=0, parents=None) == 0
    assert f(mask=None, depth=None, pos=None) == 0


def test_spec_tree_verify(lib):
    def f(logits=0x1000, dt=1, stride=100, V=100, drafted=0x2000, parents=0x3000, starts=0x4000, rows=2, tokens=9, path_n=4,
          acc=0x5000, nxt=0x6000, path=0x7000, best=0x8000):
        return lib.bqd_spec_tree_verify(logits, dt, stride, V, drafted, parents, starts, rows, tokens, path_n, acc, nxt, path,
                                        best, None)
    for kw in (dict(dt=0), dict(dt=4), dict(V=0), dict(V=1 << 31), dict(stride=99), dict(stride=1 << 41), dict(rows=-1),
               dict(tokens=-1), dict(tokens=(1 << 28) + 1), dict(path_n=0), dict(logits=None), dict(drafted=None),
               dict(parents=None), dict(starts=None), dict(acc=None), dict(nxt=None), dict(path=None), dict(best=None)):
        assert f(**kw) == INV, kw
    for kw in (dict(logits=0x1001), dict(logits=0x1002, dt=2), dict(drafted=0x2002), dict(path=0x7001), dict(best=0x8002)):
        assert f(**kw) == ALIGN, kw
    assert f(rows=0, logits=None) == 0


def test_token_logprobs(lib):
    def f(logits=0x1000, dt=3, stride=100, rows=4, V=100, tokens=0x2000, top=5, lp=0x3000, ent=0x4000, rank=0x5000, ids=0x6000,
          tops=0x7000):
        return lib.bqd_token_logprobs(logits, dt, stride, rows, V, tokens, top, lp, ent, rank, ids, tops, None)
    for kw in (dict(dt=5), dict(rows=-1), dict(V=0), dict(V=1 << 31), dict(stride=99), dict(top=-1), dict(top=33),
               dict(tokens=None), dict(tokens=None, lp=None), dict(tokens=None, rank=None), dict(logits=None)):
        assert f(**kw) == INV, kw
    for kw in (dict(logits=0x1001), dict(logits=0x1002, dt=2), dict(tokens=0x2001), dict(ids=0x6002), dict(ent=0x4001)):
        assert f(**kw) == ALIGN, kw
    assert f(rows=0, logits=None) == 0
    assert f(lp=None, ent=None, rank=None, ids=None, tops=None) == 0


def _masked(lib, c=None, tokens=6, starts=0x4000, max_new=3, window=0, mask=0xa000, words=1, depth=None, q=0x1000, out=0x2000,
            scale=0.1):
    c = c or _cache()
    return lib.bqd_kv_attend_masked(ctypes.byref(c), 0, q, 512, 128, 1, 4, starts, tokens, max_new, 0, scale, window, mask,
                                    words, depth, out, None, None, 0, None)


@pytest.mark.parametrize("kw,want", [
    (dict(words=0), INV), (dict(words=17), INV), (dict(mask=None), INV), (dict(window=4), INV), (dict(window=-1), INV),
    (dict(q=None), INV), (dict(scale=float("nan")), INV), (dict(starts=None), INV), (dict(mask=0xa004), ALIGN),
    (dict(depth=0xb002), ALIGN), (dict(out=0x2008), ALIGN), (dict(tokens=0, mask=None), 0), (dict(max_new=0), 0),
])
def test_attend_masked(lib, kw, want):
    assert _masked(lib, **kw) == want


def test_attend_masked_checks_the_cache(lib):
    assert _masked(lib, _cache(head_dim=96)) == INV


def test_accept(lib):
    c, other = _cache(), _cache(table=0x51000, lens=0x61000, refs=0x71000)
    r, o = ctypes.byref(c), ctypes.byref(other)
    f = lambda a=r, b=o, path=0x8000, width=4, starts=0x9000: lib.bqd_kv_accept(a, b, path, width, starts, None)  # noqa: E731
    assert f(b=r) == INV and f(path=None) == INV and f(width=0) == INV and f(a=None) == INV
    assert f(path=0x8002) == ALIGN and f(starts=0x9001) == ALIGN
    for kw in (dict(k_codes=0x90000), dict(pages=7), dict(rows=2), dict(refs=0x70000), dict(lens=0x60000)):
        bad = _cache(**dict(dict(table=0x51000, lens=0x61000, refs=0x71000), **kw))
        assert f(b=ctypes.byref(bad)) == INV, kw


def test_tensors_on_the_host_are_refused():
    import torch
    z, i32 = torch.zeros, torch.int32
    with pytest.raises(ValueError):
        bqd.QKNormRope(128, [1.0] * 64, device="cpu")
    for bad in (dict(head_dim=96), dict(inv_freq=[1.0] * 7), dict(inv_freq=[1.0] * 72), dict(inv_freq=[float("inf")] * 8),
                dict(eps=0.0), dict(amplitude=float("nan"))):
        kw = dict(dict(head_dim=128, inv_freq=[1.0] * 8), **bad)
        with pytest.raises(ValueError):
            bqd.QKNormRope(kw.pop("head_dim"), kw.pop("inv_freq"), device="cpu", **kw)
    with pytest.raises(ValueError):
        bqd.tree_mask(z(4, dtype=i32), z(2, dtype=i32))
    with pytest.raises(ValueError):
        bqd.spec_tree_verify(z(4, 10), z(4, dtype=i32), z(4, dtype=i32), z(2, dtype=i32), max_path=2)
    with pytest.raises(ValueError):
        bqd.token_logprobs(z(4, 10), z(4, dtype=i32), 2)


def test_frequencies_are_exact_turns():
    assert bqd.rope_frequencies([0.0]) == [0]
    for f in (1.0, 0.1, 1e-5, 7.0, -0.25):
        turns = bqd.rope_frequencies([f])[0] / 2.0 ** 64
        assert abs((turns - f / 6.283185307179586 + 0.5) % 1 - 0.5) < 1e-15
