"""Norm of query and key heads with the rotation by position, in one pass over both.

What stands between the q and k projections and the cache: each head is normalised (root mean
square, one weight a value) and its first ``rotary_dim`` values are turned by angles that grow
with the token's position.

    rope = QKNormRope(128, inv_freq, q_weight=wq, k_weight=wk)     # a layer's plan
    q, k = rope(q, k, positions)                                   # [tokens, heads, 128] each

q and k may be views of one projection's output.  Angles are exact modulo a turn for every int32
position (``rope_frequencies``).  For serving, like the rest of the library: nothing here records
gradients.
"""
from __future__ import annotations

import ctypes
from . import DTYPE_BF16, DTYPE_F16, DTYPE_F32, _check, load
from . import kv_cache as _kv

HEAD_DIMS = (64, 128, 256)
_PI = 31415926535897932384626433832795028841971693993751058209749445923078164  # pi * 10^70
_TURNS = 10 ** 70 * 2 ** 191 // _PI  # 2^192 / (2 pi)
_WEIGHTS = {"torch.float16": DTYPE_F16, "torch.bfloat16": DTYPE_BF16, "torch.float32": DTYPE_F32}


class RopeStruct(ctypes.Structure):
    """bqd_qk_rope (include/bqd.h)."""
    _fields_ = [("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p), ("freqs", ctypes.c_void_p),
                ("head_dim", ctypes.c_int32), ("rotary_dim", ctypes.c_int32), ("weight_dtype", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("norm", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("eps", ctypes.c_float), ("amplitude", ctypes.c_float)]


def declare(lib):
    """Argument types of the entry point."""
    i64, i32, vp = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p
    lib.bqd_qk_norm_rope.argtypes = [ctypes.POINTER(RopeStruct), vp, i64, i64, i32, vp, i64, i64, i32, i32, vp, i64,
                                     vp, i64, i64, vp, i64, i64, vp]
    lib.bqd_qk_norm_rope.restype = i32


def rope_frequencies(inv_freq) -> list:
    """Inverse frequencies (radians a position) in turns, as the 64-bit fractions that the kernel
    multiplies by positions: inv_freq / (2 pi) * 2^64, rounded, modulo 2^64."""
    def turns(f):
        n, d = float(f).as_integer_ratio()  # d is a power of two
        shift = 128 + d.bit_length() - 1
        return (n * _TURNS + (1 << shift - 1) >> shift) % 2 ** 64

    return [turns(f) for f in inv_freq]


class QKNormRope:
    """A layer's plan (bqd_qk_rope): y = x w / sqrt(mean(x^2) + eps), then the rotation.

    inv_freq: the rotary_dim / 2 inverse frequencies (a sequence or tensor; empty: no rotation).
    q_weight, k_weight: fp16, bf16 or fp32 [head_dim] of one type, or None (ones); with
    ``norm=False`` values are rotated as they are.  ``interleaved`` pairs value 2 j with 2 j + 1
    instead of j with j + rotary_dim / 2.  ``amplitude`` multiplies sines and cosines."""

    def __init__(self, head_dim: int, inv_freq, *, q_weight=None, k_weight=None, eps: float = 1e-6, norm: bool = True,
                 interleaved: bool = False, amplitude: float = 1.0, device=None):
        _kv._bind()
        torch = _kv.torch
        if head_dim not in HEAD_DIMS:
            raise ValueError(f"head_dim must be one of {HEAD_DIMS}, got {head_dim}")
        given = [w for w in (q_weight, k_weight) if w is not None]
        if device is None:
            device = given[0].device if given else "cuda"
        freqs = inv_freq.tolist() if hasattr(inv_freq, "tolist") else list(inv_freq)
        rotary = 2 * len(freqs)
        if rotary > head_dim or rotary % 16:
            raise ValueError(f"inv_freq: {len(freqs)} frequencies, expected a multiple of 8 up to {head_dim // 2}")
        if not all(abs(f) < float("inf") for f in freqs):
            raise ValueError("inv_freq must be finite")
        if norm and not 0 < eps < float("inf"):
            raise ValueError(f"eps must be positive, got {eps}")
        if not abs(amplitude) < float("inf"):
            raise ValueError(f"amplitude must be finite, got {amplitude}")
        turns = [f - 2 ** 64 if f >= 2 ** 63 else f for f in rope_frequencies(freqs)]
        self.freqs = torch.tensor(turns, dtype=torch.int64, device=device)
        self.device = self.freqs.device
        if self.device.type != "cuda":
            raise ValueError(f"must be on a CUDA device, got {self.device}")
        for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
            if w is None:
                continue
            if not norm:
                raise ValueError(f"{name}: without a norm there are no weights")
            if str(w.dtype) not in _WEIGHTS:
                raise ValueError(f"{name}: dtype {w.dtype}, expected float16, bfloat16 or float32")
            _kv._dense(w, name, given[0].dtype, (head_dim,), self.device)
        self.q_weight, self.k_weight = q_weight, k_weight
        self.head_dim, self.rotary_dim = head_dim, rotary
        kind = _WEIGHTS[str(given[0].dtype)] if given else DTYPE_F32
        self._kinds = (DTYPE_F16, DTYPE_BF16) if kind == DTYPE_F32 else (kind,)
        p = lambda t: None if t is None else t.data_ptr() or None
        self._c = RopeStruct(p(q_weight), p(k_weight), p(self.freqs), head_dim, rotary, kind, bool(interleaved), bool(norm),
                             0, eps if norm else 0.0, amplitude)
        self._ref, self._call, self._index = ctypes.byref(self._c), load().bqd_qk_norm_rope, self.device.index

    def _half(self, t, name, tokens, dtype):
        """The tensor's heads, checked: [tokens, heads, head_dim] on the device, head_dim contiguous."""
        shape = getattr(t, "shape", ())
        if len(shape) != 3 or t.device != self.device:
            raise ValueError(f"{name}: must be a 3-D tensor [tokens, heads, head_dim] on {self.device}")
        if t.dtype is not dtype or shape[0] != tokens or shape[2] != self.head_dim or t.stride(2) != 1:
            raise ValueError(f"{name}: {t.dtype} {tuple(shape)}, expected {dtype} [{tokens}, heads, {self.head_dim}], "
                             "head_dim contiguous")
        return shape[1]

    def __call__(self, q, k, positions=None, *, q_out=None, k_out=None, stream=None):
        """(q, k) normalised and rotated (bqd_qk_norm_rope).

        q, k: fp16 or bf16 [tokens, heads, head_dim], any strides of token and head; k may be
        None.  positions: int32 [tokens] (None without rotation).  Outputs are new and dense, or
        q_out and k_out, which may be q and k themselves."""
        dtype = getattr(q, "dtype", None)
        kind = _kv._KINDS.get(dtype)
        if kind not in self._kinds:
            raise ValueError(f"q: dtype {dtype}, expected float16 or bfloat16, and that of weights below fp32")
        tokens = q.shape[0] if q.shape else 0
        heads = self._half(q, "q", tokens, dtype)
        k_heads = 0 if k is None else self._half(k, "k", tokens, dtype)
        at = None
        if self.rotary_dim:
            _kv._dense(positions, "positions", _kv.torch.int32, (tokens,), self.device)
            at = positions.data_ptr()
        if stream is not None or _kv._device() != self._index:
            with _kv._On(self.device, stream):
                return self(q, k, positions, q_out=q_out, k_out=k_out)
        empty = _kv.torch.empty
        if q_out is None:
            q_out = empty((tokens, heads, self.head_dim), dtype=dtype, device=self.device)
        elif self._half(q_out, "q_out", tokens, dtype) != heads:
            raise ValueError(f"q_out: {q_out.shape[1]} heads, expected {heads}")
        if k is None:
            if k_out is not None:
                raise ValueError("k_out: there is no k")
            ks, kos, k_at, k_to = (0, 0), (0, 0), None, None
        else:
            if k_out is None:
                k_out = empty((tokens, k_heads, self.head_dim), dtype=dtype, device=self.device)
            elif self._half(k_out, "k_out", tokens, dtype) != k_heads:
                raise ValueError(f"k_out: {k_out.shape[1]} heads, expected {k_heads}")
            ks, kos, k_at, k_to = k.stride(), k_out.stride(), k.data_ptr(), k_out.data_ptr()
        qs, qos = q.stride(), q_out.stride()
        _check("bqd_qk_norm_rope", self._call(
            self._ref, q.data_ptr(), qs[0], qs[1], heads, k_at, ks[0], ks[1], k_heads, kind,
            at, tokens, q_out.data_ptr(), qos[0], qos[1], k_to, kos[0], kos[1],
            _kv._raw_stream(self._index)))
        return q_out, k_out


def qk_norm_rope(q, k, positions, inv_freq, *, q_out=None, k_out=None, stream=None, **plan):
    """``QKNormRope(head_dim, inv_freq, **plan)`` made for one call (the plan's own copies to the
    device wait for the host: keep one where calls repeat)."""
    if getattr(q, "dim", lambda: 0)() != 3:
        raise ValueError("q must be a 3-D tensor [tokens, heads, head_dim]")
    if stream is not None and q.is_cuda:
        with _kv._On(q.device, stream):  # the plan's frequencies too: they are freed before the stream has read them
            return qk_norm_rope(q, k, positions, inv_freq, q_out=q_out, k_out=k_out, **plan)
    return QKNormRope(q.shape[2], inv_freq, device=q.device, **plan)(q, k, positions, q_out=q_out, k_out=k_out, stream=stream)
