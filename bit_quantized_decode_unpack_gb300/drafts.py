"""Drafts as a tree: ancestor masks, and greedy verification against the target's logits.

A row's drafted nodes are tokens starts[r] .. starts[r + 1] - 1 of the ragged batch, a parent before
its children; node 0 is the last token that the target chose.

    mask, depth, positions = tree_mask(parents, starts, base=base)       # once a step, or once for all
    out, lse = cache.attend(q, starts, mask=mask, depth=depth, ...)      # per layer
    accepted, token, path = spec_tree_verify(logits, drafted, parents, starts, max_path=8)
    cache = cache.accept(path, starts)                                   # the path's tokens stay
"""
from __future__ import annotations

import ctypes

from . import DTYPE_BF16, DTYPE_F16, DTYPE_F32, _check, load
from . import kv_cache as _kv

MAX_WORDS = 16
_LOGITS = {}  # element types of logits


def declare(lib):
    """Argument types of the entry points."""
    i64, i32, vp = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p
    lib.bqd_tree_mask.argtypes = [vp, vp, i64, i64, i32, vp, vp, vp, vp, vp]
    lib.bqd_tree_mask.restype = i32
    lib.bqd_spec_tree_verify.argtypes = [vp, i32, i64, i64, vp, vp, vp, i64, i64, i32, vp, vp, vp, vp, vp]
    lib.bqd_spec_tree_verify.restype = i32


_lib = None


def _bind():
    """Binds torch, and the library once for all calls."""
    global _lib
    if _lib is None:
        _kv._bind()
        t = _kv.torch
        _LOGITS.update({t.float16: DTYPE_F16, t.bfloat16: DTYPE_BF16, t.float32: DTYPE_F32})
        _lib = load()
    return _kv.torch


def _logits(t):
    """(element type, rows, V, row stride) of logits [rows, V], V contiguous."""
    shape = getattr(t, "shape", ())
    if len(shape) != 2 or not t.is_cuda:
        raise ValueError("logits must be a 2-D CUDA tensor [rows, V]")
    kind = _LOGITS.get(t.dtype)
    if kind is None:
        raise ValueError(f"logits: dtype {t.dtype}, expected float16, bfloat16 or float32")
    (rows, v), (stride, one) = shape, t.stride()
    if v < 1 or (v > 1 and one != 1) or (rows > 1 and stride < v):
        raise ValueError(f"logits: shape {tuple(shape)} with strides {t.stride()}: rows must be contiguous and apart")
    return kind, rows, v, stride


def _tree(parents, starts):
    """(tokens, rows, device) of a batch of trees."""
    torch = _bind()
    tokens, marks = getattr(parents, "shape", ()), getattr(starts, "shape", ())
    if len(tokens) != 1 or not parents.is_cuda:
        raise ValueError("parents must be an int32 CUDA tensor [tokens]")
    if len(marks) != 1 or marks[0] < 1:
        raise ValueError("starts must be an int32 tensor [rows + 1]")
    dev = parents.device
    _kv._dense(parents, "parents", torch.int32, tokens, dev)
    _kv._dense(starts, "starts", torch.int32, marks, dev)
    return tokens[0], marks[0] - 1, dev


def _here(device, stream):
    """None, or a context for another current device or an explicit stream."""
    return None if stream is None and _kv._device() == device.index else _kv._On(device, stream)


def _out(t, name, shape, device, dtype=None):
    """The given output, checked, or a new one."""
    dtype = dtype or _kv.torch.int32
    if t is None:
        return _kv.torch.empty(shape, dtype=dtype, device=device)
    return _kv._dense(t, name, dtype, shape, device)


def _at(t):
    """Address of an optional tensor."""
    return None if t is None else t.data_ptr()


def tree_mask(parents, starts, *, words: int = 1, base=None, mask=None, depth=None, positions=None, stream=None):
    """Ancestor masks of trees of drafts (bqd_tree_mask).

    parents int32 [tokens] (the row's own indices; -1: a root), starts int32 [rows + 1].  Returns
    (mask int64 [tokens, words]: the node's ancestors and itself, 64 nodes a word; depth int32
    [tokens]; positions int32 [tokens]: base[r] + depth, or None without ``base`` int32 [rows]).
    Entries of tokens that no row has are left as they are."""
    tokens, rows, dev = _tree(parents, starts)
    if not 1 <= words <= MAX_WORDS:
        raise ValueError(f"words must be in [1, {MAX_WORDS}], got {words}")
    if base is not None:
        _kv._dense(base, "base", _kv.torch.int32, (rows,), dev)
    elif positions is not None:
        raise ValueError("positions: needs base")
    on = _here(dev, stream)
    if on is not None:
        with on:
            return tree_mask(parents, starts, words=words, base=base, mask=mask, depth=depth, positions=positions)
    mask = _out(mask, "mask", (tokens, words), dev, _kv.torch.int64)
    depth = _out(depth, "depth", (tokens,), dev)
    if base is not None:
        positions = _out(positions, "positions", (tokens,), dev)
    _check("bqd_tree_mask", _lib.bqd_tree_mask(
        parents.data_ptr(), starts.data_ptr(), rows, tokens, words, _at(base), mask.data_ptr(), depth.data_ptr(), _at(positions),
        _kv._raw_stream(dev.index)))
    return mask, depth, positions


def spec_tree_verify(logits, drafted, parents, starts, *, max_path: int, accepted=None, next_token=None, path=None,
                     argmax_out=None, stream=None):
    """Greedy verification of trees of drafts (bqd_spec_tree_verify).

    logits fp16, bf16 or fp32 [tokens, V] (row i scores the token after node i); drafted and
    parents int32 [tokens]; starts int32 [rows + 1].  From a row's node 0 the walk goes on to the
    lowest child whose token is the argmax at its parent, for ``max_path`` nodes at most.  Returns
    (accepted int32 [rows]: nodes after node 0; next_token int32 [rows]: the argmax at the last
    node; path int32 [rows, max_path]: the nodes, then -1).  ``argmax_out`` (int32 [tokens])
    receives every node's argmax."""
    tokens, rows, dev = _tree(parents, starts)
    kind, n, v, stride = _logits(logits)
    if n != tokens or logits.device != dev:
        raise ValueError(f"logits: {n} rows on {logits.device}, expected {tokens} on {dev}")
    _kv._dense(drafted, "drafted", _kv.torch.int32, (tokens,), dev)
    if not 1 <= max_path < 2 ** 31:
        raise ValueError(f"max_path must be at least 1, got {max_path}")
    on = _here(dev, stream)
    if on is not None:
        with on:
            return spec_tree_verify(logits, drafted, parents, starts, max_path=max_path, accepted=accepted,
                                    next_token=next_token, path=path, argmax_out=argmax_out)
    accepted = _out(accepted, "accepted", (rows,), dev)
    next_token = _out(next_token, "next_token", (rows,), dev)
    path = _out(path, "path", (rows, max_path), dev)
    argmax_out = _out(argmax_out, "argmax_out", (tokens,), dev)
    _check("bqd_spec_tree_verify", _lib.bqd_spec_tree_verify(
        logits.data_ptr(), kind, stride, v, drafted.data_ptr(), parents.data_ptr(), starts.data_ptr(), rows, tokens, max_path,
        accepted.data_ptr(), next_token.data_ptr(), path.data_ptr(), argmax_out.data_ptr(), _kv._raw_stream(dev.index)))
    return accepted, next_token, path
