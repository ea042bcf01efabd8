"""ctypes binding of the serving operators (C ABI in include/pi_serve.h and
include/pi_draft.h).

As in the package's other bindings, each ``pi_*`` function has the name and
argument order of its C entry point and only marshals arguments; tensors stay
the caller's, and the status is returned (see ``check``).  The package
re-exports everything here.
"""
from __future__ import annotations

import ctypes

PI_F32 = 2
PI_CACHE_MAX_SLOTS = 1024
PI_TOPK_MAX = 32
PI_TREE_MAX = 64
_DTYPES = {"f16": 0, "bf16": 1, "f32": PI_F32}


class pi_cache_desc(ctypes.Structure):
    _fields_ = [("layers", ctypes.c_int32), ("pages", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_tokens", ctypes.c_int32), ("dtype", ctypes.c_int32)]


_P, _I32, _SZ, _I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t, ctypes.c_int64
_CACHE = ctypes.POINTER(pi_cache_desc)
SIGNATURES = {
    "pi_cache_workspace_size": (_SZ, [_CACHE, _I32, _I32]),
    "pi_paged_attention": (ctypes.c_int, [_CACHE, _I32, _I32, _I32, _I32, _P, _P, _P, _P, _P, _P,
                                          ctypes.c_float, _I32, _I32, _P, _P, _P, _P, _SZ, _P]),
    "pi_selftest_attention_timeout": (ctypes.c_int, [_CACHE, _I32, _I32, _I32, _P, _P, _P, _P, _P,
                                                     _P, _P, _SZ, _I64, _P]),
    "pi_cache_append": (ctypes.c_int, [_CACHE, _I32, _I32, _I32, _I32, _P, _P, _P, _P, _P, _P, _P,
                                       _P]),
    "pi_cache_fork": (ctypes.c_int, [_CACHE, _I32, _I32, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                     _P, _P, _P, _SZ, _P]),
    "pi_cache_compact": (ctypes.c_int, [_CACHE, _I32, _I32, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                        _P, _SZ, _P]),
    "pi_cache_copy": (ctypes.c_int, [_CACHE, _P, _P, _I32, _P, _P, _P]),
    "pi_logprob_workspace_size": (_SZ, [_I32, _I32, _I32]),
    "pi_token_logprobs": (ctypes.c_int, [_P, _I32, _I32, _I32, _I64, _P, _I32, _P, _P, _P, _P, _P,
                                         _P, _SZ, _P]),
    "pi_tree_workspace_size": (_SZ, [_CACHE, _I32, _I32, _I32]),
    "pi_tree_attention": (ctypes.c_int, [_CACHE, _I32, _I32, _I32, _I32, _I32, _P, _P, _P, _P, _P, _P,
                                         _P, _P, ctypes.c_float, _I32, _I32, _P, _P, _P, _P, _SZ,
                                         _P]),
    "pi_selftest_tree_timeout": (ctypes.c_int, [_CACHE, _I32, _I32, _I32, _I32, _P, _P, _P, _P, _P, _P,
                                                _P, _SZ, _I64, _P]),
    "pi_tree_accept": (ctypes.c_int, [_CACHE, _I32, _I32, _I32, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                      _P, _P, _P]),
    "pi_sample_workspace_size": (_SZ, [_I32, _I32]),
    "pi_token_sample": (ctypes.c_int, [_P, _I32, _I32, _I32, _I64, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                       _SZ, _P]),
}


# These operators run for a few microseconds, so the binding keeps its own part
# short: entry points and torch's stream lookup are found once, and arguments
# that are tensors are taken without a call per argument.
_entry = {}
_torch = None
_raw_stream = None


def _pkg():
    from . import lib
    return lib()


def _fn(name):
    f = _entry.get(name)
    if f is None:
        f = _entry[name] = getattr(_pkg(), name)
    return f


def _ptr(t):
    """Device pointer of a tensor (or an int address, or None)."""
    if t is None:
        return None
    return t if type(t) is int else t.data_ptr()


def _current_stream():
    """Handle of torch's current stream; without making a stream object (which
    takes three microseconds) where torch offers that."""
    global _torch, _raw_stream
    if _torch is None:
        import torch
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        _torch = torch
    if _raw_stream is None:
        return _torch.cuda.current_stream().cuda_stream
    return _raw_stream(_torch.cuda.current_device())


def _stream(s):
    if s is None:
        return _current_stream()
    return s if isinstance(s, int) else s.cuda_stream


def _ws_bytes(ws, ws_bytes):
    return ws.nbytes if ws_bytes is None else ws_bytes


def make_cache_desc(layers: int, pages: int, kv_heads: int, head_dim: int, page_tokens: int,
                    dtype: str = "f16") -> pi_cache_desc:
    return pi_cache_desc(layers, pages, kv_heads, head_dim, page_tokens, _DTYPES[dtype])


def pi_cache_workspace_size(cache, slots: int, heads: int) -> int:
    return _fn("pi_cache_workspace_size")(ctypes.byref(cache), slots, heads)


def pi_logprob_workspace_size(rows: int, vocab: int, topk: int) -> int:
    return _fn("pi_logprob_workspace_size")(rows, vocab, topk)


def pi_tree_workspace_size(cache, slots: int, heads: int, drafts: int) -> int:
    return _fn("pi_tree_workspace_size")(ctypes.byref(cache), slots, heads, drafts)


def pi_sample_workspace_size(rows: int, vocab: int) -> int:
    return _fn("pi_sample_workspace_size")(rows, vocab)


def _zeros(nbytes, where, device):
    import torch

    from . import PI_ERR_SHAPE, PiError
    if nbytes == 0:
        raise PiError(PI_ERR_SHAPE, where)
    return torch.zeros(nbytes, dtype=torch.uint8, device=device)


def cache_workspace(cache, slots: int, heads: int = 0, device="cuda"):
    """A zero-filled workspace of pi_cache_workspace_size(cache, slots, heads) bytes."""
    return _zeros(pi_cache_workspace_size(cache, slots, heads), "pi_cache_workspace_size", device)


def logprob_workspace(rows: int, vocab: int, topk: int, device="cuda"):
    """A zero-filled workspace of pi_logprob_workspace_size(rows, vocab, topk) bytes."""
    return _zeros(pi_logprob_workspace_size(rows, vocab, topk), "pi_logprob_workspace_size", device)


def tree_workspace(cache, slots: int, heads: int, drafts: int, device="cuda"):
    """A zero-filled workspace of pi_tree_workspace_size(cache, slots, heads, drafts) bytes."""
    return _zeros(pi_tree_workspace_size(cache, slots, heads, drafts), "pi_tree_workspace_size", device)


def sample_workspace(rows: int, vocab: int, device="cuda"):
    """A zero-filled workspace of pi_sample_workspace_size(rows, vocab) bytes."""
    return _zeros(pi_sample_workspace_size(rows, vocab), "pi_sample_workspace_size", device)


def pi_paged_attention(cache, layer, slots, heads, max_pages, q, k_new, v_new, table, len, pool,
                       scale, window, sinks, y, lse, dev_status, ws, ws_bytes=None,
                       stream=None) -> int:
    return _fn("pi_paged_attention")(
        ctypes.byref(cache), layer, slots, heads, max_pages, _ptr(q), _ptr(k_new), _ptr(v_new),
        _ptr(table), _ptr(len), _ptr(pool), scale, window, sinks, _ptr(y), _ptr(lse),
        _ptr(dev_status), _ptr(ws), _ws_bytes(ws, ws_bytes), _stream(stream))


def pi_selftest_attention_timeout(cache, slots, heads, max_pages, q, table, len, pool, y, dev_status,
                                  ws, limit_ns, ws_bytes=None, stream=None) -> int:
    return _fn("pi_selftest_attention_timeout")(
        ctypes.byref(cache), slots, heads, max_pages, _ptr(q), _ptr(table), _ptr(len), _ptr(pool),
        _ptr(y), _ptr(dev_status), _ptr(ws), _ws_bytes(ws, ws_bytes), limit_ns, _stream(stream))


def pi_cache_append(cache, layer, slots, max_pages, tokens, slot, pos, k, v, table, pool,
                    dev_status, stream=None) -> int:
    return _fn("pi_cache_append")(
        ctypes.byref(cache), layer, slots, max_pages, tokens, _ptr(slot), _ptr(pos), _ptr(k),
        _ptr(v), _ptr(table), _ptr(pool), _ptr(dev_status), _stream(stream))


def pi_cache_fork(cache, slots, max_pages, parent, grow, held, table_in, len_in, table, len, ref,
                  pool, pairs, counts, dev_status, ws, ws_bytes=None, stream=None) -> int:
    return _fn("pi_cache_fork")(
        ctypes.byref(cache), slots, max_pages, _ptr(parent), _ptr(grow), _ptr(held),
        _ptr(table_in), _ptr(len_in), _ptr(table), _ptr(len), _ptr(ref), _ptr(pool), _ptr(pairs),
        _ptr(counts), _ptr(dev_status), _ptr(ws), _ws_bytes(ws, ws_bytes), _stream(stream))


def pi_cache_compact(cache, slots, max_pages, held, table_in, len, table, ref, map, pool, pairs,
                     counts, dev_status, ws, ws_bytes=None, stream=None) -> int:
    return _fn("pi_cache_compact")(
        ctypes.byref(cache), slots, max_pages, _ptr(held), _ptr(table_in), _ptr(len), _ptr(table),
        _ptr(ref), _ptr(map), _ptr(pool), _ptr(pairs), _ptr(counts), _ptr(dev_status), _ptr(ws),
        _ws_bytes(ws, ws_bytes), _stream(stream))


def pi_cache_copy(cache, pairs, count, cap, pool, dev_status, stream=None) -> int:
    return _fn("pi_cache_copy")(ctypes.byref(cache), _ptr(pairs), _ptr(count), cap, _ptr(pool),
                                _ptr(dev_status), _stream(stream))


def pi_token_logprobs(logits, dtype, rows, vocab, stride, tokens, topk, logprob, entropy, top_idx,
                      top_logprob, dev_status, ws, ws_bytes=None, stream=None) -> int:
    """dtype: "f16", "bf16", "f32" or the C enum's value."""
    return _fn("pi_token_logprobs")(
        _ptr(logits), _DTYPES.get(dtype, dtype), rows, vocab, stride, _ptr(tokens), topk,
        _ptr(logprob), _ptr(entropy), _ptr(top_idx), _ptr(top_logprob), _ptr(dev_status), _ptr(ws),
        _ws_bytes(ws, ws_bytes), _stream(stream))


def pi_tree_attention(cache, layer, slots, heads, max_pages, drafts, parent, count, q, k_new, v_new,
                      table, len, pool, scale, window, sinks, y, lse, dev_status, ws, ws_bytes=None,
                      stream=None) -> int:
    return _fn("pi_tree_attention")(
        ctypes.byref(cache), layer, slots, heads, max_pages, drafts, _ptr(parent), _ptr(count),
        _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(table), _ptr(len), _ptr(pool), scale, window, sinks,
        _ptr(y), _ptr(lse), _ptr(dev_status), _ptr(ws), _ws_bytes(ws, ws_bytes), _stream(stream))


def pi_selftest_tree_timeout(cache, slots, heads, max_pages, drafts, q, table, len, pool, y,
                             dev_status, ws, limit_ns, ws_bytes=None, stream=None) -> int:
    return _fn("pi_selftest_tree_timeout")(
        ctypes.byref(cache), slots, heads, max_pages, drafts, _ptr(q), _ptr(table), _ptr(len),
        _ptr(pool), _ptr(y), _ptr(dev_status), _ptr(ws), _ws_bytes(ws, ws_bytes), limit_ns,
        _stream(stream))


def pi_tree_accept(cache, slots, max_pages, drafts, parent, count, tokens, choice, table, len, pool,
                   len_out, path, accepted, next, dev_status, stream=None) -> int:
    return _fn("pi_tree_accept")(
        ctypes.byref(cache), slots, max_pages, drafts, _ptr(parent), _ptr(count), _ptr(tokens),
        _ptr(choice), _ptr(table), _ptr(len), _ptr(pool), _ptr(len_out), _ptr(path), _ptr(accepted),
        _ptr(next), _ptr(dev_status), _stream(stream))


def pi_token_sample(logits, dtype, rows, vocab, stride, temperature, top_k, top_p, min_p, u, token,
                    logprob, dev_status, ws, ws_bytes=None, stream=None) -> int:
    """dtype: "f16", "bf16", "f32" or the C enum's value."""
    return _fn("pi_token_sample")(
        _ptr(logits), _DTYPES.get(dtype, dtype), rows, vocab, stride, _ptr(temperature), _ptr(top_k),
        _ptr(top_p), _ptr(min_p), _ptr(u), _ptr(token), _ptr(logprob), _ptr(dev_status), _ptr(ws),
        _ws_bytes(ws, ws_bytes), _stream(stream))
