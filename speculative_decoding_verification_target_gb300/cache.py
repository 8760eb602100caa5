"""Operators of the scoring step around a verification: binding of the C ABI in include/speccache.h.

Argument marshalling only, as for the verification calls. A cache in 4 bits is a pool of pages, uint8
[pages, Hk, 68 D] (new_pool), a table int32 [sequences, max_pages] of page numbers, lengths int32 [sequences] and
refs int32 [pages]; the header states the format and every rule. One round of a serving loop:

    pages_reserve(pools, table, lengths, refs, n_new)          room for the last token and K drafts
    per layer:
        qk_norm_rope(q, k, positions, freqs, ...)              head norms and rotation
        cache_append(pool, table, lengths, k, v)               quantised into the pages
        cache_attention(q, pool, table, lengths + n_new)       the new tokens over the cache
    verify(logits, ...)                                        accept_len
    pages_commit(table, lengths, refs, accept_len)             keeps the accepted tokens, frees the rest

and beside it pages_fork (a sequence that shares another's pages), pages_release, pages_compact and cache_read.

Every tensor of a call is on the current device. A call runs on `stream`, or on the current one. Outputs and workspaces that
are not given are made on that stream; what is given has to be ready on it. The status word is in the workspace
(read_status, the STATUS_ bits): a caller that looks at it passes the workspace. No call records gradients: outputs are
detached, also from inputs that require them.
"""
from __future__ import annotations

import ctypes
import functools
import math

import torch

from . import SPEC_OK, SpecError, _current_device, _need, _new, load as _load

PAGE, GROUP = 64, 32
WS_HEADER = 8192
STATUS_BAD_PAGE, STATUS_BAD_LENGTH, STATUS_NO_PAGES, STATUS_BAD_SLOT = 4, 8, 16, 32
CACHE_EXPORTS = ("spec_cache_block_bytes", "spec_qk_norm_rope", "spec_cache_append", "spec_cache_read",
                 "spec_cache_attention_workspace_size", "spec_cache_attention", "spec_pages_workspace_size",
                 "spec_pages_fork", "spec_pages_reserve", "spec_pages_commit", "spec_pages_release",
                 "spec_pages_compact", "spec_cache_last_error")


class Heads(ctypes.Structure):
    """spec_heads: [B, N, heads, D] in device memory, element strides over the first three."""
    _fields_ = [("data", ctypes.c_void_p), ("stride_b", ctypes.c_longlong), ("stride_n", ctypes.c_longlong),
                ("stride_h", ctypes.c_longlong)]


@functools.cache
def _lib():
    lib = _load()
    P, I, F, Z, L = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_longlong
    H = ctypes.POINTER(Heads)
    for name, res, args in (
            ("spec_cache_block_bytes", Z, [I]),
            ("spec_qk_norm_rope", I, [H, H, I, I, I, I, I, I, P, P, I, I, P, P, F, H, H, P]),
            ("spec_cache_append", I, [P, I, P, I, P, P, H, H, I, I, I, I, I, P, Z, P]),
            ("spec_cache_read", I, [P, I, P, I, P, P, H, H, I, I, I, I, I, P, Z, P]),
            ("spec_cache_attention_workspace_size", Z, [I, I, I, I]),
            ("spec_cache_attention", I, [H, I, P, I, P, I, P, P, I, I, I, I, I, F, I, I, H, P, P, Z, P]),
            ("spec_pages_workspace_size", Z, [I, I]),
            ("spec_pages_fork", I, [P, P, P, I, I, I, P, P, I, P, Z, P]),
            ("spec_pages_reserve", I, [P, I, L, P, P, P, I, I, I, P, P, P, Z, P]),
            ("spec_pages_commit", I, [P, P, P, I, I, I, P, I, I, I, P, Z, P]),
            ("spec_pages_release", I, [P, P, P, I, I, I, P, I, P, Z, P]),
            ("spec_pages_compact", I, [P, I, L, P, P, I, I, I, P, P, Z, P]),
            ("spec_cache_last_error", ctypes.c_char_p, [])):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args
    return lib


def _ok(code):
    if code != SPEC_OK:
        raise SpecError(code, _lib().spec_cache_last_error().decode())


_DTYPES = {torch.bfloat16: 0, torch.float32: 1, torch.float16: 2}
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


# The serving loop calls these once per layer and token, so the checks are written to cost little where they pass: one
# condition, and the words for what is wrong only after it.
def _home(t, name, stream):
    """The device of a call, t's: the current one, since the library launches there. Every other tensor has to be on it."""
    d = t.get_device()
    if d < 0:
        raise ValueError("%s must be a CUDA tensor" % name)
    if d != _current_device():
        raise ValueError("%s is on cuda:%d, the current device is cuda:%d" % (name, d, _current_device()))
    if stream is not None and stream.device.index != d:
        raise ValueError("%s is on cuda:%d, the stream on cuda:%d" % (name, d, stream.device.index))
    return d


def _on(d, stream):
    """The stream's handle: the caller's, or the current one of device d."""
    if stream is not None:
        return stream.cuda_stream
    return _raw_stream(d) if _raw_stream is not None else torch.cuda.current_stream(d).cuda_stream


def _ptr(t):
    return None if t is None else t.data_ptr()


def _code(t, name, fp32=False):
    code = _DTYPES.get(t.dtype)
    if code is None or (code == 1 and not fp32):
        raise TypeError("%s must be bfloat16%s float16%s, got %s" % (name, "," if fp32 else " or",
                                                                   " or float32" if fp32 else "", t.dtype))
    return code


def _rows(t, name):
    """[B, N, heads, D] with any strides but contiguous channels, its type, shape and device known."""
    sb, sn, sh, sd = t.stride()
    if sd != 1:
        raise ValueError("%s must have contiguous channels" % name)
    return Heads(t.data_ptr(), sb, sn, sh)


def _heads(t, name, shape, dtype, d):
    """The same, with those checked."""
    if not (t.get_device() == d and t.dtype is dtype and t.shape == shape):
        if not t.is_cuda:
            raise ValueError("%s must be a CUDA tensor" % name)
        if t.dtype is not dtype:
            raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
        if t.shape != shape:
            raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
        raise ValueError("%s must be on cuda:%d, got cuda:%d" % (name, d, t.get_device()))
    return _rows(t, name)


def _own(t):
    """The same for an output made here, which needs no check."""
    sb, sn, sh, _ = t.stride()
    return Heads(t.data_ptr(), sb, sn, sh)


def _like(t, stream):
    """An output in t's order of dimensions, and its rows. Contiguous where t repeats rows in a way that would leave the order
    to a stride of 1 beside the channels'."""
    o = torch.empty_like(t) if stream is None else _new(torch.empty_like, stream, t)
    sb, sn, sh, sd = o.stride()
    if sd != 1:
        o = _new(torch.empty_like, stream, t, memory_format=torch.contiguous_format)
        sb, sn, sh, sd = o.stride()
    return o, Heads(o.data_ptr(), sb, sn, sh)


def _vector(t, name, dtype, shape, d):
    if not (t.get_device() == d and t.dtype is dtype and t.shape == shape and t.is_contiguous()):
        _need(t, name, dtype, shape)


def _pool(pool, d, name="pool"):
    if not (pool.get_device() == d and pool.dtype is torch.uint8 and pool.is_contiguous()):
        _need(pool, name, torch.uint8)
    if pool.dim() != 3:
        raise ValueError("%s must be [pages, Hk, 68 D], got %s" % (name, tuple(pool.shape)))
    P, H, n = pool.shape
    if n not in (68 * 64, 68 * 128):
        raise ValueError("%s's blocks must have 68 D bytes for D = 64 or 128, got %d" % (name, n))
    return P, H, n // 68


def _ints(t, name, shape, d):
    if not (t.get_device() == d and t.dtype is torch.int32 and t.shape == shape and t.is_contiguous()):
        _need(t, name, torch.int32, shape)


def _table(table, d):
    if not (table.get_device() == d and table.dtype is torch.int32 and table.is_contiguous()):
        _need(table, "table", torch.int32)
    if table.dim() != 2:
        raise ValueError("table must be [sequences, max_pages], got %s" % (tuple(table.shape),))
    return table.shape


def _workspace(ws, d):
    """The caller's workspace as (address, bytes)."""
    if not (ws.get_device() == d and ws.dtype is torch.uint8 and ws.is_contiguous()):
        _need(ws, "workspace", torch.uint8)
    return ws.data_ptr(), ws.numel()


def new_pool(pages, kv_heads, head_dim, layers=None, device=None):
    """A pool of free pages: uint8 [pages, Hk, 68 D], or [layers, pages, Hk, 68 D], of which pool[l] is a layer's."""
    if head_dim not in (64, 128):
        raise ValueError("head_dim must be 64 or 128, got %r" % (head_dim,))
    shape = (pages, kv_heads, 68 * head_dim)
    return torch.zeros(shape if layers is None else (layers,) + shape, dtype=torch.uint8, device=device or "cuda")


def new_attention_workspace(N, q_heads, kv_heads, head_dim, device=None):
    """Workspace of cache_attention for up to N new tokens a sequence, ready for its first use."""
    n = int(_lib().spec_cache_attention_workspace_size(N, q_heads, kv_heads, head_dim))
    if n == 0:
        raise ValueError("unsupported sizes N=%d Hq=%d Hk=%d D=%d" % (N, q_heads, kv_heads, head_dim))
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def new_pages_workspace(sequences, pages, device=None):
    """Workspace of the pages_* calls, cache_append and cache_read, ready for its first use."""
    n = int(_lib().spec_pages_workspace_size(sequences, pages))
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def rope_frequencies(rotary_dim, theta=10000.0, *, inv_freq=None, device=None):
    """The rotation's frequencies for qk_norm_rope: each pair's turns a position in 2^-64 of a turn, int64 (the bits of
    a uint64) [rotary_dim / 2], from theta ** (-2 i / rotary_dim), or from inv_freq (radians a position)."""
    if inv_freq is None:
        inv = theta ** (torch.arange(0, rotary_dim, 2, dtype=torch.float64) / -rotary_dim)
    else:
        inv = torch.as_tensor(inv_freq, dtype=torch.float64, device="cpu")
        if inv.numel() != rotary_dim // 2:
            raise ValueError("inv_freq must have rotary_dim / 2 = %d values, got %d" % (rotary_dim // 2, inv.numel()))
    high = torch.remainder(inv / (2.0 * math.pi), 1.0) * 2.0 ** 32
    low = (high - high.floor()) * 2.0 ** 32      # exact: a double's 53 bits, in two steps
    return (high.floor().long() << 32 | low.floor().long()).to(device or "cuda")


def qk_norm_rope(q, k, positions, freqs, *, q_weight=None, k_weight=None, eps=1e-6, interleaved=False, q_out=None,
                 k_out=None, stream=None):
    """Root-mean-square norm of each head of q [B, N, Hq, D] and k [B, N, Hk, D], times a weight [D], and rotation of the
    first 2 len(freqs) channels by position (int32 [B, N]). bf16, fp16 or fp32. freqs from rope_frequencies, or None
    for the norm alone. q_out, k_out may be q and k; unless given they are laid out in q's and k's order. Returns
    dict(q, k)."""
    B, N, Hq, D = q.shape
    Hk = k.shape[2]
    dt = q.dtype
    code = _code(q, "q", True)
    d = _home(q, "q", stream)
    qi, ki = _rows(q, "q"), _heads(k, "k", (B, N, Hk, D), dt, d)
    rotary, pos, fr = 0, None, None
    if freqs is not None:
        _vector(freqs, "freqs", torch.int64, (freqs.numel(),), d)
        _ints(positions, "positions", (B, N), d)
        rotary, pos, fr = 2 * freqs.numel(), positions.data_ptr(), freqs.data_ptr()
    if q_weight is not None:
        _vector(q_weight, "q_weight", dt, (D,), d)
    if k_weight is not None:
        _vector(k_weight, "k_weight", dt, (D,), d)
    if q_out is None:
        q_out, qo = _like(q, stream)
    else:
        qo = _heads(q_out, "q_out", (B, N, Hq, D), dt, d)
    if k_out is None:
        k_out, ko = _like(k, stream)
    else:
        ko = _heads(k_out, "k_out", (B, N, Hk, D), dt, d)
    _ok(_lib().spec_qk_norm_rope(qi, ki, code, B, N, Hq, Hk, D, pos, fr, rotary, interleaved, _ptr(q_weight),
                                 _ptr(k_weight), eps, qo, ko, _on(d, stream)))
    return dict(q=q_out, k=k_out)


def cache_append(pool, table, start, k, v, *, counts=None, workspace=None, stream=None):
    """Quantises k and v [B, N, Hk, D] (bf16 or fp16) into pool [pages, Hk, 68 D]: token i of sequence b to position
    start[b] + i, for i < counts[b] (None: N). Returns the workspace."""
    d = _home(pool, "pool", stream)
    P, H, D = _pool(pool, d)
    B, M = _table(table, d)
    N = k.shape[1]
    code = _code(k, "k")
    _ints(start, "start", (B,), d)
    if counts is not None:
        _ints(counts, "counts", (B,), d)
    if workspace is None:
        workspace = _new(torch.zeros, stream, WS_HEADER, dtype=torch.uint8, device=pool.device)
    _ok(_lib().spec_cache_append(pool.data_ptr(), P, table.data_ptr(), M, start.data_ptr(), _ptr(counts),
                                 _heads(k, "k", (B, N, H, D), k.dtype, d), _heads(v, "v", (B, N, H, D), k.dtype, d), code, B, N,
                                 H, D, *_workspace(workspace, d), _on(d, stream)))
    return workspace


def cache_read(pool, table, start, n, *, counts=None, dtype=torch.bfloat16, k=None, v=None, workspace=None, stream=None):
    """The cached keys and values of positions start[b] .. start[b] + n - 1 as [B, n, Hk, D] in bf16 or fp16, exactly;
    zeros past counts[b] and where there is no page. Returns dict(k, v, workspace)."""
    d = _home(pool, "pool", stream)
    P, H, D = _pool(pool, d)
    B, M = _table(table, d)
    _ints(start, "start", (B,), d)
    if counts is not None:
        _ints(counts, "counts", (B,), d)
    if k is None:
        k = _new(torch.empty, stream, (B, n, H, D), dtype=dtype, device=pool.device)
        ki = _own(k)
    else:
        ki = _heads(k, "k", (B, n, H, D), dtype, d)
    if v is None:
        v = _new(torch.empty, stream, (B, n, H, D), dtype=dtype, device=pool.device)
        vi = _own(v)
    else:
        vi = _heads(v, "v", (B, n, H, D), dtype, d)
    code = _code(k, "k")
    if workspace is None:
        workspace = _new(torch.zeros, stream, WS_HEADER, dtype=torch.uint8, device=pool.device)
    _ok(_lib().spec_cache_read(pool.data_ptr(), P, table.data_ptr(), M, start.data_ptr(), _ptr(counts), ki, vi, code, B, n, H, D,
                               *_workspace(workspace, d), _on(d, stream)))
    return dict(k=k, v=v, workspace=workspace)


def cache_attention(q, pool, table, kv_len, *, q_len=None, scale=None, window=0, sinks=0, out=None, lse=None,
                    want_lse=False, workspace=None, stream=None):
    """Attention of the newest tokens q [B, N, Hq, D] (bf16 or fp16) over the cache. kv_len [B] counts every cached
    token, the new ones included; query i of sequence b stands at kv_len[b] - q_len[b] + i (q_len None: N). window > 0
    limits each query to the window last tokens and the first `sinks`. scale: 1 / sqrt(D) unless given. Returns
    dict(out, lse, workspace), lse [B, N, Hq] where wanted."""
    d = _home(q, "q", stream)
    P, H, D = _pool(pool, d)
    B, M = _table(table, d)
    Bq, N, Hq, Dq = q.shape
    code = _code(q, "q")
    if Bq != B or Dq != D:
        raise ValueError("q must have shape %s, got %s" % ((B, N, Hq, D), tuple(q.shape)))
    _ints(kv_len, "kv_len", (B,), d)
    if q_len is not None:
        _ints(q_len, "q_len", (B,), d)
    qi = _rows(q, "q")
    if out is None:
        out, oi = _like(q, stream)
    else:
        oi = _heads(out, "out", (B, N, Hq, D), q.dtype, d)
    if lse is not None:
        _vector(lse, "lse", torch.float32, (B, N, Hq), d)
    elif want_lse:
        lse = _new(torch.empty, stream, (B, N, Hq), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = _new(new_attention_workspace, stream, max(N, 1), Hq, H, D, q.device)
    _ok(_lib().spec_cache_attention(qi, code, pool.data_ptr(), P, table.data_ptr(), M, kv_len.data_ptr(), _ptr(q_len), B, N,
                                    Hq, H, D, D ** -0.5 if scale is None else scale, window, sinks, oi, _ptr(lse),
                                    *_workspace(workspace, d), _on(d, stream)))
    return dict(out=out, lse=lse, workspace=workspace)


def _books(table, lengths, refs, stream):
    d = _home(table, "table", stream)
    S, M = _table(table, d)
    if lengths is not None:
        _ints(lengths, "lengths", (S,), d)
    P = refs.numel()
    _ints(refs, "refs", (P,), d)
    return S, M, P, d


def _layers(pool, P, d):
    """[pages, ...] or [layers, pages, ...] as (layers, bytes of a page)."""
    if not (pool.get_device() == d and pool.dtype is torch.uint8 and pool.is_contiguous()):
        _need(pool, "pool", torch.uint8)
    if pool.dim() not in (3, 4) or pool.shape[-3] != P:
        raise ValueError("pool must be [%d, Hk, 68 D] or [layers, %d, Hk, 68 D], got %s" % (P, P, tuple(pool.shape)))
    return (pool.shape[0] if pool.dim() == 4 else 1), pool.shape[-2] * pool.shape[-1]


def _pages_ws(workspace, S, P, device, stream):
    return _new(new_pages_workspace, stream, S, P, device) if workspace is None else workspace


def pages_fork(table, lengths, refs, src, dst, *, workspace=None, stream=None):
    """Sequence dst[f] becomes a copy of src[f] that shares its pages (int32 [F] each). Returns the workspace."""
    S, M, P, d = _books(table, lengths, refs, stream)
    F = src.numel()
    _ints(src, "src", (F,), d)
    _ints(dst, "dst", (F,), d)
    ws = _pages_ws(workspace, S, P, table.device, stream)
    _ok(_lib().spec_pages_fork(table.data_ptr(), _ptr(lengths), refs.data_ptr(), S, M, P, src.data_ptr(), dst.data_ptr(), F,
                               *_workspace(ws, d), _on(d, stream)))
    return ws


def pages_reserve(pool, table, lengths, refs, n_new, *, served=None, workspace=None, stream=None):
    """Pages of its own for each sequence's next n_new[s] tokens; a shared part-filled page is copied in every layer of
    pool. Returns served, int32 [sequences]: 0 where there was no room."""
    S, M, P, d = _books(table, lengths, refs, stream)
    layers, page_bytes = _layers(pool, P, d)
    _ints(n_new, "n_new", (S,), d)
    if served is None:
        served = _new(torch.empty, stream, S, dtype=torch.int32, device=table.device)
    else:
        _ints(served, "served", (S,), d)
    ws = _pages_ws(workspace, S, P, table.device, stream)
    _ok(_lib().spec_pages_reserve(pool.data_ptr(), layers, page_bytes, table.data_ptr(), _ptr(lengths), refs.data_ptr(), S, M, P,
                                  n_new.data_ptr(), served.data_ptr(), *_workspace(ws, d), _on(d, stream)))
    return served


def pages_commit(table, lengths, refs, advance, *, extra=1, window=0, sinks=0, workspace=None, stream=None):
    """lengths += advance + extra (a verification's accept_len and the token before the drafts); pages past the new
    lengths, or with window > 0 out of every later query's view, are let go. Returns the workspace."""
    S, M, P, d = _books(table, lengths, refs, stream)
    _ints(advance, "advance", (S,), d)
    ws = _pages_ws(workspace, S, P, table.device, stream)
    _ok(_lib().spec_pages_commit(table.data_ptr(), _ptr(lengths), refs.data_ptr(), S, M, P, advance.data_ptr(), extra, window,
                                 sinks, *_workspace(ws, d), _on(d, stream)))
    return ws


def pages_release(table, lengths, refs, slots, *, workspace=None, stream=None):
    """Lets go of every page of the sequences slots (int32 [F]). Returns the workspace."""
    S, M, P, d = _books(table, lengths, refs, stream)
    F = slots.numel()
    _ints(slots, "slots", (F,), d)
    ws = _pages_ws(workspace, S, P, table.device, stream)
    _ok(_lib().spec_pages_release(table.data_ptr(), _ptr(lengths), refs.data_ptr(), S, M, P, slots.data_ptr(), F,
                                  *_workspace(ws, d), _on(d, stream)))
    return ws


def pages_compact(pool, table, refs, *, used=None, workspace=None, stream=None):
    """Moves the pages in use to the front of the pool, in every layer; table and refs follow. Returns used, int32 [1]:
    how many there are."""
    S, M, P, d = _books(table, None, refs, stream)
    layers, page_bytes = _layers(pool, P, d)
    if used is None:
        used = _new(torch.empty, stream, 1, dtype=torch.int32, device=table.device)
    else:
        _ints(used, "used", (1,), d)
    ws = _pages_ws(workspace, S, P, table.device, stream)
    _ok(_lib().spec_pages_compact(pool.data_ptr(), layers, page_bytes, table.data_ptr(), refs.data_ptr(), S, M, P, used.data_ptr(),
                                  *_workspace(ws, d), _on(d, stream)))
    return used
