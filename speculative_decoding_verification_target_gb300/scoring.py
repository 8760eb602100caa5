"""Operators between the target's last layer and a verification: binding of the C ABI in include/specscore.h.

Argument marshalling only, as for the other calls; the header states every rule. What a serving loop runs on the tokens
that it is about to verify:

    residual_norm(x, residual, weight, quantize=True)      x + residual, its norm, in 8 bits with a scale per token
    int8_matmul(codes, scale, w, w_scale)                  the vocabulary's product (w, w_scale: quantize_rows of the weights)
    process_logits(logits, tokens=..., history=..., ...)   biases, penalties for repeated tokens, grammar masks
    verify(logits, ...)

Activations, codes and logits are [rows, values] or [B, N, values] with any strides but contiguous values. Every tensor of a
call is on the current device. A call runs on `stream`, or on the current one. Outputs and workspaces that are not given are
made on that stream; what is given has to be ready on it. The product's status word is in its workspace (read_status). No call
records gradients: outputs are detached, also from inputs that require them.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import SPEC_OK, SpecError, _current_device, _need, _new, load as _load
from .cache import _DTYPES, _code, _home, _on, _raw_stream, _vector, _workspace

WS_HEADER = 256
INT8 = 3
SCORE_EXPORTS = ("spec_residual_norm", "spec_quantize_rows", "spec_int8_matmul_workspace_size", "spec_int8_matmul",
                 "spec_process_logits", "spec_score_last_error")


class Rows(ctypes.Structure):
    """spec_rows: [B, N] rows in device memory, element strides over both."""
    _fields_ = [("data", ctypes.c_void_p), ("stride_b", ctypes.c_longlong), ("stride_n", ctypes.c_longlong)]


@functools.cache
def _lib():
    lib = _load()
    P, I, F, Z, L = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_longlong
    R = ctypes.POINTER(Rows)
    for name, res, args in (
            ("spec_residual_norm", I, [R, R, I, I, I, I, P, F, R, R, I, P, P]),
            ("spec_quantize_rows", I, [R, I, I, I, I, R, P, P]),
            ("spec_int8_matmul_workspace_size", Z, [I, I, I]),
            ("spec_int8_matmul", I, [R, P, P, L, P, P, I, I, I, I, R, I, P, Z, P]),
            ("spec_process_logits", I, [R, I, I, I, I, P, I, P, P, P, I, P, P, P, P, P, I, P, L, L, R, P]),
            ("spec_score_last_error", ctypes.c_char_p, [])):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args
    return lib


def _ok(code):
    if code != SPEC_OK:
        raise SpecError(code, _lib().spec_score_last_error().decode())


# A serving loop makes these calls for every few tokens, where the host takes longer than the device: what passes is looked at in one
# condition, and functions are called for what does not.
def _rows(t, name):
    """[rows, values] or [B, N, values] as (B, N, values) and its rows; type and device known."""
    shape, strides = t.shape, t.stride()
    if len(shape) == 2:
        N, D = shape
        sn, sd = strides
        B, sb = 1, 0
    elif len(shape) == 3:
        B, N, D = shape
        sb, sn, sd = strides
    else:
        raise ValueError("%s must be [rows, values] or [B, N, values], got %s" % (name, tuple(shape)))
    if sd != 1 and D > 1:
        raise ValueError("%s must have contiguous values" % name)
    return B, N, D, Rows(t.data_ptr(), sb, sn)


def _rows_like(t, name, shape, dtype, d):
    """The rows of t, whose shape, type and device are checked."""
    if not (t.get_device() == d and t.dtype is dtype and t.shape == shape):
        if not t.is_cuda:
            raise ValueError("%s must be a CUDA tensor" % name)
        if t.dtype is not dtype:
            raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
        if t.shape != shape:
            raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
        raise ValueError("%s must be on cuda:%d, got cuda:%d" % (name, d, t.get_device()))
    return _rows(t, name)[3]


def _make(shape, dtype, device, stream):
    """A new output, and its rows."""
    t = torch.empty(shape, dtype=dtype, device=device) if stream is None else _new(torch.empty, stream, shape, dtype=dtype, device=device)
    n = shape[-1]
    return t, Rows(t.data_ptr(), n * shape[-2], n)


def _scales(t, shape, d, device, stream):
    if t is not None:
        _vector(t, "scale", torch.float32, shape, d)
        return t
    if stream is None:
        return torch.empty(shape, dtype=torch.float32, device=device)
    return _new(torch.empty, stream, shape, dtype=torch.float32, device=device)


def _device_of(t, name, stream):
    """The device of a call: the current one, where t is and the stream."""
    d = t.get_device()
    return d if stream is None and d >= 0 and d == _current_device() else _home(t, name, stream)


def _handle(d, stream):
    return _raw_stream(d) if stream is None and _raw_stream is not None else _on(d, stream)


def residual_norm(x, residual=None, weight=None, eps=1e-6, *, quantize=False, out=None, scale=None, residual_out=None,
                  stream=None):
    """r = x + residual and its root-mean-square norm times a weight [D], in x's type (bf16, fp16 or fp32) or, with quantize, in
    8 bits with a scale per token. residual_out may be x or residual, out (not in 8 bits) may be the other one. Returns dict(out,
    scale, residual); scale is None without quantize, residual without a residual."""
    shape, dt = x.shape, x.dtype
    code = _code(x, "x", True)
    d = _device_of(x, "x", stream)
    B, N, D, xi = _rows(x, "x")
    ri = ro = w = sp = None
    if residual is not None:
        ri = _rows_like(residual, "residual", shape, dt, d)
        if residual_out is None:
            residual_out, ro = _make(shape, dt, x.device, stream)
        else:
            ro = _rows_like(residual_out, "residual_out", shape, dt, d)
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    if weight is not None:
        _vector(weight, "weight", dt, (D,), d)
        w = weight.data_ptr()
    if quantize:
        scale = _scales(scale, shape[:-1], d, x.device, stream)
        sp = scale.data_ptr()
    elif scale is not None:
        raise ValueError("scale needs quantize")
    if out is None:
        out, oi = _make(shape, torch.int8 if quantize else dt, x.device, stream)
    else:
        oi = _rows_like(out, "out", shape, torch.int8 if quantize else dt, d)
    _ok(_lib().spec_residual_norm(xi, ri, code, B, N, D, w, eps, ro, oi, INT8 if quantize else code, sp, _handle(d, stream)))
    return dict(out=out, scale=scale, residual=residual_out)


def quantize_rows(x, *, out=None, scale=None, stream=None):
    """Each row of x (bf16, fp16 or fp32) in 8 bits: code = the integer nearest to 127 x / m, scale = m / 127, m the row's largest
    magnitude. For weights [C, K] once, for activations each time. Returns dict(out, scale)."""
    code = _code(x, "x", True)
    d = _device_of(x, "x", stream)
    B, N, D, xi = _rows(x, "x")
    shape = x.shape
    scale = _scales(scale, shape[:-1], d, x.device, stream)
    if out is None:
        out, oi = _make(shape, torch.int8, x.device, stream)
    else:
        oi = _rows_like(out, "out", shape, torch.int8, d)
    _ok(_lib().spec_quantize_rows(xi, code, B, N, D, oi, scale.data_ptr(), _handle(d, stream)))
    return dict(out=out, scale=scale)


def new_matmul_workspace(tokens, C, K, device=None):
    """Workspace of int8_matmul for up to these sizes, ready for its first use."""
    n = int(_lib().spec_int8_matmul_workspace_size(tokens, C, K))
    if n == 0:
        raise ValueError("unsupported sizes tokens=%d C=%d K=%d" % (tokens, C, K))
    if n <= 1 << 16:
        return torch.zeros(n, dtype=torch.uint8, device="cuda" if device is None else device)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda" if device is None else device)
    ws[:WS_HEADER].zero_()
    return ws


def int8_matmul(a, a_scale, w, w_scale, *, bias=None, dtype=torch.bfloat16, out=None, workspace=None, stream=None):
    """a [tokens, K] or [B, N, K] times w [C, K], both int8, with scales for each token and each channel and a bias (float32)
    [C]: the sum in integers, exactly, then scaled and rounded to dtype (bf16, fp16 or fp32). Returns dict(out, workspace)."""
    if a.dtype is not torch.int8:
        raise TypeError("a must be torch.int8, got %s" % a.dtype)
    d = _device_of(a, "a", stream)
    B, N, K, ai = _rows(a, "a")
    size, strides = w.shape, w.stride()
    if len(size) != 2:
        raise ValueError("w must be [C, K], got %s" % (tuple(size),))
    C = size[0]
    if not (size[1] == K and w.dtype is torch.int8 and w.get_device() == d and (strides[1] == 1 or K == 1)):
        _rows_like(w, "w", (C, K), torch.int8, d)
    tokens = a.shape[:-1]
    _vector(a_scale, "a_scale", torch.float32, tokens, d)
    _vector(w_scale, "w_scale", torch.float32, (C,), d)
    bp = None
    if bias is not None:
        _vector(bias, "bias", torch.float32, (C,), d)
        bp = bias.data_ptr()
    if out is not None:
        dtype = out.dtype
    code = _DTYPES.get(dtype)
    if code is None:
        raise TypeError("out must be bfloat16, float16 or float32, got %s" % dtype)
    if out is None:
        out, oi = _make(tokens + (C,), dtype, a.device, stream)
    else:
        oi = _rows_like(out, "out", tokens + (C,), dtype, d)
    if workspace is None:
        workspace = _new(new_matmul_workspace, stream, max(B * N, 1), C, K, a.device)
    wp, held = _workspace(workspace, d)
    _ok(_lib().spec_int8_matmul(ai, a_scale.data_ptr(), w.data_ptr(), strides[0], w_scale.data_ptr(), bp, B, N, C, K, oi, code, wp, held,
                                _handle(d, stream)))
    return dict(out=out, workspace=workspace)


def _ints(t, name, shape, d):
    if not (t.get_device() == d and t.dtype is torch.int32 and t.shape == shape and t.is_contiguous()):
        _need(t, name, torch.int32, shape)
    return t.data_ptr()


def process_logits(logits, *, tokens=None, history=None, lengths=None, prompt=None, repetition=None, frequency=None,
                   presence=None, bias_tokens=None, bias=None, mask=None, out=None, stream=None):
    """Logits [B, R, V] (bf16 or fp32) as they are sampled from: biases (bias_tokens int32 [B, n], bias float32 [B, n]), the
    penalties repetition, frequency and presence (float32 [B]) over each sequence's history (int32 [B, L], with lengths and, if part
    of it is a prompt, prompt, int32 [B]) and the drafts before a row (tokens int32 [B, T], T >= R - 1), and a grammar's mask (int32 [B, R, ceil(V / 32)],
    or expanded to it). out may be logits. Returns dict(out)."""
    if logits.dim() != 3:
        raise ValueError("logits must be [B, R, V], got %s" % (tuple(logits.shape),))
    code = _code(logits, "logits", True)
    d = _device_of(logits, "logits", stream)
    B, R, V, xi = _rows(logits, "logits")
    T = L = n = 0
    tp = hp = lp = pp = bt = bp = mp = None
    sb = sr = 0
    if tokens is not None:
        T = tokens.shape[-1]
        tp = _ints(tokens, "tokens", (B, T), d)
    if history is not None:
        L = history.shape[-1]
        hp = _ints(history, "history", (B, L), d)
        if lengths is None:
            raise ValueError("history needs lengths")
        lp = _ints(lengths, "lengths", (B,), d)
        pp = None if prompt is None else _ints(prompt, "prompt", (B,), d)
    elif lengths is not None or prompt is not None:
        raise ValueError("%s needs history" % ("prompt" if lengths is None else "lengths"))
    rates = []
    for t, name in ((repetition, "repetition"), (frequency, "frequency"), (presence, "presence")):
        if t is not None:
            _vector(t, name, torch.float32, (B,), d)
        rates.append(None if t is None else t.data_ptr())
    if bias_tokens is not None:
        n = bias_tokens.shape[-1]
        bt = _ints(bias_tokens, "bias_tokens", (B, n), d)
        if bias is None:
            raise ValueError("bias_tokens needs bias")
        _vector(bias, "bias", torch.float32, (B, n), d)
        bp = bias.data_ptr()
    elif bias is not None:
        raise ValueError("bias needs bias_tokens")
    if mask is not None:
        mi = _rows_like(mask, "mask", (B, R, (V + 31) // 32), torch.int32, d)
        mp, sb, sr = mi.data, mi.stride_b, mi.stride_n
    if out is None:
        out, oi = _make(logits.shape, logits.dtype, logits.device, stream)
    else:
        oi = _rows_like(out, "out", logits.shape, logits.dtype, d)
    _ok(_lib().spec_process_logits(xi, code, B, R, V, tp, T, hp, lp, pp, L, *rates, bt, bp, n, mp, sb, sr, oi, _handle(d, stream)))
    return dict(out=out)
