"""CPU checks of the operators between the last layer and a verification: exports, refusals of the C ABI before any CUDA call, the
binding around a launch on stand-ins (fake_cuda), and the plain forms of score_util."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import fake_cuda as fc
import score_util as su
import speculative_decoding_verification_target_gb300 as sv
from speculative_decoding_verification_target_gb300 import _build, scoring

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p
I32, BF16, F32, I8, U8 = torch.int32, torch.bfloat16, torch.float32, torch.int8, torch.uint8
INVALID, UNSUPPORTED = 1, 3


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return scoring._lib()


def H(data=1 << 20, b=1 << 16, n=1 << 13):
    return scoring.Rows(data, b, n)


def test_every_declared_symbol_is_exported(lib):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "specscore.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(spec_[a-z0-9_]+)\s*\(", text))
    assert names == set(scoring.SCORE_EXPORTS)
    for n in names:
        assert hasattr(lib, n), n
    assert "SPEC_SCORE_WS_HEADER %d" % scoring.WS_HEADER in text and "SPEC_INT8 = %d" % scoring.INT8 in text


def norm(lib, **kw):
    a = dict(x=H(), res=H(2 << 20), dtype=0, B=2, N=3, D=512, w=1 << 23, eps=1e-6, ro=H(3 << 20), out=H(4 << 20), kind=3, scale=1 << 24)
    a.update(kw)
    return lib.spec_residual_norm(a["x"], a["res"], a["dtype"], a["B"], a["N"], a["D"], P(a["w"]), a["eps"], a["ro"], a["out"],
                                  a["kind"], P(a["scale"]), None)


@pytest.mark.parametrize("kw,code,words", [
    (dict(dtype=3), UNSUPPORTED, "dtype must be"), (dict(dtype=-1), UNSUPPORTED, "dtype must be"), (dict(D=0), UNSUPPORTED, "D must be"),
    (dict(D=32769), UNSUPPORTED, "D must be"), (dict(B=-1), INVALID, "B must be"), (dict(N=-1), INVALID, "N must be"),
    (dict(B=65536), INVALID, "B must be"), (dict(B=60000, N=1 << 10), INVALID, "B N must be"), (dict(eps=-1.0), INVALID, "eps"),
    (dict(eps=float("nan")), INVALID, "eps"), (dict(eps=float("inf")), INVALID, "eps"), (dict(kind=2), UNSUPPORTED, "out_type"),
    (dict(x=None), INVALID, "x must not be NULL"), (dict(x=H(0)), INVALID, "x must not be NULL"), (dict(out=None), INVALID, "out must not"),
    (dict(res=None), INVALID, "come together"), (dict(ro=None), INVALID, "come together"), (dict(scale=None), INVALID, "scale"),
    (dict(x=H((1 << 20) + 1)), INVALID, "multiple of 2"), (dict(w=(1 << 23) + 1), INVALID, "multiple of 2"),
    (dict(out=H(4 << 20, n=511)), INVALID, "rows overlap"), (dict(out=H(4 << 20, b=0)), INVALID, "rows overlap"),
    (dict(ro=H(3 << 20, b=600, n=512)), INVALID, "rows overlap"), (dict(ro=H(3 << 20, n=-100)), INVALID, "rows overlap"),
    (dict(out=H(3 << 20)), INVALID, "out must not be residual_out"), (dict(out=H()), INVALID, "8 bits must not be an input"),
    (dict(out=H(2 << 20)), INVALID, "8 bits must not be an input"), (dict(ro=H(1 << 20, n=1 << 14, b=1 << 17)), INVALID, "have its strides"),
    (dict(kind=0, out=H(2 << 20, b=1 << 17)), INVALID, "have its strides"),
])
def test_norm_refusals(lib, kw, code, words):
    assert norm(lib, **kw) == code and words in lib.spec_score_last_error().decode()


def test_norm_empty_calls_do_nothing(lib):
    assert norm(lib, B=0, x=None, out=None) == 0 and norm(lib, N=0, x=None, out=None) == 0


def quantize(lib, **kw):
    a = dict(x=H(), dtype=0, B=2, N=3, D=512, out=H(4 << 20), scale=1 << 24)
    a.update(kw)
    return lib.spec_quantize_rows(a["x"], a["dtype"], a["B"], a["N"], a["D"], a["out"], P(a["scale"]), None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=3), UNSUPPORTED), (dict(D=0), UNSUPPORTED), (dict(B=-1), INVALID), (dict(x=None), INVALID), (dict(out=None), INVALID),
    (dict(scale=None), INVALID), (dict(out=H(4 << 20, n=100)), INVALID), (dict(out=H()), INVALID), (dict(dtype=1, x=H((1 << 20) + 2)), INVALID),
])
def test_quantize_refusals(lib, kw, code):
    assert quantize(lib, **kw) == code and lib.spec_score_last_error()


def product(lib, **kw):
    a = dict(a=H(), sa=1 << 22, w=1 << 25, ws_=512, sw=1 << 23, bias=0, B=2, N=3, C=100, K=512, out=H(4 << 20), kind=0, ws=1 << 26,
             size=1 << 30)
    a.update(kw)
    return lib.spec_int8_matmul(a["a"], P(a["sa"]), P(a["w"]), a["ws_"], P(a["sw"]), P(a["bias"]), a["B"], a["N"], a["C"], a["K"],
                                a["out"], a["kind"], P(a["ws"]), a["size"], None)


@pytest.mark.parametrize("kw,code,words", [
    (dict(kind=3), UNSUPPORTED, "dtype"), (dict(K=0), UNSUPPORTED, "K must be"), (dict(K=131072), UNSUPPORTED, "K must be"),
    (dict(C=-1), INVALID, "C must be"), (dict(B=-1), INVALID, "B must be"), (dict(a=None), INVALID, "a must not"),
    (dict(w=None), INVALID, "must not be NULL"), (dict(sa=None), INVALID, "must not be NULL"), (dict(sw=None), INVALID, "must not be NULL"),
    (dict(out=H(4 << 20, n=99)), INVALID, "rows overlap"), (dict(ws=None), INVALID, "workspace"), (dict(ws=(1 << 26) + 8), INVALID, "workspace"),
    (dict(size=100), INVALID, "needed"), (dict(ws_=-512), INVALID, "w_stride"), (dict(kind=1, out=H((4 << 20) + 2)), INVALID, "multiple of 4"),
])
def test_product_refusals(lib, kw, code, words):
    assert product(lib, **kw) == code and words in lib.spec_score_last_error().decode()


def test_product_sizes(lib):
    f = lib.spec_int8_matmul_workspace_size
    assert f(1, 1, 0) == 0 and f(1, 1, 131072) == 0 and f(-1, 1, 1) == 0 and f(1, 1 << 21, 1) == 0 and f(0, 0, 1) >= 256
    for K in (1, 16, 500, 512, 4096, 131056):
        for C in (1, 100, 128, 257, 128256):
            sizes = [f(t, C, K) for t in (1, 2, 15, 16, 17, 64, 100, 192, 193, 250, 384, 385, 400, 577, 1000, 8192)]
            assert all(a <= b for a, b in zip(sizes, sizes[1:])) and sizes[0] >= 256
    for t in (1, 100, 1000):
        for axis in (lambda n: f(t, n, 4096), lambda n: f(t, 4096, n)):
            sizes = [axis(n) for n in (1, 15, 16, 17, 127, 128, 129, 255, 512, 1000, 1024, 4095, 4096, 10000, 38913, 130000)]
            assert all(a <= b for a, b in zip(sizes, sizes[1:]))


def logits(lib, **kw):
    a = dict(x=H(), dtype=0, B=2, R=3, V=1000, tokens=1 << 21, T=2, history=1 << 22, lengths=1 << 23, prompt=0, L=10, rep=0, freq=0,
             pres=0, bt=1 << 24, bias=1 << 24, n=4, mask=0, sb=0, sr=0, out=H(4 << 20))
    a.update(kw)
    return lib.spec_process_logits(a["x"], a["dtype"], a["B"], a["R"], a["V"], P(a["tokens"]), a["T"], P(a["history"]), P(a["lengths"]),
                                   P(a["prompt"]), a["L"], P(a["rep"]), P(a["freq"]), P(a["pres"]), P(a["bt"]), P(a["bias"]), a["n"],
                                   P(a["mask"]), a["sb"], a["sr"], a["out"], None)


@pytest.mark.parametrize("kw,code,words", [
    (dict(dtype=2), UNSUPPORTED, "dtype"), (dict(B=-1), INVALID, "B must be"), (dict(R=-1), INVALID, "R must be"), (dict(R=66), INVALID, "R must be"),
    (dict(V=0), INVALID, "V must be"), (dict(V=262145), INVALID, "V must be"), (dict(L=-1), INVALID, "L must be"),
    (dict(L=1000001), INVALID, "L must be"), (dict(n=1025), INVALID, "biases"), (dict(n=-1), INVALID, "biases"),
    (dict(x=None), INVALID, "logits must not"), (dict(out=None), INVALID, "out must not"), (dict(T=1), INVALID, "tokens"),
    (dict(lengths=None), INVALID, "lengths"), (dict(bias=None), INVALID, "bias must not"), (dict(out=H(4 << 20, n=999)), INVALID, "rows overlap"),
    (dict(out=H(1 << 20, b=1 << 17)), INVALID, "have its strides"), (dict(dtype=1, x=H((1 << 20) + 2)), INVALID, "multiple of 4"),
])
def test_logits_refusals(lib, kw, code, words):
    assert logits(lib, **kw) == code and words in lib.spec_score_last_error().decode()


@pytest.mark.parametrize("call,name,off", [(norm, "scale", 2), (quantize, "scale", 1), (product, "sa", 3), (product, "sw", 2), (product, "bias", 2)]
                         + [(logits, n, 2) for n in ("tokens", "history", "lengths", "prompt", "rep", "freq", "pres", "bt", "bias", "mask")])
def test_pointers_off_their_words_are_refused(lib, call, name, off):
    assert call(lib, **{name: (1 << 27) + off}) == INVALID and "multiple of 4 bytes" in lib.spec_score_last_error().decode()


THREADS = r"""
#include "norm_threads.h"
extern "C" void threads(long long rows, int pieces, int vec, int codes, int full, int sms, int* out) {
    const specs::NormThreads t = specs::norm_threads(rows, pieces, vec, codes, full, sms);
    out[0] = t.slots, out[1] = t.tpr, out[2] = t.per, out[3] = static_cast<int>(t.room);
}
"""


@pytest.fixture(scope="module")
def threads(tmp_path_factory):
    d = tmp_path_factory.mktemp("threads")
    (d / "threads.cpp").write_text(THREADS)
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I", _build.SCORE, "-o", str(d / "threads.so"), str(d / "threads.cpp")], check=True)
    fn = ctypes.CDLL(str(d / "threads.so")).threads
    fn.argtypes, fn.restype = [ctypes.c_longlong] + [ctypes.c_int] * 5 + [ctypes.POINTER(ctypes.c_int)], None

    def call(*a):
        out = (ctypes.c_int * 4)()
        fn(*a, out)
        return tuple(out)
    return call


@pytest.mark.parametrize("sms", [152, 148])
def test_threads_of_a_row(threads, sms):
    """Each choice is one that a kernel stands behind; rows for codes whose places of two pieces a thread fit side by side have those."""
    for full, room in ((1, 512), (0, 1024)):
        for pieces in (1, 2, 31, 32, 33, 64, 100, 128, 255, 256, 257, 511, 512, 513, 1000, 1024, 1025, 2048):
            row = ((pieces + 1) // 2 + 31) // 32 * 32
            most = room * sms // row
            for rows in {1, 2, most // 2 + 1, most - 1, most, most + 1, 4 * sms, 4 * sms + 1, 10 * most + 7}:
                for codes in (0, 1):
                    slots, tpr, per, got = threads(max(rows, 1), pieces, 1, codes, full, sms)
                    assert slots in (1, 2, 4) and tpr % 32 == 0 and slots * tpr >= pieces and tpr * per <= 512 and got == room
                    assert slots * (tpr - 32) < pieces
                    if codes and pieces <= 1024 and rows <= most:
                        assert slots <= 2, (rows, pieces)
                    if rows > most:
                        assert slots == 4 or pieces <= 32 or rows * tpr <= room * sms
        for pieces in (1, 33, 261, 512, 2048, 2049, 4097, 8192):
            for rows in (1, 100, 5000):
                slots, tpr, per, _ = threads(rows, pieces, 0, 1, full, sms)
                assert slots in (4, 16) and tpr % 32 == 0 and slots * tpr >= pieces and tpr * per <= 512


# ------------------------------------------------------------------------------------ the binding, on stand-ins
B, N, D, C, V, L = 3, 2, 64, 40, 100, 7


class Args:
    def __init__(self, index=0):
        t = lambda shape, dtype=F32: fc.Tensor(shape, dtype, index)  # noqa: E731
        self.x, self.residual, self.weight = t((B, N, D), BF16), t((B, N, D), BF16), t((D,), BF16)
        self.a, self.a_scale, self.w, self.w_scale, self.bias = t((B, N, D), I8), t((B, N)), t((C, D), I8), t((C,)), t((C,))
        self.logits, self.tokens, self.history, self.lengths, self.prompt = t((B, N, V)), t((B, N), I32), t((B, L), I32), t((B,), I32), t((B,), I32)
        self.repetition, self.frequency, self.presence = t((B,)), t((B,)), t((B,))
        self.bias_tokens, self.biases, self.mask = t((B, 5), I32), t((B, 5)), t((B, N, 4), I32)


CALLS = {
    "residual_norm": lambda a, **kw: sv.residual_norm(a.x, a.residual, a.weight, quantize=True, **kw),
    "quantize_rows": lambda a, **kw: sv.quantize_rows(a.x, **kw),
    "int8_matmul": lambda a, **kw: sv.int8_matmul(a.a, a.a_scale, a.w, a.w_scale, bias=a.bias, **kw),
    "process_logits": lambda a, **kw: sv.process_logits(
        a.logits, tokens=a.tokens, history=a.history, lengths=a.lengths, prompt=a.prompt, repetition=a.repetition, frequency=a.frequency,
        presence=a.presence, bias_tokens=a.bias_tokens, bias=a.biases, mask=a.mask, **kw),
}
LOOKED_AT = {"residual_norm": "residual weight", "quantize_rows": "", "int8_matmul": "a_scale w w_scale bias",
             "process_logits": "tokens history lengths prompt repetition frequency presence bias_tokens biases mask"}


@pytest.fixture
def fake(monkeypatch):
    t, lib = fc.install(monkeypatch, sv)
    monkeypatch.setattr(scoring, "torch", t)
    monkeypatch.setattr(scoring, "_lib", lambda: lib)
    monkeypatch.setattr(scoring, "_raw_stream", None)
    monkeypatch.setattr(scoring, "_current_device", t.cuda.current_device)
    return t, lib


@pytest.mark.parametrize("name", CALLS)
def test_what_a_call_makes_is_made_on_its_stream(fake, name):
    t, lib = fake
    here, s = t.cuda.now, fc.Stream("given")
    CALLS[name](Args(), stream=s)
    assert t.made and all(x.made_on is s and x.used_on == [here] for x in t.made)
    assert lib.calls[-1][1][-1] == s.cuda_stream and t.cuda.now is here
    del t.made[:]
    CALLS[name](Args())
    assert all(x.made_on is here and x.used_on == [] for x in t.made) and lib.calls[-1][1][-1] == here.cuda_stream


@pytest.mark.parametrize("where,words", [(1, "must be on cuda:0, got cuda:1"), (-1, "must be a CUDA tensor")])
@pytest.mark.parametrize("name,which", [(n, w) for n, ws in LOOKED_AT.items() for w in ws.split()])
def test_every_argument_is_on_the_call_s_device(fake, name, which, where, words):
    a = Args()
    getattr(a, which).index = where
    with pytest.raises(ValueError, match=words):
        CALLS[name](a)
    assert fake[1].calls == []


@pytest.mark.parametrize("name", CALLS)
def test_other_devices_and_their_streams_are_refused(fake, name):
    with pytest.raises(ValueError, match="is on cuda:1, the current device is cuda:0"):
        CALLS[name](Args(1))
    with pytest.raises(ValueError, match="is on cuda:0, the stream on cuda:1"):
        CALLS[name](Args(), stream=fc.Stream("far", 1))
    assert fake[1].calls == []


@pytest.mark.parametrize("name,given,shape,dtype", [
    ("residual_norm", "out", (B, N, D), I8), ("residual_norm", "scale", (B, N), F32), ("residual_norm", "residual_out", (B, N, D), BF16),
    ("quantize_rows", "out", (B, N, D), I8), ("quantize_rows", "scale", (B, N), F32), ("int8_matmul", "out", (B, N, C), BF16),
    ("int8_matmul", "workspace", (1 << 16,), U8), ("process_logits", "out", (B, N, V), F32),
])
def test_outputs_and_workspaces_given(fake, name, given, shape, dtype):
    CALLS[name](Args(), **{given: fc.Tensor(shape, dtype)})
    del fake[1].calls[:]
    for where in (-1, 1):
        with pytest.raises(ValueError, match="CUDA tensor" if where < 0 else "must be on cuda:0, got cuda:1"):
            CALLS[name](Args(), **{given: fc.Tensor(shape, dtype, where)})
    with pytest.raises((TypeError, ValueError)):
        CALLS[name](Args(), **{given: fc.Tensor(shape, torch.float64)})
    if given != "workspace":
        with pytest.raises(ValueError):
            CALLS[name](Args(), **{given: fc.Tensor((shape[0] + 1,) + shape[1:], dtype)})
    assert fake[1].calls == []


@pytest.mark.parametrize("call,error,words", [
    (lambda a: sv.residual_norm(fc.Tensor((2, 64), torch.float64)), TypeError, "x must be"),
    (lambda a: sv.residual_norm(fc.Tensor((64,), BF16)), ValueError, "rows, values"),
    (lambda a: sv.residual_norm(fc.Tensor((2, 64), BF16, strides=(128, 2))), ValueError, "contiguous values"),
    (lambda a: sv.residual_norm(a.x, residual_out=a.residual), ValueError, "needs a residual"),
    (lambda a: sv.residual_norm(a.x, scale=a.a_scale), ValueError, "needs quantize"),
    (lambda a: sv.residual_norm(a.x, fc.Tensor((B, N, D), F32)), TypeError, "residual must be"),
    (lambda a: sv.residual_norm(a.x, None, fc.Tensor((D + 1,), BF16)), ValueError, "weight"),
    (lambda a: sv.int8_matmul(a.x, a.a_scale, a.w, a.w_scale), TypeError, "a must be"),
    (lambda a: sv.int8_matmul(a.a, a.a_scale, fc.Tensor((C, D + 1), I8), a.w_scale), ValueError, "w must have"),
    (lambda a: sv.int8_matmul(a.a, a.a_scale, fc.Tensor((C, D), U8), a.w_scale), TypeError, "w must be"),
    (lambda a: sv.int8_matmul(a.a, a.a_scale, fc.Tensor((C,), I8), a.w_scale), ValueError, "w must be"),
    (lambda a: sv.int8_matmul(a.a, a.w_scale, a.w, a.w_scale), ValueError, "a_scale"),
    (lambda a: sv.int8_matmul(a.a, a.a_scale, a.w, a.w_scale, dtype=torch.float64), TypeError, "out must be"),
    (lambda a: sv.process_logits(fc.Tensor((2, 100), F32)), ValueError, "logits must be"),
    (lambda a: sv.process_logits(a.logits, history=a.history), ValueError, "needs lengths"),
    (lambda a: sv.process_logits(a.logits, bias_tokens=a.bias_tokens), ValueError, "needs bias"),
    (lambda a: sv.process_logits(a.logits, mask=fc.Tensor((B, N, 3), I32)), ValueError, "mask must have"),
    (lambda a: sv.process_logits(a.logits, mask=fc.Tensor((B, N, 4), torch.int64)), TypeError, "mask must be"),
    (lambda a: sv.process_logits(a.logits, tokens=fc.Tensor((B + 1, 2), I32)), ValueError, "tokens"),
])
def test_binding_refusals(fake, call, error, words):
    with pytest.raises(error, match=words):
        call(Args())
    assert fake[1].calls == []


@pytest.mark.parametrize("alone,partner", [("bias", "bias_tokens"), ("lengths", "history"), ("prompt", "history")])
def test_what_says_nothing_without_its_partner_is_refused(fake, alone, partner):
    a = Args()
    given = dict(bias=a.biases, lengths=a.lengths, prompt=a.prompt)
    with pytest.raises(ValueError, match="%s needs %s" % (alone, partner)):
        sv.process_logits(a.logits, tokens=a.tokens, **{alone: given[alone]})
    assert fake[1].calls == []


def test_a_mask_may_be_expanded(fake):
    sv.process_logits(Args().logits, mask=fc.Tensor((B, N, 4), I32, strides=(0, 0, 1)))
    assert fake[1].calls[-1][1][-5:-2] == (fake[1].calls[-1][1][-5], 0, 0)


@pytest.mark.parametrize("new", [lambda **kw: sv.new_matmul_workspace(4, 4, 16, **kw), lambda **kw: sv.new_workspace(2, 3, 64, **kw),
                                 lambda **kw: sv.new_pool(3, 2, 64, **kw), lambda **kw: sv.new_attention_workspace(1, 8, 2, 64, **kw),
                                 lambda **kw: sv.new_pages_workspace(2, 3, **kw), lambda **kw: sv.HedgeFeedback(2, 3, 4, **kw)])
def test_a_device_may_be_named_by_its_number(fake, new):
    """The first one too, while another is the current one."""
    t = fake[0]
    t.cuda.device_index = 1
    for device, index in ((0, 0), (1, 1), (None, 1)):
        del t.made[:]
        new(device=device)
        assert t.made and all(x.index == index for x in t.made)


# --------------------------------------------------------------------------------------------- the plain forms
def test_exact_codes_against_fractions():
    from fractions import Fraction
    g = torch.Generator().manual_seed(0)
    p = torch.cat([(torch.randn(20, 40, generator=g)).bfloat16().float(), torch.cat([torch.full((1, 1), 254.0), torch.arange(-39.0, 39, 2)[None]], 1)])
    codes, s = su.exact_codes(p)
    for row, got, sc in zip(p.tolist(), codes.tolist(), s.tolist()):
        m = max(abs(Fraction(v)) for v in row)
        assert got == [round(127 * Fraction(v) / m) for v in row]      # Python rounds fractions half to even
        assert abs(sc - float(m / 127)) <= 2e-16 * sc


def test_plain_logits_by_hand():
    x = torch.tensor([[[1.0, -1.0, 2.0, 0.0], [1.0, -1.0, 2.0, 0.0]]])
    i = lambda *v: torch.tensor([v], dtype=I32)  # noqa: E731
    out, _, same = su.logits(x, tokens=i(2), history=i(0, 1, 1, 9), lengths=i(4)[0], prompt=i(1)[0], repetition=torch.tensor([2.0]),
                             frequency=torch.tensor([0.5]), presence=torch.tensor([0.25]), bias_tokens=i(3, 3), bias=torch.tensor([[7.0, 1.0]]),
                             mask=torch.tensor([[[15], [13]]], dtype=I32))
    assert out[0, 0].tolist() == [0.5, -2 - 1.25, 2.0, 1.0]
    assert out[0, 1].tolist() == [0.5, -torch.inf, 1 - 0.75, 1.0]
    assert same[0].tolist() == [[False, False, True, False], [False, False, False, False]]
