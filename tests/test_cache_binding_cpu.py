"""CPU checks of what the cache's binding does around a launch, on stand-ins for CUDA tensors and streams (fake_cuda)."""
import ctypes

import pytest
import torch

import fake_cuda as fc
import speculative_decoding_verification_target_gb300 as sv

I32, BF16, U8 = torch.int32, torch.bfloat16, torch.uint8
S, M, P, B, N, HQ, HK, D = 3, 4, 9, 3, 2, 8, 2, 64


class Args:
    """Arguments of every call, on one device."""

    def __init__(self, index=0):
        t = lambda shape, dtype=I32: fc.Tensor(shape, dtype, index)  # noqa: E731
        self.q, self.k, self.v = t((B, N, HQ, D), BF16), t((B, N, HK, D), BF16), t((B, N, HK, D), BF16)
        self.positions, self.freqs = t((B, N)), t((D // 2,), torch.int64)
        self.pool, self.table, self.lengths, self.refs = t((P, HK, 68 * D), U8), t((S, M)), t((S,)), t((P,))
        self.n, self.pairs, self.workspace = t((S,)), t((2,)), t((1 << 15,), U8)
        self.q_weight, self.lse, self.served = t((D,), BF16), t((B, N, HQ), torch.float32), t((S,))


CALLS = {
    "qk_norm_rope": lambda a, **kw: sv.qk_norm_rope(a.q, a.k, a.positions, a.freqs, q_weight=a.q_weight, **kw),
    "cache_append": lambda a, **kw: sv.cache_append(a.pool, a.table, a.lengths, a.k, a.v, counts=a.n, **kw),
    "cache_read": lambda a, **kw: sv.cache_read(a.pool, a.table, a.lengths, 5, **kw),
    "cache_attention": lambda a, **kw: sv.cache_attention(a.q, a.pool, a.table, a.lengths, q_len=a.n, want_lse=True, **kw),
    "pages_fork": lambda a, **kw: sv.pages_fork(a.table, a.lengths, a.refs, a.pairs, a.pairs, **kw),
    "pages_reserve": lambda a, **kw: sv.pages_reserve(a.pool, a.table, a.lengths, a.refs, a.n, **kw),
    "pages_commit": lambda a, **kw: sv.pages_commit(a.table, a.lengths, a.refs, a.n, **kw),
    "pages_release": lambda a, **kw: sv.pages_release(a.table, a.lengths, a.refs, a.pairs, **kw),
    "pages_compact": lambda a, **kw: sv.pages_compact(a.pool, a.table, a.refs, **kw),
}
WITH_WORKSPACE = [n for n in CALLS if n != "qk_norm_rope"]


@pytest.fixture
def fake(monkeypatch):
    return fc.install(monkeypatch, sv)


def launch_stream(lib):
    """The stream of the last call: the C ABI's last argument."""
    s = lib.calls[-1][1][-1]
    return s.value if isinstance(s, ctypes.c_void_p) else s


@pytest.mark.parametrize("name", CALLS)
def test_what_a_call_makes_is_made_on_its_stream(fake, name):
    """Outputs and the workspace are cleared and owned in the order of the stream that the kernel runs on; before the
    allocator may give their memory away, it waits for the current stream too, where the caller may read them."""
    t, lib = fake
    here, s = t.cuda.now, fc.Stream("given")
    CALLS[name](Args(), stream=s)
    assert t.made and all(x.made_on is s for x in t.made)
    assert all(x.used_on == [here] for x in t.made)
    assert launch_stream(lib) == s.cuda_stream and t.cuda.now is here


@pytest.mark.parametrize("name", CALLS)
def test_without_a_stream_the_current_one_serves(fake, name):
    t, lib = fake
    CALLS[name](Args())
    assert all(x.made_on is t.cuda.now and x.used_on == [] for x in t.made)
    assert launch_stream(lib) == t.cuda.now.cuda_stream


@pytest.mark.parametrize("name", CALLS)
def test_the_current_stream_may_be_given(fake, name):
    t, lib = fake
    CALLS[name](Args(), stream=t.cuda.now)
    assert all(x.made_on is t.cuda.now and x.used_on == [] for x in t.made)


@pytest.mark.parametrize("name", WITH_WORKSPACE)
def test_a_workspace_made_for_a_call_is_clear_and_one_given_is_used(fake, name):
    t, lib = fake
    CALLS[name](Args())
    made = [x for x in t.made if x.dtype is U8]
    assert len(made) == 1 and made[0].clear
    del t.made[:]
    CALLS[name](Args(), workspace=fc.Tensor((1 << 16,), U8))
    assert not [x for x in t.made if x.dtype is U8] and 1 << 16 in lib.calls[-1][1]


# the arguments that each call looks at, beside its first one
LOOKED_AT = {
    "qk_norm_rope": "k positions freqs q_weight", "cache_append": "table lengths k v n", "cache_read": "table lengths",
    "cache_attention": "pool table lengths n", "pages_fork": "lengths refs pairs", "pages_reserve": "pool lengths refs n",
    "pages_commit": "lengths refs n", "pages_release": "lengths refs pairs", "pages_compact": "pool refs",
}


@pytest.mark.parametrize("where,words", [(1, "must be on cuda:0, got cuda:1"), (-1, "must be a CUDA tensor")])
@pytest.mark.parametrize("name,which", [(n, w) for n, ws in LOOKED_AT.items() for w in ws.split()])
def test_every_argument_is_on_the_call_s_device(fake, name, which, where, words):
    _, lib = fake
    a = Args()
    getattr(a, which).index = where
    with pytest.raises(ValueError, match=words):
        CALLS[name](a)
    assert lib.calls == []


@pytest.mark.parametrize("name", CALLS)
def test_tensors_of_another_device_than_the_current_one_are_refused(fake, name):
    _, lib = fake
    with pytest.raises(ValueError, match="is on cuda:1, the current device is cuda:0"):
        CALLS[name](Args(1))
    assert lib.calls == []


@pytest.mark.parametrize("name", CALLS)
def test_a_stream_of_another_device_is_refused(fake, name):
    _, lib = fake
    with pytest.raises(ValueError, match="is on cuda:0, the stream on cuda:1"):
        CALLS[name](Args(), stream=fc.Stream("far", 1))
    assert lib.calls == []


@pytest.mark.parametrize("workspace,error", [
    (fc.Tensor((1 << 15,), U8, -1), ValueError), (fc.Tensor((1 << 15,), U8, 1), ValueError), (fc.Tensor((1 << 15,), I32), TypeError),
    (fc.Tensor((1 << 14,), U8, strides=(2,)), ValueError),
])
@pytest.mark.parametrize("name", WITH_WORKSPACE)
def test_workspaces_that_are_not_device_bytes_are_refused(fake, name, workspace, error):
    _, lib = fake
    with pytest.raises(error):
        CALLS[name](Args(), workspace=workspace)
    assert lib.calls == []


@pytest.mark.parametrize("name,given", [
    ("qk_norm_rope", "q_out"), ("qk_norm_rope", "k_out"), ("cache_read", "k"), ("cache_read", "v"), ("cache_attention", "out"),
    ("cache_attention", "lse"), ("pages_reserve", "served"), ("pages_compact", "used"),
])
@pytest.mark.parametrize("where", [-1, 1])
def test_outputs_elsewhere_are_refused(fake, name, given, where):
    _, lib = fake
    t = {"q_out": ((B, N, HQ, D), BF16), "k_out": ((B, N, HK, D), BF16), "k": ((S, 5, HK, D), BF16), "v": ((S, 5, HK, D), BF16),
         "out": ((B, N, HQ, D), BF16), "lse": ((B, N, HQ), torch.float32), "served": ((S,), I32), "used": ((1,), I32)}[given]
    CALLS[name](Args(), **{given: fc.Tensor(*t)})
    del lib.calls[:]
    with pytest.raises(ValueError, match="CUDA tensor" if where < 0 else "must be on cuda:0, got cuda:1"):
        CALLS[name](Args(), **{given: fc.Tensor(*t, where)})
    assert lib.calls == []


@pytest.mark.parametrize("G,H", [(1, 1), (1, 8), (2, 4), (3, 2), (4, 8), (5, 1), (8, 8), (16, 2), (64, 1), (1024, 1)])
@pytest.mark.parametrize("D", [64, 128])
def test_an_attention_workspace_serves_fewer_tokens_too(G, H, D):
    from speculative_decoding_verification_target_gb300 import _build, cache
    _build.build()
    sizes = [cache._lib().spec_cache_attention_workspace_size(n, G * H, H, D) for n in range(1, 1025)]
    assert sizes[0] > 0 and all(a <= b for a, b in zip(sizes, sizes[1:]))


@pytest.mark.parametrize("kw", [dict(b=0), dict(n=0), dict(h=0), dict(b=64), dict(n=-64), dict(h=120)])
def test_outputs_whose_rows_overlap_are_refused(kw):
    """A stride below D = 128 over more than one entry: rows would overwrite one another. Inputs may repeat."""
    import test_cache_cpu as ct
    from speculative_decoding_verification_target_gb300 import _build, cache
    _build.build()
    lib = cache._lib()
    bad = ct.H(**kw)
    for call in (lambda: ct.norm(lib, qo=bad), lambda: ct.norm(lib, ko=bad), lambda: ct.tokens("spec_cache_read", lib, k=bad),
                 lambda: ct.tokens("spec_cache_read", lib, v=bad), lambda: ct.attend(lib, out=bad)):
        assert call() == 1 and b"rows overlap" in lib.spec_cache_last_error()


def test_attention_of_no_tokens_needs_no_workspace(fake):
    """An empty call does nothing, whether a workspace is given or not."""
    _, lib = fake
    lib.spec_cache_attention_workspace_size = lambda N, *heads: (1 << 15) * (1 <= N <= 1024)
    a = Args()
    a.q = fc.Tensor((B, 0, HQ, D), BF16)
    r = CALLS["cache_attention"](a)
    assert r["out"].shape == (B, 0, HQ, D) and r["lse"].shape == (B, 0, HQ) and r["workspace"].numel() == 1 << 15
    assert len(lib.calls) == 1
    a.q = fc.Tensor((B, 1025, HQ, D), BF16)
    with pytest.raises(ValueError, match="unsupported sizes N=1025"):
        CALLS["cache_attention"](a)


def test_compaction_without_sequences_is_no_empty_call():
    """The pages counted are still to be moved and counted, so the pool is looked at; the other page calls have nothing to do."""
    from speculative_decoding_verification_target_gb300 import _build, cache
    _build.build()
    lib, p = cache._lib(), ctypes.c_void_p(1 << 20)
    assert lib.spec_pages_compact(None, 1, 32, None, p, 0, 4, 8, p, p, 1 << 20, None) == 1
    assert b"pool" in lib.spec_cache_last_error()
    assert lib.spec_pages_compact(p, 1, 32, None, None, 0, 4, 8, p, p, 1 << 20, None) == 1
    assert lib.spec_pages_compact(p, 1, 32, None, p, 0, 4, 8, p, p, 8192, None) == 1
    assert lib.spec_pages_reserve(None, 1, 32, None, None, None, 0, 4, 8, None, None, p, 1 << 20, None) == 0
    assert lib.spec_pages_commit(None, None, None, 0, 4, 8, None, 1, 0, 0, None, 0, None) == 0


@pytest.mark.parametrize("shape,strides", [
    ((1, 2, 1, 64), (1, 0, 0)), ((2, 1, 3, 64), (64, 1, 0)), ((1, 3, 2, 64), (1, 128, 0)), ((2, 3, 4, 64), (0, 0, 0)),
    ((1, 1, 2, 64), (128, 1, 0)), ((2, 3, 4, 64), (768, 0, 64)),
])
def test_outputs_of_broadcast_inputs_have_contiguous_channels(fake, shape, strides):
    """Outputs follow the inputs' order of dimensions; where an input repeats rows and that order says nothing, they are contiguous."""
    _, lib = fake
    x = fc.Tensor(shape, BF16, strides=strides + (1,))
    pos, freqs = fc.Tensor(shape[:2], I32), fc.Tensor((32,), torch.int64)
    r = sv.qk_norm_rope(x, x, pos, freqs)
    a = sv.cache_attention(x, fc.Tensor((P, 1, 68 * 64), U8), fc.Tensor((shape[0], M), I32), fc.Tensor((shape[0],), I32))
    for t in (r["q"], r["k"], a["out"]):
        assert t.strides[3] == 1 and all(n == 1 or s >= 64 for n, s in zip(shape[:3], t.strides))


def test_status_bits_are_the_headers_and_exported():
    import os
    import re
    text = "".join(open(os.path.join(os.path.dirname(sv.__file__), os.pardir, "include", f)).read() for f in ("specverify.h", "speccache.h"))
    bits = dict(re.findall(r"#define SPEC_(STATUS_\w+) (\d+)u?", text))
    assert {"STATUS_BAD_TOKEN", "STATUS_TIMEOUT", "STATUS_BAD_PAGE", "STATUS_BAD_LENGTH", "STATUS_NO_PAGES", "STATUS_BAD_SLOT"} <= set(bits)
    for name, value in bits.items():
        assert getattr(sv, name) == int(value), name
