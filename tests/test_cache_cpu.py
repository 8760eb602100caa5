"""CPU checks of the 4-bit cache's operators: the C ABI's exports and refusals (before any CUDA call), the binding's
refusals, and the plain forms of cache_util against brute force."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import cache_util as cu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p
F = ctypes.c_float


@pytest.fixture(scope="module")
def sv():
    from speculative_decoding_verification_target_gb300 import _build
    _build.build()
    import speculative_decoding_verification_target_gb300 as sv
    return sv


@pytest.fixture(scope="module")
def lib(sv):
    from speculative_decoding_verification_target_gb300 import cache
    return cache._lib()


def H(data=1 << 20, b=1 << 14, n=1 << 12, h=128):
    from speculative_decoding_verification_target_gb300.cache import Heads
    return Heads(data, b, n, h)


def test_every_declared_symbol_is_exported(lib):
    from speculative_decoding_verification_target_gb300 import cache
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "speccache.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(spec_[a-z0-9_]+)\s*\(", text))
    assert names == set(cache.CACHE_EXPORTS)
    for n in names:
        assert hasattr(lib, n), n
    assert "SPEC_CACHE_WS_HEADER %d" % cache.WS_HEADER in text


def test_sizes(lib):
    assert [lib.spec_cache_block_bytes(d) for d in (64, 128, 0, 96, 256)] == [4352, 8704, 0, 0, 0]
    for bad in ((0, 8, 8, 128), (1025, 8, 8, 128), (1, 8, 0, 128), (1, 9, 4, 128), (1, 8, 8, 96), (1, 4, 8, 64)):
        assert lib.spec_cache_attention_workspace_size(*bad) == 0
    assert lib.spec_cache_attention_workspace_size(6, 32, 8, 128) >= 8192
    assert lib.spec_pages_workspace_size(64, 1000) >= 8192 + 4 * (3 * 64 + 3 * 1000 + 2)
    assert lib.spec_pages_workspace_size(-1, 5) == 0


def norm(lib, **kw):
    a = dict(q=H(), k=H(), dtype=0, B=2, N=3, Hq=8, Hk=2, D=128, pos=1 << 21, freqs=1 << 22, rotary=128, qw=1 << 23, kw=0,
             eps=1e-6, qo=H(), ko=H())
    a.update(kw)
    return lib.spec_qk_norm_rope(a["q"], a["k"], a["dtype"], a["B"], a["N"], a["Hq"], a["Hk"], a["D"], P(a["pos"]),
                                 P(a["freqs"]), a["rotary"], 0, P(a["qw"]), P(a["kw"]), a["eps"], a["qo"], a["ko"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), 1), (dict(N=-1), 1), (dict(B=70000), 1), (dict(Hq=-1), 1), (dict(Hq=0, Hk=0), 1), (dict(D=96), 3), (dict(dtype=3), 3),
    (dict(rotary=24), 1), (dict(rotary=144), 1), (dict(rotary=-16), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
    (dict(pos=0), 1), (dict(freqs=0), 1), (dict(q=H(data=0)), 1), (dict(q=None), 1), (dict(q=H(data=(1 << 20) + 2)), 1),
    (dict(k=H(h=129)), 1), (dict(qo=H(data=0)), 1), (dict(ko=H(n=4)), 1), (dict(qw=(1 << 23) + 8), 1),
    (dict(B=0), 0), (dict(N=0), 0),
])
def test_norm_rope_refusals(lib, kw, code):
    assert norm(lib, **kw) == code
    assert code == 0 or lib.spec_cache_last_error()


def tokens(fn, lib, **kw):
    a = dict(pool=1 << 20, pages=10, table=1 << 21, M=4, start=1 << 22, counts=0, k=H(), v=H(), dtype=0, B=2, N=3, Hk=2, D=128,
             ws=1 << 23, n=8192)
    a.update(kw)
    return getattr(lib, fn)(P(a["pool"]), a["pages"], P(a["table"]), a["M"], P(a["start"]), P(a["counts"]), a["k"], a["v"],
                            a["dtype"], a["B"], a["N"], a["Hk"], a["D"], P(a["ws"]), a["n"], None)


@pytest.mark.parametrize("fn", ["spec_cache_append", "spec_cache_read"])
@pytest.mark.parametrize("kw,code", [
    (dict(dtype=1), 3), (dict(D=256), 3), (dict(B=-1), 1), (dict(N=-2), 1), (dict(N=1 << 21), 1), (dict(Hk=0), 1),
    (dict(pool=0), 1), (dict(pool=(1 << 20) + 8), 1), (dict(table=0), 1), (dict(pages=0), 1), (dict(M=0), 1),
    (dict(M=1 << 26), 1), (dict(start=0), 1), (dict(ws=0), 1), (dict(ws=(1 << 23) + 4), 1), (dict(n=8191), 1),
    (dict(k=H(h=4)), 1), (dict(v=H(data=(1 << 20) + 4)), 1), (dict(B=0, pool=0), 0), (dict(N=0, pool=0), 0),
])
def test_token_refusals(lib, fn, kw, code):
    assert tokens(fn, lib, **kw) == code


def test_append_needs_both_and_read_one(lib):
    assert tokens("spec_cache_append", lib, k=None) == 1
    assert tokens("spec_cache_append", lib, v=H(data=0)) == 1
    assert tokens("spec_cache_read", lib, k=None, v=H(data=0)) == 1


def attend(lib, **kw):
    a = dict(q=H(), dtype=0, pool=1 << 20, pages=10, table=1 << 21, M=4, kv=1 << 22, ql=0, B=2, N=3, Hq=8, Hk=2, D=128,
             scale=0.1, window=0, sinks=0, out=H(), lse=0, ws=1 << 23, n=1 << 30)
    a.update(kw)
    return lib.spec_cache_attention(a["q"], a["dtype"], P(a["pool"]), a["pages"], P(a["table"]), a["M"], P(a["kv"]), P(a["ql"]),
                                    a["B"], a["N"], a["Hq"], a["Hk"], a["D"], a["scale"], a["window"], a["sinks"], a["out"],
                                    P(a["lse"]), P(a["ws"]), a["n"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=1), 3), (dict(dtype=9), 3), (dict(D=96), 3), (dict(N=1025), 1), (dict(Hq=9), 1), (dict(Hk=0), 1),
    (dict(scale=float("inf")), 1), (dict(window=-1), 1), (dict(sinks=-1), 1), (dict(q=None), 1), (dict(out=H(data=0)), 1),
    (dict(q=H(n=12)), 1), (dict(pool=0), 1), (dict(table=0), 1), (dict(kv=0), 1), (dict(ws=0), 1), (dict(n=100), 1),
    (dict(B=0, q=None), 0), (dict(N=0), 0),
])
def test_attention_refusals(lib, kw, code):
    assert attend(lib, **kw) == code


def test_pages_refusals(lib):
    t, w, n = P(1 << 20), P(1 << 23), 1 << 20
    assert lib.spec_pages_fork(t, t, t, 4, 4, 8, t, t, 5000, w, n, None) == 1
    assert lib.spec_pages_fork(t, t, t, 4, 4, 8, None, t, 2, w, n, None) == 1
    assert lib.spec_pages_fork(None, t, t, 4, 4, 8, t, t, 2, w, n, None) == 1
    assert lib.spec_pages_fork(t, t, t, 4, 4, 8, t, t, 0, w, n, None) == 0
    assert lib.spec_pages_reserve(t, 1, 24, t, t, t, 4, 4, 8, t, None, w, n, None) == 1      # page bytes not of 16
    assert lib.spec_pages_reserve(t, 0, 32, t, t, t, 4, 4, 8, t, None, w, n, None) == 1
    assert lib.spec_pages_reserve(t, 1, 32, t, t, t, 4, 4, 8, None, None, w, n, None) == 1
    assert lib.spec_pages_reserve(t, 1, 32, t, t, t, 4, 4, 8, t, None, w, 8192, None) == 1   # workspace
    assert lib.spec_pages_reserve(t, 1, 32, t, t, t, 0, 4, 8, t, None, w, n, None) == 0
    assert lib.spec_pages_commit(t, t, t, 4, 4, 0, t, 1, 0, 0, w, n, None) == 1
    assert lib.spec_pages_commit(t, t, t, 4, 4, 8, t, 1, -1, 0, w, n, None) == 1
    assert lib.spec_pages_commit(t, t, t, 4, 4, 8, None, 1, 0, 0, w, n, None) == 1
    assert lib.spec_pages_release(t, t, t, 4, 4, 8, t, -1, w, n, None) == 1
    assert lib.spec_pages_release(t, t, t, 4, 4, 8, t, 0, w, n, None) == 0
    assert lib.spec_pages_compact(None, 1, 32, t, t, 4, 4, 8, None, w, n, None) == 1
    assert lib.spec_pages_compact(t, 1, 32, t, t, -1, 4, 8, None, w, n, None) == 1


def test_binding_refuses_host_tensors_and_wrong_types(sv):
    pool = torch.zeros((4, 2, 8704), dtype=torch.uint8)
    table, n = torch.zeros((2, 2), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    x = torch.zeros((2, 1, 2, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        sv.cache_attention(x, pool, table, n)
    with pytest.raises(ValueError, match="CUDA tensor"):
        sv.cache_append(pool, table, n, x, x)
    with pytest.raises(ValueError, match="CUDA tensor"):
        sv.pages_commit(table, n, n, n)
    with pytest.raises(ValueError, match="CUDA tensor"):
        sv.qk_norm_rope(x, x, None, None, q_out=x, k_out=x)
    with pytest.raises(TypeError, match="float16"):
        sv.qk_norm_rope(x.double(), x, None, None)
    with pytest.raises(ValueError, match="head_dim"):
        sv.new_pool(1, 1, 96, device="cpu")


def test_frequencies_are_the_angles_to_2_pow_minus_50_of_a_turn(sv):
    f = sv.rope_frequencies(128, 10000.0, device="cpu").numpy().view(np.uint64)
    inv = 10000.0 ** (-np.arange(64) / 64)
    got = f.astype(object)
    for i in range(64):
        assert abs(int(got[i]) - inv[i] / (2 * np.pi) * 2.0 ** 64) <= 2.0 ** 13   # fp64 of a turn's fraction
    with pytest.raises(ValueError, match="rotary_dim / 2"):
        sv.rope_frequencies(8, inv_freq=[1.0], device="cpu")


def test_plain_quantiser_is_the_nearest_of_both_grids():
    rng = np.random.default_rng(0)
    x = rng.normal(size=(50, 64)) * np.exp(rng.normal(size=(50, 1)) * 4)
    x[3] = 0
    c, b = cu.quantise(x)
    grid = cu.scale_grid()
    for r in range(50):
        for g in range(2):
            v = x[r, 32 * g:32 * g + 32]
            top = np.abs(v).max() / 7
            assert abs(grid[b[r, g]] - min(top, grid[-1])) <= np.abs(grid - min(top, grid[-1])).min() + 1e-18
            if grid[b[r, g]] > 0:
                err = np.abs((c[r, 32 * g:32 * g + 32].astype(float) - 8) * grid[b[r, g]] - v)
                best = np.abs(np.arange(-7, 8)[None] * grid[b[r, g]] - v[:, None]).min(1)
                assert np.allclose(err, best, rtol=0, atol=1e-12 * (1 + top))
    pool = np.zeros((1, 1, 68 * 64), np.uint8)
    cu.write_token(pool, 0, 0, 17, c[0], b[0], c[1], b[1])
    k, v = cu.block_values(pool[0, 0])
    assert np.array_equal(k[17], (c[0].astype(float) - 8) * np.repeat(grid[b[0]], 32))
    assert np.array_equal(v[17], (c[1].astype(float) - 8) * np.repeat(grid[b[1]], 32))


def test_plain_pages_keep_every_count():
    """Random rounds of the plain bookkeeping: every page's count is the number of entries that name it."""
    rng = np.random.default_rng(1)
    S, M, NP = 6, 8, 40
    pool = rng.integers(0, 256, (1, NP, 4)).astype(np.uint8)
    table, lengths, refs = np.full((S, M), -1, np.int32), np.zeros(S, np.int32), np.zeros(NP, np.int32)
    for _ in range(60):
        n = rng.integers(0, 90, S)
        served, _ = cu.reserve(pool, table, lengths, refs, n)
        cu.commit(table, lengths, refs, np.where(served, rng.integers(0, 90, S) * (n > 0) % np.maximum(n, 1), 0), 0, rng.choice([0, 100]), 3)
        cu.fork(table, lengths, refs, rng.integers(0, S, 1), rng.integers(0, S, 1))
        assert np.array_equal(np.bincount(table[table >= 0], minlength=NP), refs)
        used = cu.compact(pool, table, refs)
        assert (refs[:used] > 0).all() and (refs[used:] == 0).all()
        lengths[lengths > 64 * M - 90] = 0
        for s in range(S):
            if lengths[s] == 0:
                for p in table[s][table[s] >= 0]:
                    refs[p] -= 1
                table[s] = -1
