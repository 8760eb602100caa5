"""GPU tests of the 4-bit cache's operators against the plain 64-bit forms of cache_util.

Tolerances, from the formats: a result of type T is off by half a step, eps(T) / 2 of its value. The norm and rotation
add fp32 sums, a reciprocal square root and a sine of an angle rounded to 2^-25 of a turn: within 2^-20 of the pair's
magnitudes. The attention rounds each probability to fp16 (2^-11 of it, or 2^-25 where it is below 2^-14 of the largest)
and its scores are fp32 sums of D = 128 products: each within delta = 2^-17 sum |q k| scale, which moves a probability by
2 delta; so out is within (2^-11 + 2^-13 + 2 delta) sum p |v| + 2^-25 sum |v|, and lse within delta + 2^-20 |lse|. The quantiser and the pages are exact.
"""
import numpy as np
import pytest
import torch

import cache_util as cu
import speculative_decoding_verification_target_gb300 as sv

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def f64(t):
    return t.detach().cpu().double().numpy()


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


# ------------------------------------------------------------------------------------------------ norm and rotation
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("B,N,Hq,Hk,D,R,inter,weights", [
    (1, 1, 1, 1, 64, 64, False, False), (3, 5, 8, 2, 128, 128, False, True), (2, 7, 5, 3, 128, 64, True, True),
    (2, 3, 4, 1, 256, 256, False, True), (1, 2, 3, 2, 256, 16, True, False), (2, 2, 40, 8, 64, 32, False, True),
    (1, 4, 2, 2, 64, 0, False, True), (70, 11, 33, 7, 128, 96, False, True),
])
def test_norm_rope(dtype, B, N, Hq, Hk, D, R, inter, weights):
    dt = DT[dtype]
    g = torch.Generator().manual_seed(D + R + N)
    qkv = (3 * torch.randn((B, N, Hq + 2 * Hk, D), generator=g)).to(dt).cuda()
    q, k = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk]
    pos = torch.randint(0, 1 << 20, (B, N), generator=g, dtype=torch.int32)
    if N > 1:
        pos[0, 0], pos[0, 1] = 0, 1
    qw = (1 + 0.2 * torch.randn(D, generator=g)).to(dt).cuda() if weights else None
    kw = (1 + 0.2 * torch.randn(D, generator=g)).to(dt).cuda() if weights else None
    freqs = sv.rope_frequencies(R, 10000.0) if R else None
    r = sv.qk_norm_rope(q, k, pos.cuda(), freqs, q_weight=qw, k_weight=kw, eps=1e-5, interleaved=inter)
    ang = pos.double().numpy()[:, :, None, None] * (10000.0 ** (-np.arange(0, R, 2) / R) if R else np.zeros(0))
    co, si = np.cos(ang), np.sin(ang)
    for x, w, got in ((q, qw, r["q"]), (k, kw, r["k"])):
        y = f64(x)
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + float(np.float32(1e-5)))
        if w is not None:
            y = y * f64(w)
        ref, size = y.copy(), np.abs(y)
        a, b = (slice(0, R, 2), slice(1, R, 2)) if inter else (slice(0, R // 2), slice(R // 2, R))
        ref[..., a], ref[..., b] = y[..., a] * co - y[..., b] * si, y[..., b] * co + y[..., a] * si
        size[..., a] = size[..., b] = np.abs(y[..., a]) + np.abs(y[..., b])
        # the table-free angle is the fp64 one to 2^-50 of a turn times the position
        tol = torch.finfo(dt).eps / 2 * np.abs(ref) + (2.0 ** -20 + torch.finfo(dt).eps * 2.0 ** -20) * size + torch.finfo(dt).tiny
        assert got.dtype == dt and (np.abs(f64(got) - ref) <= tol).all()


def test_norm_rope_in_place_and_on_another_stream():
    g = torch.Generator().manual_seed(5)
    qkv = torch.randn((4, 6, 12, 128), generator=g).bfloat16().cuda()
    pos = torch.randint(0, 5000, (4, 6), generator=g, dtype=torch.int32).cuda()
    freqs = sv.rope_frequencies(128)
    ref = sv.qk_norm_rope(qkv[:, :, :8], qkv[:, :, 8:10], pos, freqs)
    v = qkv[:, :, 10:].clone()
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    sv.qk_norm_rope(qkv[:, :, :8], qkv[:, :, 8:10], pos, freqs, q_out=qkv[:, :, :8], k_out=qkv[:, :, 8:10], stream=st)
    st.synchronize()
    assert torch.equal(qkv[:, :, :8], ref["q"]) and torch.equal(qkv[:, :, 8:10], ref["k"]) and torch.equal(qkv[:, :, 10:], v)


@pytest.mark.parametrize("Hq,Hk", [(5, 0), (0, 3), (8, 0), (1, 0)])
def test_norm_rope_of_queries_or_keys_alone(Hq, Hk):
    x = torch.randn((3, 4, 8, 128), generator=torch.Generator().manual_seed(6)).bfloat16().cuda()
    pos, freqs = torch.arange(12, dtype=torch.int32, device="cuda").view(3, 4), sv.rope_frequencies(128)
    both = sv.qk_norm_rope(x, x, pos, freqs)
    r = sv.qk_norm_rope(x[:, :, :Hq], x[:, :, :Hk], pos, freqs)
    assert torch.equal(r["q"], both["q"][:, :, :Hq]) and torch.equal(r["k"], both["k"][:, :, :Hk])


def test_norm_of_zeros_and_nan_rows_stay_their_own():
    q = torch.randn((1, 2, 4, 64)).half().cuda()
    q[0, 0, 1] = 0
    q[0, 1, 2, 5] = float("nan")
    r = sv.qk_norm_rope(q, q[:, :, :1], torch.zeros((1, 2), dtype=torch.int32, device="cuda"), sv.rope_frequencies(64))["q"]
    assert (r[0, 0, 1] == 0).all() and r[0, 1, 2].isnan().all()
    r[0, 1, 2] = 0
    assert torch.isfinite(r).all()


# ------------------------------------------------------------------------------------------------- append and read
def make_table(rng, B, M, extra=2):
    P = B * M + extra
    return rng.permutation(P)[:B * M].reshape(B, M).astype(np.int32), P


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("B,N,H,D,starts", [
    (1, 1, 1, 64, [0]), (1, 1, 8, 128, [63]), (3, 6, 2, 128, [0, 61, 64]), (2, 65, 3, 64, [1, 127]), (2, 200, 1, 128, [15, 48]),
    (1, 64, 2, 64, [64]), (2, 17, 2, 128, [16, 33]),
])
def test_append_and_read(dtype, B, N, H, D, starts):
    dt = DT[dtype]
    rng = np.random.default_rng(B * 1000 + N + D)
    x = rng.normal(size=(B, N, 3 * H, D)) * np.exp(rng.normal(size=(B, N, 3 * H, 1)) * 3)
    x[0, 0, H, :32] = 0                                        # an empty group
    x[0, 0, H, 32:64] = np.linspace(-7, 7, 32).round(1) / 2    # ties
    x[-1, -1, 2 * H, :32] = 1e-7                               # below the smallest scale
    x[-1, -1, 2 * H, 32:40] = [4e4, -4e4, 6300, 1, 0, -6272, 896, 448]
    qkv = torch.from_numpy(x).to(dt).cuda()
    k, v = qkv[:, :, H:2 * H], qkv[:, :, 2 * H:]
    M = (max(starts) + N) // 64 + 2
    table, P = make_table(rng, B, M)
    before = rng.integers(0, 256, (P, H, 68 * D)).astype(np.uint8)
    pool, start = dev(before), np.array(starts, np.int32)
    counts = np.array([N if b == 0 else rng.integers(0, N + 1) for b in range(B)], np.int32)
    ws = sv.new_pages_workspace(B, P)
    sv.cache_append(pool, dev(table), dev(start), k, v, counts=dev(counts), workspace=ws)
    ref, kc, vc = before.copy(), cu.quantise(f64(k)), cu.quantise(f64(v))
    for b in range(B):
        for i in range(counts[b]):
            t = int(start[b]) + i
            for h in range(H):
                cu.write_token(ref, table[b, t // 64], h, t % 64, kc[0][b, i, h], kc[1][b, i, h], vc[0][b, i, h], vc[1][b, i, h])
    assert np.array_equal(pool.cpu().numpy(), ref)             # the new tokens' bytes, and no other
    out = sv.cache_read(pool, dev(table), dev(start), N, counts=dev(counts), dtype=dt, workspace=ws)
    grid = cu.scale_grid()
    for (c, s), got in ((kc, out["k"]), (vc, out["v"])):
        val = (c.astype(float) - 8) * np.repeat(grid[s], 32, -1)
        for b in range(B):
            val[b, counts[b]:] = 0
        assert np.array_equal(f64(got), val)
    assert sv.read_status(ws) == 0


def test_append_nan_and_inf_stay_in_their_group():
    k = torch.ones((1, 1, 1, 64), dtype=torch.float16, device="cuda")
    k[0, 0, 0, 3], k[0, 0, 0, 40] = float("nan"), float("-inf")
    pool, table = sv.new_pool(1, 1, 64), torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    start = torch.zeros(1, dtype=torch.int32, device="cuda")
    sv.cache_append(pool, table, start, k, k)
    r = sv.cache_read(pool, table, start, 1, dtype=torch.float16)
    want = torch.ones(64)
    c, s = cu.quantise(np.ones((1, 64)))
    want[:32] = (c[0, 0] - 8.0) * cu.scale_grid()[s[0, 0]]
    want[3], want[32:], want[40] = 0, 0, -6272
    assert torch.equal(r["k"].cpu().flatten().float(), want) and torch.equal(r["v"], r["k"])


def test_append_and_read_with_bad_pages_and_lengths():
    B, N, H, D = 5, 10, 2, 64
    pool = torch.full((4, H, 68 * D), 7, dtype=torch.uint8, device="cuda")
    # a missing page, one outside the pool, a run past the table, a negative start, a good one
    table = dev(np.array([[-1, 0], [4, 0], [0, 1], [2, 0], [3, 0]], np.int32))
    start = dev(np.array([0, 60, 125, -4, 2], np.int32))
    k = torch.ones((B, N, H, D), dtype=torch.bfloat16, device="cuda")
    ws = sv.new_pages_workspace(B, 4)
    sv.cache_append(pool, table, start[:1].expand(5).contiguous() * 0, k, k, counts=dev(np.array([10, 0, 0, 0, 0], np.int32)), workspace=ws)
    assert sv.read_status(ws) == 4 and (pool == 7).all()
    sv.clear_status(ws)
    counts = dev(np.array([10, 4, 10, 10, 10], np.int32))
    sv.cache_append(pool, table, start, k, k, counts=counts, workspace=ws)
    assert sv.read_status(ws) == 4 | 8
    r = sv.cache_read(pool, table, start, N, counts=counts, workspace=ws)["k"].cpu().float()[:, :, 0, 0]
    assert (r[0] == 0).all() and (r[1] == 0).all()
    assert (r[2, :3] != 0).all() and (r[2, 3:] == 0).all() and (r[3, :4] == 0).all() and (r[3, 4:] != 0).all() and (r[4] != 0).all()
    sv.clear_status(ws)
    sv.cache_append(pool, table[4:].contiguous(), start[4:].contiguous(), k[4:], k[4:], counts=dev(np.array([11], np.int32)), workspace=ws)
    assert sv.read_status(ws) == 8


# ------------------------------------------------------------------------------------------------------- attention
def attention_case(rng, B, N, Hq, H, D, lens, dt, window=0, sinks=0, q_len=None, scale=None, spread=1.0):
    lens = np.array(lens, np.int32)
    M = max(1, (int(lens.max()) + 63) // 64)
    table, P = make_table(rng, B, M)
    pool = rng.integers(0, 256, (P, H, 68 * D)).astype(np.uint8)     # unused slots hold anything, NaN scales too
    for b in range(B):
        for j in range((int(lens[b]) + 63) // 64):
            for h in range(H):
                blk, n, m = pool[table[b, j], h], D // 32, min(64, int(lens[b]) - j * 64)
                blk[:32 * D] |= 0x11
                blk[32 * D:32 * D + m * n] = rng.integers(100, 116, m * n)     # scales 0.06 .. 0.25
                blk[66 * D:66 * D + m * n] = rng.integers(100, 116, m * n)
        if window:
            dead = int(lens[b]) - N - window + 1
            for j in range(M):
                if j * 64 >= sinks and j * 64 + 64 <= dead:
                    table[b, j] = -1
    q = torch.from_numpy(rng.normal(size=(B, N, Hq + 2, D)) * spread).to(dt).cuda()[:, :, 1:Hq + 1]
    ql = np.full(B, N, np.int32) if q_len is None else np.array(q_len, np.int32)
    return q, pool, table, lens, ql


def check_attention(q, pool, table, lens, ql, window=0, sinks=0, scale=None, status=0):
    D = q.shape[-1]
    ws = sv.new_attention_workspace(q.shape[1], q.shape[2], pool.shape[1], D)
    out = torch.full((q.shape[0], q.shape[2], q.shape[1], D), 9.0, dtype=q.dtype, device="cuda").transpose(1, 2)   # heads first
    lse = torch.full(q.shape[:3], 9.0, device="cuda")
    args = (q, dev(pool), dev(table), dev(lens))
    kw = dict(q_len=dev(ql), window=window, sinks=sinks, scale=scale, workspace=ws)
    for _ in range(2):         # twice on one workspace: it is left as it was found
        sv.cache_attention(*args, out=out, lse=lse, **kw)
    assert sv.read_status(ws) == status
    ref, rl, mass, big, total = cu.attention(f64(q), pool, table, lens, ql, D ** -0.5 if scale is None else scale, window, sinks)
    delta = 2.0 ** -17 * big
    tol = torch.finfo(q.dtype).eps / 2 * np.abs(ref) + (2.0 ** -11 + 2.0 ** -13 + 2 * delta[..., None]) * mass + 2.0 ** -25 * total + torch.finfo(q.dtype).tiny
    err = np.abs(f64(out) - ref)
    assert (err <= tol).all(), float((err / np.maximum(tol, 1e-30)).max())
    got, empty = f64(lse), np.isinf(rl)
    assert np.array_equal(np.isneginf(got), empty)
    assert (np.abs(got - rl)[~empty] <= (delta + 2.0 ** -20 * (1 + np.abs(rl)))[~empty]).all()
    again = sv.cache_attention(*args, **kw)
    assert torch.equal(again["out"], out)


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp16", 64), ("fp16", 128), ("bf16", 64)])
@pytest.mark.parametrize("B,N,Hq,H,lens", [
    (1, 1, 1, 1, [1]), (1, 1, 8, 8, [64]), (4, 1, 4, 2, [0, 63, 65, 129]), (3, 6, 8, 2, [3, 6, 700]),
    (2, 9, 16, 1, [1500, 9]), (1, 33, 5, 5, [100]), (5, 3, 14, 2, [1, 2, 300, 128, 192]), (1, 70, 8, 2, [333]),
    (33, 2, 2, 2, list(range(60, 93))),
])
def test_attention(dtype, D, B, N, Hq, H, lens):
    rng = np.random.default_rng(B * 100 + N + D)
    check_attention(*attention_case(rng, B, N, Hq, H, D, lens, DT[dtype]))


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (64, 4), (63, 64), (65, 130), (100, 5000), (5000, 3), (200, 65)])
@pytest.mark.parametrize("N,D", [(1, 128), (6, 64), (40, 128)])
def test_attention_window_and_sinks(window, sinks, N, D):
    rng = np.random.default_rng(window + sinks + N)
    check_attention(*attention_case(rng, 4, N, 6, 2, D, [1, 64, 400, 777], torch.bfloat16, window, sinks), window=window, sinks=sinks)


def device_check(q, pool, table, lens, window=0, sinks=0):
    """As check_attention, with the plain form in fp64 on the GPU over what cache_read gives (exact)."""
    B, N, Hq, D = q.shape
    H, n = pool.shape[1], int(lens.max())
    G = Hq // H
    r = sv.cache_attention(q, pool, table, lens, window=window, sinks=sinks, want_lse=True)
    assert sv.read_status(r["workspace"]) == 0
    held = sv.cache_read(pool, table, torch.zeros_like(lens), n, counts=lens, dtype=torch.float16)
    at = torch.arange(n, device="cuda")
    for b in range(B):
        k, v = held["k"][b].double().transpose(0, 1), held["v"][b].double().transpose(0, 1)          # [H, n, D]
        x = q[b].double().view(N, H, G, D).permute(1, 0, 2, 3).reshape(H, N * G, D)
        pos = (int(lens[b]) - N + torch.arange(N, device="cuda"))[:, None]
        see = at <= pos
        if window:
            see &= (at > pos - window) | (at < sinks)
        see = see.repeat_interleave(G, 0)[None]
        sc = (x @ k.transpose(1, 2) * D ** -0.5).masked_fill(~see, -torch.inf)
        lse = sc.logsumexp(-1)
        p = torch.where(see, (sc - torch.where(lse.isinf(), 0, lse)[..., None]).exp(), 0)
        ref, mass = p @ v, p @ v.abs()
        delta = 2.0 ** -17 * ((x.abs() @ k.abs().transpose(1, 2)) * see).amax(-1) * D ** -0.5
        total = see.double().expand(H, -1, -1) @ v.abs()
        out = r["out"][b].double().view(N, H, G, D).permute(1, 0, 2, 3).reshape(H, N * G, D)
        tol = torch.finfo(q.dtype).eps / 2 * ref.abs() + (2.0 ** -11 + 2.0 ** -13 + 2 * delta[..., None]) * mass + 2.0 ** -25 * total
        assert ((out - ref).abs() <= tol + torch.finfo(q.dtype).tiny).all(), b
        got = r["lse"][b].double().view(N, H, G).permute(1, 0, 2).reshape(H, N * G)
        assert torch.equal(got.isinf(), lse.isinf()) and ((got - lse).abs()[~lse.isinf()] <= (delta + 2.0 ** -20 * (1 + lse.abs()))[~lse.isinf()]).all(), b


def device_case(seed, B, N, Hq, H, D, lens, dt):
    g = torch.Generator(device="cuda").manual_seed(seed)
    lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    M = (int(lens.max()) + 63) // 64
    table = torch.randperm(B * M, generator=g, device="cuda").to(torch.int32).view(B, M)
    pool = sv.new_pool(B * M, H, D)
    step = 8192
    for a in range(0, M * 64, step):
        n = min(step, M * 64 - a)
        kv = torch.randn((2, B, n, H, D), generator=g, device="cuda").to(dt)
        sv.cache_append(pool, table, torch.full_like(lens, a), kv[0], kv[1])
    return torch.randn((B, N, Hq, D), generator=g, device="cuda").to(dt), pool, table, lens


@pytest.mark.parametrize("B,N,Hq,H,D,lens,window,sinks", [
    (400, 2, 4, 2, 64, [(37 * b) % 301 for b in range(400)], 0, 0),              # more sequences than a CTA has threads, empty ones too
    (200, 1, 8, 1, 128, [1 + (91 * b) % 777 for b in range(200)], 100, 3),
    (1, 3, 4, 1, 128, [131035], 0, 0),                                           # one unit over all CTAs
    (2, 1, 1, 1, 64, [65536, 3], 0, 0),
    (1, 300, 4, 2, 128, [1000], 0, 0),                                           # many query blocks
    (2, 1024, 2, 2, 64, [1024, 2500], 300, 70),
    (3, 20, 2, 1, 128, [5000, 40, 129], 0, 0), (2, 7, 8, 1, 64, [700, 3000], 1000, 10),    # widths 48 and 64
])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_attention_on_larger_shapes(dtype, B, N, Hq, H, D, lens, window, sinks):
    q, pool, table, lens = device_case(B + N, B, N, Hq, H, D, lens, DT[dtype])
    device_check(q, pool, table, lens, window, sinks)


def test_attention_ragged_queries():
    rng = np.random.default_rng(7)
    check_attention(*attention_case(rng, 6, 5, 8, 2, 128, [0, 1, 3, 70, 128, 500], torch.bfloat16, q_len=[5, 0, 5, 1, 3, 5]))


def test_attention_steep_and_flat_scores():
    """Scores spread over hundreds (the running maximum moves often), one token far above the rest at the end, all equal."""
    rng = np.random.default_rng(8)
    case = attention_case(rng, 3, 2, 8, 2, 128, [900, 1024, 2000], torch.bfloat16, spread=30.0)
    check_attention(*case)
    check_attention(*case, scale=0.0)
    check_attention(*case, scale=-0.02)
    q = attention_case(rng, 1, 1, 2, 1, 64, [700], torch.float16)
    q[1][q[2][0, 10], 0, 32 * 64:32 * 64 + (700 - 640) * 2] = 150
    check_attention(*q)
    tiny = attention_case(rng, 1, 2, 2, 1, 64, [300], torch.bfloat16, spread=1e-30)
    check_attention(*tiny)
    check_attention(*attention_case(rng, 1, 2, 2, 1, 64, [300], torch.bfloat16, spread=3e4), scale=1e-5)


def test_attention_bad_pages_and_lengths():
    rng = np.random.default_rng(9)
    q, pool, table, lens, ql = attention_case(rng, 3, 2, 4, 2, 128, [300, 200, 256], torch.bfloat16)
    table[0, 1], table[1, :], table[2, 3] = -1, -1, len(pool)
    check_attention(q, pool, table, lens, ql, status=4)
    q, pool, table, lens, ql = attention_case(rng, 3, 2, 4, 2, 128, [320, 200, 256], torch.bfloat16)   # 320: the whole table
    lens[0], lens[1], ql[2] = 100000, -5, 1
    check_attention(q, pool, table, lens, ql, status=8)


def test_attention_in_a_graph_and_on_another_stream():
    rng = np.random.default_rng(10)
    q, pool, table, lens, ql = attention_case(rng, 4, 3, 8, 2, 128, [300, 200, 256, 2000], torch.bfloat16)
    pool, table, kv = dev(pool), dev(table), dev(lens)
    ws = sv.new_attention_workspace(3, 8, 2, 128)
    ref = sv.cache_attention(q, pool, table, kv, workspace=ws)["out"].clone()
    out, st = torch.zeros_like(ref), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        sv.cache_attention(q, pool, table, kv, out=out, workspace=ws)
        st.synchronize()
        out.zero_()
        with torch.cuda.graph(graph, stream=st):
            sv.cache_attention(q, pool, table, kv, out=out, workspace=ws)
        for _ in range(3):
            graph.replay()
        kv.fill_(150)           # lengths are read on the device: the same graph serves the next round
        graph.replay()
    st.synchronize()
    torch.cuda.synchronize()
    short = sv.cache_attention(q, pool, table, torch.full_like(kv, 150), workspace=ws)["out"]
    assert torch.equal(out, short)
    kv.copy_(dev(lens))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref)


def test_cache_past_four_gigabytes():
    """Page offsets beyond 32 bits: the pages used are the pool's last."""
    P, H, D = 62000, 8, 128
    pool = torch.zeros((P, H, 68 * D), dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(11)
    q, small, table, lens, ql = attention_case(rng, 2, 2, 8, 8, 128, [150, 64], torch.bfloat16)
    n = small.shape[0]
    pool[P - n:] = dev(small)
    far = sv.cache_attention(q, pool, dev(table + (P - n)).to(torch.int32), dev(lens))["out"]
    near = sv.cache_attention(q, dev(small), dev(table), dev(lens))["out"]
    assert torch.equal(far, near)
    k = torch.randn((1, 3, H, D), dtype=torch.bfloat16, device="cuda")
    t, s = torch.full((1, 1), P - 1, dtype=torch.int32, device="cuda"), torch.full((1,), 5, dtype=torch.int32, device="cuda")
    sv.cache_append(pool, t, s, k, k)
    t2 = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    one = sv.new_pool(1, H, D)
    sv.cache_append(one, t2, s, k, k)
    assert torch.equal(sv.cache_read(pool, t, s, 3)["k"], sv.cache_read(one, t2, s, 3)["k"])


# ----------------------------------------------------------------------------------------------------------- pages
def books(rng, S, M, P, fill=0.6):
    lengths = (rng.random(S) * fill * M * 64).astype(np.int32)
    table, refs, order, at = np.full((S, M), -1, np.int32), np.zeros(P, np.int32), rng.permutation(P), 0
    for s in range(S):
        for j in range((lengths[s] + 63) // 64):
            if at == P:
                lengths[s] = j * 64
                break
            table[s, j] = order[at]
            refs[order[at]] = 1
            at += 1
    return table, lengths, refs


@pytest.mark.parametrize("S,M,P,layers", [(1, 2, 3, 1), (7, 5, 40, 2), (64, 16, 700, 1), (300, 8, 1500, 2), (40, 40, 9000, 1)])
def test_pages_rounds(S, M, P, layers):
    """Rounds of fork, reserve, commit, release and compact, each call against the sequential plain form."""
    rng = np.random.default_rng(S + P)
    table, lengths, refs = books(rng, S, M, P)
    pool = rng.integers(0, 256, (layers, P, 1, 32)).astype(np.uint8)
    g = [dev(pool), dev(table), dev(lengths), dev(refs)]
    ws = sv.new_pages_workspace(S, P)

    def same(*names):
        for name, a, t in zip(("pool", "table", "lengths", "refs"), (pool, table, lengths, refs), g):
            assert np.array_equal(t.cpu().numpy(), a), (names, name)

    for rnd in range(6):
        F = int(rng.integers(0, max(1, S // 2)))
        src, dst = rng.integers(0, S, F).astype(np.int32), rng.integers(0, S, F).astype(np.int32)
        st = cu.fork(table, lengths, refs, src, dst)
        sv.pages_fork(*g[1:], dev(src), dev(dst), workspace=ws)
        assert sv.read_status(ws) == st
        same("fork", rnd)
        sv.clear_status(ws)
        n = (rng.integers(-1, 8, S) if rnd % 2 else rng.integers(0, 200, S)).astype(np.int32)
        served, st = cu.reserve(pool, table, lengths, refs, n)
        got = sv.pages_reserve(*g, dev(n), workspace=ws)
        assert np.array_equal(got.cpu().numpy(), served) and sv.read_status(ws) == st
        same("reserve", rnd)
        sv.clear_status(ws)
        adv = (rng.integers(0, 8, S) * (served > 0) % np.maximum(n, 1) - 1).astype(np.int32)
        window, sinks = ((0, 0), (100, 0), (70, 65))[rnd % 3]
        st = cu.commit(table, lengths, refs, adv, 1, window, sinks)
        sv.pages_commit(*g[1:], dev(adv), window=window, sinks=sinks, workspace=ws)
        assert sv.read_status(ws) == st
        same("commit", rnd)
        slots = rng.integers(0, S, 1 + S // 8).astype(np.int32)
        for s in slots:
            for p in table[s][table[s] >= 0]:
                refs[p] -= 1
            table[s], lengths[s] = -1, 0
        sv.pages_release(*g[1:], dev(slots), workspace=ws)
        same("release", rnd)
        if rnd % 2:
            n_used = cu.compact(pool, table, refs)
            got = sv.pages_compact(g[0], g[1], g[3], workspace=ws)
            assert int(got) == n_used
            same("compact", rnd)
        assert np.array_equal(np.bincount(table[table >= 0], minlength=P), refs)
    assert sv.read_status(ws) == 0


def test_pages_bad_entries_are_reported_not_followed():
    S, M, P = 3, 3, 6
    ws = sv.new_pages_workspace(S, P)
    table = dev(np.array([[0, 99, -1], [1, -7, -1], [2, 3, -1]], np.int32))
    lengths, refs = dev(np.array([70, 70, 100], np.int32)), dev(np.array([1, 1, 1, 1, 0, 0], np.int32))
    sv.pages_release(table, lengths, refs, dev(np.array([0, -1, 3, 0], np.int32)), workspace=ws)
    assert sv.read_status(ws) == 4 | 32 and refs.tolist() == [0, 1, 1, 1, 0, 0] and table[0].tolist() == [-1, -1, -1]
    sv.clear_status(ws)
    sv.pages_commit(table, lengths, refs, dev(np.array([0, 1000, -1000], np.int32)), workspace=ws)
    assert sv.read_status(ws) == 8 and lengths.tolist() == [1, 192, 0] and refs.tolist() == [0, 1, 0, 0, 0, 0]
    sv.clear_status(ws)
    sv.pages_fork(table, lengths, refs, dev(np.array([1, 5, 0], np.int32)), dev(np.array([2, 0, -1], np.int32)), workspace=ws)
    assert sv.read_status(ws) == 32 and table[2, 0].item() == 1 and refs.tolist() == [0, 2, 0, 0, 0, 0]


def test_whole_round_in_one_graph():
    """Reserve, norm and rotation, append, attention and commit captured once and replayed as lengths grow."""
    B, N, Hq, H, D, M, P = 3, 4, 8, 2, 64, 6, 20
    g = torch.Generator().manual_seed(3)
    qkv = torch.randn((B, N, Hq + 2 * H, D), generator=g).bfloat16().cuda()
    freqs, i32 = sv.rope_frequencies(D), dict(dtype=torch.int32, device="cuda")
    step = torch.arange(N, **i32)

    def fresh():
        return dict(pool=sv.new_pool(P, H, D), table=torch.full((B, M), -1, **i32), lengths=torch.tensor([0, 30, 61], **i32) * 0,
                    refs=torch.zeros(P, **i32), n=torch.full((B,), N, **i32), acc=torch.tensor([3, 0, 2], **i32),
                    pw=sv.new_pages_workspace(B, P), aw=sv.new_attention_workspace(N, Hq, H, D),
                    out=torch.zeros((B, N, Hq, D), dtype=torch.bfloat16, device="cuda"), served=torch.zeros(B, **i32))

    def once(s):
        sv.pages_reserve(s["pool"], s["table"], s["lengths"], s["refs"], s["n"], served=s["served"], workspace=s["pw"])
        r = sv.qk_norm_rope(qkv[:, :, :Hq], qkv[:, :, Hq:Hq + H], s["lengths"][:, None] + step, freqs)
        sv.cache_append(s["pool"], s["table"], s["lengths"], r["k"], qkv[:, :, Hq + H:], workspace=s["pw"])
        sv.cache_attention(r["q"], s["pool"], s["table"], s["lengths"] + N, out=s["out"], workspace=s["aw"])
        sv.pages_commit(s["table"], s["lengths"], s["refs"], s["acc"], workspace=s["pw"])

    a, b = fresh(), fresh()
    for _ in range(30):
        once(a)
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        once(b)
        st.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            once(b)
        for _ in range(29):
            graph.replay()
    torch.cuda.synchronize()
    assert a["lengths"].tolist() == [120, 30, 90] and sv.read_status(a["pw"]) == 0
    for k in a:
        if k not in ("aw", "pw"):
            assert torch.equal(a[k], b[k]), k
