"""GPU tests of the cache's operators where they can go wrong: streams, workspaces, far smaller probabilities, page sizes, infinities."""
import numpy as np
import pytest
import torch

import cache_util as cu
import speculative_decoding_verification_target_gb300 as sv

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device="cuda")


def test_calls_on_a_stream_beside_a_busy_one():
    """Without workspaces and outputs, on a stream of their own while the current one has work queued before and behind them: the
    results are those of calls on the current stream."""
    B, N, Hq, H, D, M = 2, 3, 8, 2, 64, 80
    g = torch.Generator().manual_seed(1)
    qkv = torch.randn((B, N, Hq + 2 * H, D), generator=g).bfloat16().cuda()
    q, k, v = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + H], qkv[:, :, Hq + H:]
    blocks = torch.randint(0, 256, (2 * B * M, H, 68 * D), generator=g, dtype=torch.uint8)
    blocks[:, :, 32 * D:34 * D] = blocks[:, :, 32 * D:34 * D] % 100 + 20      # scales of written tokens
    blocks[:, :, 66 * D:] = blocks[:, :, 66 * D:] % 100 + 20
    start = dict(pool=blocks.cuda(), table=torch.full((B, M), -1, **I32), lengths=torch.tensor([M * 64 - 70, 100], **I32),
                 refs=torch.zeros(2 * B * M, **I32))
    for b in range(B):
        n = (int(start["lengths"][b]) + 63) // 64
        start["table"][b, :n] = torch.randperm(B * M, generator=g)[:n].to(torch.int32).cuda() + b * B * M
        start["refs"][start["table"][b, :n].long()] = 1
    n_new, freqs = torch.full((B,), N, **I32), sv.rope_frequencies(D)
    src, dst = torch.zeros(1, **I32), torch.ones(1, **I32)

    def calls(stream):
        s = {k: t.clone() for k, t in start.items()}
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
            torch.cuda._sleep(200_000_000)                  # a tenth of a second of the current stream
        kw = dict(stream=stream)
        sv.pages_fork(s["table"], s["lengths"], s["refs"], src, dst, **kw)
        served = sv.pages_reserve(s["pool"], s["table"], s["lengths"], s["refs"], n_new, **kw)
        r = sv.qk_norm_rope(q, k, pos, freqs, **kw)
        sv.cache_append(s["pool"], s["table"], s["lengths"], r["k"], v, **kw)
        a = sv.cache_attention(r["q"], s["pool"], s["table"], after, want_lse=True, **kw)
        held = sv.cache_read(s["pool"], s["table"], s["lengths"], N, **kw)
        sv.pages_commit(s["table"], s["lengths"], s["refs"], n_new, extra=0, **kw)
        sv.pages_release(s["table"], s["lengths"], s["refs"], src, **kw)
        used = sv.pages_compact(s["pool"], s["table"], s["refs"], **kw)
        (stream or torch.cuda.current_stream()).synchronize()
        out = dict(s, served=served, used=used, out=a["out"], lse=a["lse"], hk=held["k"], hv=held["v"], q=r["q"])
        return {k: t.cpu() for k, t in out.items()}

    after = torch.full((B,), M * 64 - 70 + N, **I32)       # both as long as sequence 0 after the fork
    pos = (after - N)[:, None] + torch.arange(N, **I32)
    want = calls(None)
    assert want["served"].tolist() == [1, 1] and torch.isfinite(want["out"].float()).all()
    st = torch.cuda.Stream()
    for _ in range(3):
        got = calls(st)
        for name in want:
            assert torch.equal(got[name], want[name]), name


def test_verification_on_a_stream_beside_a_busy_one():
    g = torch.Generator().manual_seed(2)
    target, draft = torch.randn((4, 4, 1000), generator=g).cuda(), torch.randn((4, 3, 1000), generator=g).cuda()
    tokens, seeds = torch.randint(0, 1000, (4, 3), generator=g, dtype=torch.int32).cuda(), torch.arange(4, device="cuda")
    want = [sv.verify(target, draft, tokens, seeds), sv.verify_filtered(target, draft, tokens, seeds, top_k=20),
            sv.greedy_verify(target, tokens)]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    torch.cuda._sleep(200_000_000)
    got = [sv.verify(target, draft, tokens, seeds, stream=st), sv.verify_filtered(target, draft, tokens, seeds, top_k=20, stream=st),
           sv.greedy_verify(target, tokens, stream=st)]
    st.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a["accept_len"], b["accept_len"])
        for n, x, y in zip(a["accept_len"].tolist(), a["out_tokens"].tolist(), b["out_tokens"].tolist()):
            assert x[:n + 1] == y[:n + 1]


@pytest.mark.parametrize("Hq,H,D,most", [(64, 8, 128, 9), (32, 8, 128, 12), (8, 8, 64, 70)])
def test_one_attention_workspace_for_every_number_of_tokens(Hq, H, D, most):
    g = torch.Generator().manual_seed(most)
    lens = torch.tensor([400, 90], **I32)
    table, zero = torch.arange(14, **I32).view(2, 7), torch.zeros(2, **I32)
    kv = torch.randn((2, 400, 2 * H, D), generator=g).half().cuda()
    pool = sv.new_pool(14, H, D)
    sv.cache_append(pool, table, zero, kv[:, :, :H], kv[:, :, H:])
    ws = sv.new_attention_workspace(most, Hq, H, D)
    for N in range(most, 0, -1):
        q = torch.randn((2, N, Hq, D), generator=g).half().cuda()
        got = sv.cache_attention(q, pool, table, lens, workspace=ws)["out"]
        assert torch.equal(got, sv.cache_attention(q, pool, table, lens)["out"]), N
    assert sv.read_status(ws) == 0


def sink_case(n, D, H, N, gap, dtype, dominant):
    """n cached tokens with the same key and value 1 each, but for `dominant`, whose score is `gap` above and whose value is 0."""
    k = torch.full((1, n, H, D), -1.0)
    k[:, dominant] = 1.0
    v = torch.ones((1, n, H, D))
    v[:, dominant] = 0.0
    M = (n + 63) // 64
    pool, table = sv.new_pool(M, H, D), torch.randperm(M, generator=torch.Generator().manual_seed(n)).to(torch.int32).cuda().view(1, M)
    sv.cache_append(pool, table, torch.zeros(1, **I32), k.to(dtype).cuda(), v.to(dtype).cuda())
    held = sv.cache_read(pool, table, torch.zeros(1, **I32), n, dtype=torch.float16)
    step = float(held["k"][0, dominant, 0, 0] - held["k"][0, 1 if dominant == 0 else 0, 0, 0])      # between the two keys
    q = torch.full((1, N, 2 * H, D), gap / (step * D ** 0.5)).to(dtype).cuda()
    return q, pool, table, held


@pytest.mark.parametrize("gap", [6.0, 9.5, 12.0, 15.0, 17.0, 17.5, 18.0, 20.0])
@pytest.mark.parametrize("n,D,H,N,dominant", [
    (131072, 128, 1, 1, 0), (131072, 64, 2, 1, 0), (100001, 128, 1, 20, 0),     # a first token that takes the weight, parts joined
    (3000, 128, 1, 3, 1500), (3000, 64, 1, 5, 2990), (130, 128, 4, 1, 129),     # one that comes later: the reference moves
])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_small_probabilities_beside_a_dominant_one(gap, n, D, H, N, dominant, dtype):
    """The rest's share, held by many tokens with less than 2^-14 of the largest probability each. A probability is off by 2^-11 of itself
    or by 2^-32 of the largest: with the reference seven binary orders below the maximum or more, the largest is 2^7 or more in
    the kernel's units and half a step of the smallest halves 2^-25. Else as in test_gpu_cache: scores within
    delta = 2^-17 sum |q k| scale, the output rounded once."""
    q, pool, table, held = sink_case(n, D, H, N, gap, dtype, dominant)
    r = sv.cache_attention(q, pool, table, torch.tensor([n], **I32), want_lse=True)
    k, v = held["k"][0].double().transpose(0, 1), held["v"][0].double().transpose(0, 1)           # [H, n, D]
    x = q[0].double().view(N, H, 2, D).permute(1, 0, 2, 3).reshape(H, N * 2, D)
    see = (torch.arange(n, device="cuda") <= (n - N + torch.arange(N, device="cuda"))[:, None]).repeat_interleave(2, 0)[None]
    sc = (x @ k.transpose(1, 2) * D ** -0.5).masked_fill(~see, -torch.inf)
    lse = sc.logsumexp(-1)
    p = (sc - lse[..., None]).exp()
    ref, mass, total = p @ v, p @ v.abs(), see.double().expand(H, -1, -1) @ v.abs()
    delta = 2.0 ** -17 * (x.abs() @ k.abs().transpose(1, 2)).amax(-1) * D ** -0.5
    tol = torch.finfo(dtype).eps / 2 * ref.abs() + (2.0 ** -11 + 2.0 ** -13 + 2 * delta[..., None]) * mass + 2.0 ** -32 * total
    out = r["out"][0].double().view(N, H, 2, D).permute(1, 0, 2, 3).reshape(H, N * 2, D)
    err = (out - ref).abs()
    assert (err <= tol + torch.finfo(dtype).tiny).all(), float((err / tol).max())
    got = r["lse"][0].double().view(N, H, 2).permute(1, 0, 2).reshape(H, N * 2)
    assert ((got - lse).abs() <= delta + 2.0 ** -20 * (1 + lse.abs())).all()


@pytest.mark.parametrize("gap", [12.0, 15.0, 17.0, 17.5, 18.0])
@pytest.mark.parametrize("D", [64, 128])
def test_small_probabilities_of_sequences_that_are_not_cut(gap, D):
    """As above, with so many sequences (all of them the same pages) that a sequence's tokens are mostly one part's, beside its dominant one."""
    n, S = 20000, 700
    q, pool, table, held = sink_case(n, D, 1, 1, gap, torch.float16, 0)
    out = sv.cache_attention(q.expand(S, 1, 2, D).contiguous(), pool, table.expand(S, -1).contiguous(), torch.full((S,), n, **I32))["out"]
    k, v = held["k"][0, :, 0].double(), held["v"][0, :, 0].double()
    sc = k @ q[0, 0, 0].double() * D ** -0.5
    p = sc.softmax(-1)
    ref = p @ v
    delta = 2.0 ** -17 * float((k.abs() @ q[0, 0, 0].double().abs()).max()) * D ** -0.5
    tol = (2.0 ** -11 + 2.0 ** -11 + 2.0 ** -13 + 2 * delta) * ref + 2.0 ** -32 * n + 2.0 ** -25      # fp16 outputs: half a step, 2^-25 at least
    assert ((out.double() - ref).abs() <= tol).all(), float(((out.double() - ref).abs() / tol).max())


@pytest.mark.parametrize("P", [1, 7, 9000])
def test_compaction_without_sequences(P):
    rng = np.random.default_rng(P)
    refs, pool = rng.integers(0, 2, P).astype(np.int32), rng.integers(0, 256, (2, P, 1, 32)).astype(np.uint8)
    table = np.zeros((0, 3), np.int32)
    gp, gr = torch.from_numpy(pool.copy()).cuda(), torch.from_numpy(refs.copy()).cuda()
    used = sv.pages_compact(gp, torch.from_numpy(table).cuda(), gr)
    assert int(used) == cu.compact(pool, table, refs)
    assert np.array_equal(gp.cpu().numpy(), pool) and np.array_equal(gr.cpu().numpy(), refs)


@pytest.mark.parametrize("layers", [1, 2])
@pytest.mark.parametrize("page_bytes", [32, 4096, 16384, 16400, 69632])
def test_page_copies_of_every_size(page_bytes, layers):
    """A copy's pieces are 16384 bytes: pages of less, of one, of one and a little, of 4.25 (8 heads of 128), byte for byte."""
    rng = np.random.default_rng(page_bytes + layers)
    S, M, P = 9, 4, 40
    pool = rng.integers(0, 256, (layers, P, 1, page_bytes)).astype(np.uint8)
    table, refs, lengths = np.full((S, M), -1, np.int32), np.zeros(P, np.int32), np.zeros(S, np.int32)
    order = rng.permutation(P)
    for s in range(4):
        lengths[s] = [100, 63, 1, 129][s]
        n = (lengths[s] + 63) // 64
        table[s, :n], order = order[:n], order[n:]
        refs[table[s, :n]] = 1
    g = [torch.from_numpy(a.copy()).cuda() for a in (pool, table, lengths, refs)]
    src, dst = np.array([0, 0, 1, 2, 3], np.int32), np.array([4, 5, 6, 7, 8], np.int32)
    i32 = lambda a: torch.from_numpy(np.asarray(a, np.int32)).cuda()  # noqa: E731
    cu.fork(table, lengths, refs, src, dst)
    sv.pages_fork(*g[1:], i32(src), i32(dst))
    n_new = np.full(S, 3, np.int32)
    served, _ = cu.reserve(pool, table, lengths, refs, n_new)      # every sequence's last page is shared: nine copies
    assert served.all() and np.array_equal(sv.pages_reserve(*g, i32(n_new)).cpu().numpy(), served)
    for t, a in zip(g, (pool, table, lengths, refs)):
        assert np.array_equal(t.cpu().numpy(), a)
    assert int(sv.pages_compact(g[0], g[1], g[3])) == cu.compact(pool, table, refs)
    for t, a in zip(g, (pool, table, lengths, refs)):
        assert np.array_equal(t.cpu().numpy(), a)


def test_norm_and_attention_of_inputs_that_repeat_rows():
    """One row for every head (stride 0), also with a single sequence whose stride says nothing."""
    g = torch.Generator().manual_seed(4)
    row = torch.randn((3, 64), generator=g).bfloat16().cuda()
    q = row.as_strided((1, 3, 2, 64), (1, 64, 0, 1))
    pos, freqs = torch.arange(3, **I32)[None], sv.rope_frequencies(64)
    got, want = sv.qk_norm_rope(q, q, pos, freqs), sv.qk_norm_rope(q.contiguous(), q.contiguous(), pos, freqs)
    assert torch.equal(got["q"], want["q"]) and torch.equal(got["k"], want["k"])
    pool, table = sv.new_pool(2, 1, 64), torch.arange(2, **I32)[None]
    kv = torch.randn((1, 90, 1, 64), generator=g).bfloat16().cuda()
    sv.cache_append(pool, table, torch.zeros(1, **I32), kv, kv)
    lens = torch.tensor([90], **I32)
    assert torch.equal(sv.cache_attention(q, pool, table, lens)["out"], sv.cache_attention(q.contiguous(), pool, table, lens)["out"])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("D,R", [(64, 32), (128, 64), (128, 128), (256, 16), (64, 0)])
@pytest.mark.parametrize("inter", [False, True])
def test_norm_of_infinite_channels(dtype, D, R, inter):
    """A row with an infinity has an infinite norm: its finite channels are 0, the infinite one is NaN, and so is what a rotation mixes it
    with, but no other channel."""
    H = D + 1
    x = (torch.rand((1, 1, H, D), generator=torch.Generator().manual_seed(D)) + 0.5).to(dtype)
    for h in range(D):
        x[0, 0, h, h] = float("inf") if h % 2 else float("-inf")                  # the last head has none
    freqs = sv.rope_frequencies(R) if R else None
    q = sv.qk_norm_rope(x.cuda(), x[:, :, :1].cuda(), torch.full((1, 1), 5, **I32), freqs, interleaved=inter)["q"].cpu()[0, 0]
    for h in range(D):
        mate = h if h >= R else h ^ 1 if inter else (h + R // 2) % R
        want = torch.zeros(D, dtype=dtype)
        want[[h, mate]] = float("nan")
        assert torch.equal(q[h].isnan(), want.isnan()) and (q[h][~want.isnan()] == 0).all(), h
    assert torch.isfinite(q[D]).all() and (q[D] != 0).all()
