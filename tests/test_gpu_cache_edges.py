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
