"""The serving example end to end: the cache holds exactly the committed text, forks go their own way, and the target's
logits over the 4-bit cache are those of plain attention over the values that the cache holds."""
import os
import sys

import pytest
import torch

import speculative_decoding_verification_target_gb300 as sv

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window", [0, 70])
def test_serving_loop(window):
    import serve_drafts as ex
    prompt = [100, 64, 5, 130]
    cache, target, text, accepted = ex.serve(rounds=16, prompts=prompt, window=window)
    lengths = cache.lengths.tolist()
    assert cache.status() == 0
    assert lengths == [len(t) - 1 for t in text]                   # all but the last token, which the next round scores
    for s, n in enumerate(prompt):
        assert len(text[s]) == n + sum(a[s] + 1 for a in accepted)
    table, refs = cache.table.cpu(), cache.refs.cpu()
    assert torch.equal(torch.bincount(table[table >= 0].flatten(), minlength=refs.numel()).to(torch.int32), refs)
    forked = len(text[0]) - sum(a[0] + 1 for a in accepted[8:])
    assert text[4][:forked] == text[0][:forked] and text[4] != text[0]
    if not window:                                                 # the forked prefix's full pages are held once
        assert table[0, :(forked - 1) // 64].tolist() == table[4, :(forked - 1) // 64].tolist() and int(refs.max()) == 2
    # the cached keys and values are those of the committed text
    for s in range(5):
        t = torch.tensor(text[s][:-1], dtype=torch.int32, device="cuda")[None]
        pos = torch.arange(t.shape[1], dtype=torch.int32, device="cuda")[None]
        x, q, k, v = target.project(t, pos)
        fresh = sv.new_pool(8, target.Hk, target.D)
        one = torch.arange(8, dtype=torch.int32, device="cuda")[None]
        zero = torch.zeros(1, dtype=torch.int32, device="cuda")
        sv.cache_append(fresh, one, zero, k, v)
        want = sv.cache_read(fresh, one, zero, t.shape[1])
        row = cache.table[s:s + 1].contiguous()
        got = sv.cache_read(cache.pool, row, zero, t.shape[1])
        held = (row[0] >= 0).repeat_interleave(64)[:t.shape[1]]
        assert held.all() or window
        # projections of one row at a time and of many may differ in the last place of bf16, which moves few codes by one step
        for name in ("k", "v"):
            d = (got[name].float() - want[name].float())[0][held].abs()
            assert (d <= 0.6).all() and (d > 0).float().mean() < 0.02
    # one more token over the cache, against plain attention in fp64 over what the cache holds
    last = torch.tensor([t[-1] for t in text], dtype=torch.int32, device="cuda")[:, None]
    ones = torch.ones(5, dtype=torch.int32, device="cuda")
    before = cache.lengths.clone()
    assert bool(cache.reserve(ones).all())
    logits = target.score(cache, last, ones).double()
    n = int(before.max()) + 1
    read = sv.cache_read(cache.pool, cache.table, torch.zeros_like(before), n)
    x, q, _, _ = target.project(last, before[:, None])
    G = target.Hq // target.Hk
    k, v = (read[a].double().repeat_interleave(G, 2) for a in ("k", "v"))
    sc = torch.einsum("bnhd,bthd->bhnt", q.double(), k) * target.D ** -0.5
    at = torch.arange(n, device="cuda")[None, None, None]
    see = at <= before[:, None, None, None]
    if window:
        see &= (at > before[:, None, None, None] - window) | (at < target.sinks)
    att = torch.einsum("bhnt,bthd->bnhd", sc.masked_fill(~see, -torch.inf).softmax(-1), v)
    want = target.finish(x, att.bfloat16()).double()
    # both go through the same bf16 products from an attention that is the same to a step of bf16
    assert (logits - want).abs().max() <= 2.0 ** -5 * want.abs().max()


def test_serving_is_lossless_in_distribution_of_the_first_token():
    """The first emitted token of a round follows the target's distribution over the cache, whatever the drafter: over many
    seeds, its frequencies on a small vocabulary are the target's probabilities (five standard deviations)."""
    import serve_drafts as ex
    target = ex.Target(vocab=16, width=128, seed=3)
    S, K = 2048, 2
    cache = ex.Cache(target, S, pages=S, max_pages=1)
    prompt = torch.randint(0, 16, (1, 9), generator=torch.Generator().manual_seed(1), dtype=torch.int32).cuda()
    eight = torch.full((S,), 8, dtype=torch.int32, device="cuda")
    assert bool(cache.reserve(eight).all())
    target.score(cache, prompt[:, :8].expand(S, 8).contiguous(), eight)
    cache.commit(eight, extra=0)
    gen = torch.Generator(device="cuda").manual_seed(5)
    bigram = torch.randn((16, 16), generator=gen, device="cuda").bfloat16()
    last = prompt[:, 8].expand(S).contiguous()
    proposed, dl = ex.draft(bigram, last, K, 1.0, gen)
    counts = torch.full((S,), K + 1, dtype=torch.int32, device="cuda")
    assert bool(cache.reserve(counts).all())
    logits = target.score(cache, torch.cat([last[:, None], proposed], 1), counts).contiguous()
    v = sv.verify(logits, dl, proposed, torch.arange(S, dtype=torch.int64, device="cuda") + 77, 1.0, want_diag=False)
    p = logits[0, 0].double().softmax(-1)
    freq = torch.bincount(v["out_tokens"][:, 0].long(), minlength=16).double() / S
    assert ((freq - p).abs() <= 5 * (p * (1 - p) / S).sqrt() + 1e-9).all()
