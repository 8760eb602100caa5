"""A small serving loop with drafts: scoring over the 4-bit paged cache, verification, commit.

A one-layer target (head norms, rotation, grouped queries, sliding window with sinks if wanted) and a bigram drafter,
both with random weights, extend a batch of prompts. Every round the drafter proposes K tokens per sequence, the target
scores the last token and the K drafts in one pass over the cache, spec_verify's chain accepts a prefix and draws one
token more, and the pages' commit keeps exactly the accepted tokens. Half-way, sequence 0 is forked into the spare
slot, which from then on shares its pages and goes its own way; at the end the pool is compacted.

    python examples/serve_drafts.py [--rounds 24] [--window 0]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import speculative_decoding_verification_target_gb300 as sv  # noqa: E402


class Target:
    """Embedding, one attention layer over the cache, a gated feed-forward part and the vocabulary's logits."""

    def __init__(self, vocab=2048, width=512, q_heads=8, kv_heads=2, head_dim=64, seed=0, window=0, sinks=4, int8=False):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.Hq, self.Hk, self.D, self.window, self.sinks = q_heads, kv_heads, head_dim, window, sinks

        def w(*shape):
            return (torch.randn(shape, generator=g, device="cuda") * shape[0] ** -0.5).bfloat16()

        self.embed = torch.randn((vocab, width), generator=g, device="cuda").bfloat16()
        self.qkv, self.o = w(width, (q_heads + 2 * kv_heads) * head_dim), w(q_heads * head_dim, width)
        self.up, self.down, self.head = w(width, 4 * width), w(2 * width, width), 4 * w(width, vocab)
        self.q_weight = self.k_weight = torch.ones(head_dim, dtype=torch.bfloat16, device="cuda")
        self.freqs = sv.rope_frequencies(head_dim, 10000.0)
        # a row of 8-bit weights is an output channel
        self.int8 = {k: sv.quantize_rows(getattr(self, k).t().contiguous()) for k in ("up", "down", "head")} if int8 else None
        self._product_ws = {}

    def product(self, name, codes):
        """Tokens in 8 bits (out, scale) times one of the weights in 8 bits."""
        a, w = codes["out"], self.int8[name]
        tokens = a.shape[0] * a.shape[1]
        if tokens > max(self._product_ws, default=0):      # the one for the most tokens serves every call with fewer
            weights = [m["out"].shape for m in self.int8.values()]
            self._product_ws = {tokens: sv.new_matmul_workspace(tokens, max(C for C, _ in weights), max(K for _, K in weights))}
        workspace, = self._product_ws.values()
        return sv.int8_matmul(a, codes["scale"], w["out"], w["scale"], workspace=workspace)["out"]

    def project(self, tokens, positions):
        """The new tokens' residual stream, rotated queries and keys, and values."""
        x = self.embed[tokens.long()]
        B, N = tokens.shape
        qkv = (x @ self.qkv).view(B, N, self.Hq + 2 * self.Hk, self.D)
        r = sv.qk_norm_rope(qkv[:, :, :self.Hq], qkv[:, :, self.Hq:self.Hq + self.Hk], positions, self.freqs,
                            q_weight=self.q_weight, k_weight=self.k_weight)
        return x, r["q"], r["k"], qkv[:, :, self.Hq + self.Hk:]

    def finish(self, x, attended):
        if self.int8:
            r = sv.residual_norm(attended.flatten(2) @ self.o, x, quantize=True)
            a, b = self.product("up", r).chunk(2, -1)
            inner = sv.quantize_rows(torch.nn.functional.silu(a) * b)
            r = sv.residual_norm(self.product("down", inner), r["residual"], quantize=True)
            return self.product("head", r)
        x = x + attended.flatten(2) @ self.o
        a, b = (x @ self.up).chunk(2, -1)
        return (x + (torch.nn.functional.silu(a) * b) @ self.down) @ self.head

    def score(self, cache, tokens, counts):
        """Logits [B, N, vocab] of the new tokens, which are appended to the cache; counts[b] of them are real."""
        step = torch.arange(tokens.shape[1], dtype=torch.int32, device="cuda")
        x, q, k, v = self.project(tokens, cache.lengths[:, None] + step)
        sv.cache_append(cache.pool, cache.table, cache.lengths, k, v, counts=counts, workspace=cache.pages_ws)
        r = sv.cache_attention(q, cache.pool, cache.table, cache.lengths + counts, q_len=counts, window=self.window,
                               sinks=self.sinks, workspace=cache.attention_ws(q))
        return self.finish(x, r["out"])


class Cache:
    """The pool with its bookkeeping; a slot of length 0 is free."""

    def __init__(self, target, slots, pages, max_pages):
        i32 = dict(dtype=torch.int32, device="cuda")
        self.pool = sv.new_pool(pages, target.Hk, target.D)
        self.table = torch.full((slots, max_pages), -1, **i32)
        self.lengths, self.refs = torch.zeros(slots, **i32), torch.zeros(pages, **i32)
        self.pages_ws = sv.new_pages_workspace(slots, pages)
        self.target, self._ws = target, {}

    def attention_ws(self, q):
        N = q.shape[1]
        if N not in self._ws:
            self._ws[N] = sv.new_attention_workspace(N, self.target.Hq, self.target.Hk, self.target.D)
        return self._ws[N]

    def reserve(self, counts):
        return sv.pages_reserve(self.pool, self.table, self.lengths, self.refs, counts, workspace=self.pages_ws)

    def commit(self, advance, extra=1):
        sv.pages_commit(self.table, self.lengths, self.refs, advance, extra=extra, window=self.target.window,
                        sinks=self.target.sinks, workspace=self.pages_ws)

    def status(self):
        return sv.read_status(self.pages_ws) | max(sv.read_status(w) for w in self._ws.values())


def draft(bigram, last, K, temperature, gen):
    """K tokens per sequence from the bigram table, with their logits."""
    tokens, logits = [], []
    for _ in range(K):
        row = bigram[last.long()]
        u = torch.rand(row.shape, generator=gen, device="cuda").clamp_(1e-20, 1 - 1e-7)
        last = (row.float() / temperature - torch.log(-torch.log(u))).argmax(-1).to(torch.int32)
        tokens.append(last)
        logits.append(row)
    return torch.stack(tokens, 1), torch.stack(logits, 1).contiguous()


def process(logits, text, prompts, proposed, penalties, allowed):
    """The target's logits with the penalties over each slot's text and the drafts before a row, and with the mask."""
    i32 = dict(dtype=torch.int32, device="cuda")
    longest = max(1, max(map(len, text)))
    history = torch.tensor([t + [-1] * (longest - len(t)) for t in text], **i32)
    lengths = torch.tensor([len(t) for t in text], **i32)
    rates = {k: torch.full((len(text),), float(v), device="cuda") for k, v in (penalties or {}).items()}
    mask = None if allowed is None else allowed.expand(logits.shape[0], logits.shape[1], -1)
    return sv.process_logits(logits, tokens=proposed, history=history, lengths=lengths, prompt=torch.tensor(prompts, **i32),
                             mask=mask, out=logits, **rates)["out"]


def serve(rounds=24, K=4, prompts=(37, 64, 5, 130), window=0, seed=0, temperature=1.0, int8=False, penalties=None, allowed=None):
    """Returns the cache, the target, every slot's tokens, and the accepted lengths [rounds, slots]. penalties: dict(repetition,
    frequency, presence), any of them; allowed: a mask int32 [vocab / 32] of the tokens that may come."""
    target = Target(seed=seed, window=window, int8=int8)
    slots, S = len(prompts) + 1, len(prompts)
    cache = Cache(target, slots, pages=64, max_pages=8)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    vocab = target.embed.shape[0]
    bigram = target.finish(target.embed[None], torch.zeros((1, vocab, target.Hq, target.D), dtype=torch.bfloat16,
                                                           device="cuda"))[0].contiguous()
    text = [torch.randint(0, vocab, (n,), generator=gen, device="cuda", dtype=torch.int32).tolist() for n in prompts] + [[]]
    # the prompts, all but their last tokens, in one pass
    counts = torch.tensor([len(t) - 1 if t else 0 for t in text], dtype=torch.int32, device="cuda")
    N = int(counts.max())
    first = torch.tensor([(t[:-1] + [0] * N)[:N] for t in text], dtype=torch.int32, device="cuda")
    assert bool(cache.reserve(counts).all())
    target.score(cache, first, counts)
    cache.commit(counts, extra=0)
    seeds = torch.arange(slots, dtype=torch.int64, device="cuda") + 1000 * (seed + 1)
    accepted = []
    for r in range(rounds):
        if r == rounds // 2:      # the spare slot continues sequence 0 by itself
            sv.pages_fork(cache.table, cache.lengths, cache.refs, torch.zeros(1, dtype=torch.int32, device="cuda"),
                          torch.full((1,), S, dtype=torch.int32, device="cuda"), workspace=cache.pages_ws)
            text[S] = list(text[0])
        live = torch.tensor([bool(t) for t in text], device="cuda")
        last = torch.tensor([t[-1] if t else 0 for t in text], dtype=torch.int32, device="cuda")
        proposed, draft_logits = draft(bigram, last, K, temperature, gen)
        counts = torch.where(live, K + 1, 0).to(torch.int32)
        served = cache.reserve(counts)
        assert bool(served.all())
        logits = target.score(cache, torch.cat([last[:, None], proposed], 1), counts).contiguous()
        if penalties or allowed is not None:      # the drafts keep the distribution that they were drawn from
            logits = process(logits, text, list(prompts) + [prompts[0]], proposed, penalties, allowed)
        v = sv.verify(logits, draft_logits, proposed, seeds + r * slots, temperature, want_diag=False)
        # a free slot stays empty: its advance takes the one token back that every live sequence gains
        cache.commit(torch.where(live, v["accept_len"], -1).to(torch.int32))
        accepted.append(v["accept_len"].tolist())
        for t, n, out in zip(text, accepted[-1], v["out_tokens"].tolist()):
            if t:
                t.extend(out[:n + 1])
    return cache, target, text, accepted


def main():
    a = argparse.ArgumentParser()
    a.add_argument("--rounds", type=int, default=24)
    a.add_argument("--window", type=int, default=0)
    a.add_argument("--int8", action="store_true")
    a.add_argument("--penalties", action="store_true")
    o = a.parse_args()
    rates = dict(repetition=1.2, frequency=0.3, presence=0.2) if o.penalties else None
    cache, target, text, accepted = serve(o.rounds, window=o.window, int8=o.int8, penalties=rates)
    used = sv.pages_compact(cache.pool, cache.table, cache.refs, workspace=cache.pages_ws)
    print("mean accepted drafts a round: %.2f" % (sum(map(sum, accepted)) / sum(map(len, accepted))))
    print("tokens per slot: %s, cached: %s" % ([len(t) for t in text], cache.lengths.tolist()))
    print("pages in use: %d, at the front of the pool; status %d" % (int(used), cache.status()))


if __name__ == "__main__":
    main()
