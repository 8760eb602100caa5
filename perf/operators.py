"""The operators of the target's scoring step around a verification, as cases to be measured.

A serving loop scores K + 1 tokens of every sequence with the target, verifies the drafts, keeps the accepted
ones and drops the rest. Around the verification it needs four operators, over a paged key / value cache held
in 4 bits:

- norm_rope: the norm of each query and key head and the rotation by the token's position;
- append: the new keys and values quantised into their pages, and the cached values read back;
- attend: the new tokens' attention over the cache, whole or with a sliding window and first tokens that stay;
- pages: forking sequences, reserving pages for drafts, committing the accepted length and freeing the rest;
  compacting the pages in use to the front of the pool.

The cache's format, for head size D and pages of 64 tokens: one block of 68 D bytes per page and key head,
[key codes 32 D][key scales 2 D][value codes 32 D][value scales 2 D]. A scale s is shared by a token's 32
neighbouring channels and held in 8 bits (5 of exponent, 3 of mantissa, no sign: the upper bits of a half). A
code c in -7..7 is held as c + 8 in 4 bits and stands for c s. Key codes are ordered [group of 32 channels]
[token][16 bytes, two neighbouring channels each], value codes [16 tokens][channel r < D / 2][token], a byte
holding channel r in its low and channel r + D / 2 in its high half; scales [token][group].
"""
import math

import torch

own = False

PAGE = 64
GROUP = 32
SCALE_TOP = 198          # the largest scale's bits: 896


# ------------------------------------------------------------------------------------------------------ the cases
def _attend(name, B, N, Hq, Hkv, D, lo, hi, dtype="bf16", window=0, sinks=0, lse=False):
    return dict(name=name, op="attend", B=B, N=N, Hq=Hq, Hkv=Hkv, D=D, lo=lo, hi=hi, dtype=dtype, window=window,
                sinks=sinks, lse=lse)


def _norm(name, B, N, Hq, Hkv, D, rot, far, dtype="bf16", weights=True, interleaved=False):
    return dict(name=name, op="norm_rope", B=B, N=N, Hq=Hq, Hkv=Hkv, D=D, rot=rot, far=far, dtype=dtype,
                weights=weights, interleaved=interleaved)


def _append(name, B, N, Hkv, D, hi, dtype="bf16", ragged=False):
    return dict(name=name, op="append", B=B, N=N, Hkv=Hkv, D=D, hi=hi, dtype=dtype, ragged=ragged)


def listed():
    return [
        # one user's next token after a short prompt: latency
        _attend("attend_one_short", 1, 1, 32, 8, 128, 700, 700, lse=True),
        # a batch that decodes without drafts, lengths as they come
        _attend("attend_single_ragged", 48, 1, 32, 8, 128, 130, 8191, dtype="fp16"),
        # K = 5 drafts and the last token scored for 64 sequences, the batch of the standard chain workload
        _attend("attend_chain", 64, 6, 32, 8, 128, 1000, 16384),
        # a layer with a sliding window and four sinks, heads of 64
        _attend("attend_window_sinks", 96, 6, 16, 4, 64, 100, 32768, window=4096, sinks=4, lse=True),
        # a few long documents, K = 8 drafts, eight query heads to a key head
        _attend("attend_long_chain", 4, 9, 64, 8, 128, 100001, 131072),
        # a draft chain's queries and keys of 64 sequences, at positions of a long context
        _norm("norm_rope_chain", 64, 6, 32, 8, 128, 128, 131072),
        # a prompt's tokens: many rows, bandwidth
        _norm("norm_rope_prompt", 4, 4096, 32, 8, 128, 128, 16384),
        # one token of a model that rotates half of each head's channels in neighbouring pairs, without weights
        _norm("norm_rope_one_partial", 1, 1, 8, 2, 64, 32, 1 << 20, dtype="fp32", weights=False, interleaved=True),
        # a draft chain's keys and values of 64 sequences
        _append("append_chain", 64, 6, 8, 128, 16384),
        # prompts of several lengths
        _append("append_prompt_ragged", 8, 4096, 8, 128, 777, dtype="fp16", ragged=True),
        # 64 sequences of which a quarter forks, reserve for six tokens and commit what was accepted
        dict(name="pages_round", op="pages", S=64, M=256, P=8192, Hkv=8, D=128, N=6, forks=16, window=0, sinks=0),
        # half the pages of a pool of two layers in use, spread out
        dict(name="compact_half", op="compact", S=64, M=128, P=8192, L=2, Hkv=8, D=128, used=0.5),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "norm_rope", "append", "pages", "compact"])
    D = rng.choice([64, 128])
    Hkv = _log(rng, 1, 8)
    G = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    dt = rng.choice(["bf16", "fp16"])
    if op == "attend":
        N = rng.choice([1, 1, _log(rng, 2, 33)])
        hi = _log(rng, 1, 131072)
        room = max(1, min(96, int(3e8 / (hi * Hkv * D))))
        B = _log(rng, 1, room)
        while B * hi * Hkv * G * N > 3e8 and N > 1:
            N = (N + 1) // 2
        windowed = rng.random() < 0.4
        return dict(op=op, B=B, N=N, Hq=Hkv * G, Hkv=Hkv, D=D, lo=rng.randint(max(1, hi // 8), hi), hi=hi, dtype=dt,
                    window=_log(rng, 1, 8192) if windowed else 0, sinks=rng.randint(0, 200) if windowed else 0,
                    lse=rng.random() < 0.5)
    if op == "norm_rope":
        N = rng.choice([1, _log(rng, 2, 4096)])
        B = _log(rng, 1, max(1, min(128, 16384 // N)))
        dt = rng.choice(["bf16", "fp16", "fp32"])
        Hq = min(Hkv * G, 40)
        return dict(op=op, B=B, N=N, Hq=Hq, Hkv=Hkv, D=D, rot=rng.choice([D, D, D // 2, 16]), far=_log(rng, 2, 1 << 20),
                    dtype=dt, weights=rng.random() < 0.7, interleaved=rng.random() < 0.4)
    if op == "append":
        N = rng.choice([1, _log(rng, 2, 4096)])
        return dict(op=op, B=_log(rng, 1, max(1, min(128, 32768 // N))), N=N, Hkv=Hkv, D=D, hi=_log(rng, 1, 16384),
                    dtype=dt, ragged=rng.random() < 0.5)
    if op == "pages":
        S = _log(rng, 2, 512)
        M = min(_log(rng, 8, 512), 32768 // S)
        N = rng.randint(1, min(65, 64 * M // 4))
        return dict(op=op, S=S, M=M, P=S * (M // 2 + 4) + rng.randint(0, 1000), Hkv=Hkv, D=64, N=N,
                    forks=rng.randint(0, S // 3), window=rng.choice([0, _log(rng, 1, 32 * M)]), sinks=rng.randint(0, 130))
    S, M = _log(rng, 1, 256), _log(rng, 4, 256)
    P = max(16, min(_log(rng, 16, 16384), 2 * S * M))
    return dict(op="compact", S=S, M=M, P=P, L=rng.randint(1, 2), Hkv=Hkv, D=64,
                used=min(rng.uniform(0.05, 0.95), S * M / P))


# ------------------------------------------------------------------------------------------------ inputs and sizes
def _type(name):
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[name]


def _lens(case):
    """Ragged lengths that depend on the case alone, so that its work does."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    return [hi if b == 0 else lo + int((hi - lo) * ((b * 0.6180339887498949) % 1.0)) for b in range(B)]


def _new_counts(case):
    B, N = case["B"], case["N"]
    return [N if b == 0 or not case["ragged"] else int(N * ((b * 0.7548776662466927) % 1.0)) for b in range(B)]


def _inv_freq(rot):
    return 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)


def _visible(length, n, window, sinks):
    """Cached tokens that any of the last n tokens of `length` sees."""
    if not window:
        return length
    first = max(0, length - n - window + 1)
    return length - first + min(sinks, first)


def _random_blocks(P, Hkv, D, gen, dev):
    """A pool of P pages of keys (some channels larger) and values, quantised."""
    pool = torch.empty((P, Hkv, 68 * D), dtype=torch.uint8, device=dev)
    gain = torch.exp(0.4 * torch.randn((Hkv, D), generator=gen, device=dev))
    step = max(1, (1 << 26) // (PAGE * Hkv * D))
    for a in range(0, P, step):
        n = min(step, P - a)
        k = torch.randn((n, PAGE, Hkv, D), generator=gen, device=dev) * gain
        v = torch.randn((n, PAGE, Hkv, D), generator=gen, device=dev)
        pool[a:a + n] = _pack(k.bfloat16().float(), v.bfloat16().float())
    return pool


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    op, D = case["op"], case["D"]
    st = dict(case=case)
    if op == "attend":
        B, N, Hq, Hkv, dt = case["B"], case["N"], case["Hq"], case["Hkv"], _type(case["dtype"])
        lens = _lens(case)
        M = (max(lens) + PAGE - 1) // PAGE
        counts = torch.tensor([(n + PAGE - 1) // PAGE for n in lens], device=dev)
        P = int(counts.sum()) + 3
        order = torch.randperm(P, generator=gen, device=dev).to(torch.int32)
        held = torch.arange(M, device=dev)[None, :] < counts[:, None]
        table = torch.full((B, M), -1, dtype=torch.int32, device=dev)
        table[held] = order[:int(counts.sum())]
        if case["window"]:      # pages that no later token sees are gone, as a commit leaves them
            j = torch.arange(M, device=dev)[None, :] * PAGE
            first = torch.tensor(lens, device=dev)[:, None] - N - case["window"] + 1
            table[(j >= case["sinks"]) & (j + PAGE <= first)] = -1
        qkv = torch.randn((B, N, Hq + 2 * Hkv, D), generator=gen, device=dev).to(dt)
        st.update(q=qkv[:, :, :Hq], pool=_random_blocks(P, Hkv, D, gen, dev), table=table,
                  kv_len=torch.tensor(lens, dtype=torch.int32, device=dev))
        if own:
            import speculative_decoding_verification_target_gb300 as sv
            st["workspace"] = sv.new_attention_workspace(N, Hq, Hkv, D)
    elif op == "norm_rope":
        B, N, Hq, Hkv, dt = case["B"], case["N"], case["Hq"], case["Hkv"], _type(case["dtype"])
        qkv = (2.0 * torch.randn((B, N, Hq + 2 * Hkv, D), generator=gen, device=dev)).to(dt)
        start = torch.randint(0, max(1, case["far"] - N), (B, 1), generator=gen, device=dev, dtype=torch.int32)
        st.update(q=qkv[:, :, :Hq], k=qkv[:, :, Hq:Hq + Hkv],
                  positions=(start + torch.arange(N, dtype=torch.int32, device=dev)).contiguous(),
                  inv_freq=_inv_freq(case["rot"]).to(dev), q_weight=None, k_weight=None)
        if case["weights"]:
            st["q_weight"] = (1 + 0.1 * torch.randn(D, generator=gen, device=dev)).to(dt)
            st["k_weight"] = (1 + 0.1 * torch.randn(D, generator=gen, device=dev)).to(dt)
        if own:
            import speculative_decoding_verification_target_gb300 as sv
            st["freqs"] = sv.rope_frequencies(case["rot"], 10000.0, device=dev)
    elif op == "append":
        B, N, Hkv, dt = case["B"], case["N"], case["Hkv"], _type(case["dtype"])
        qkv = torch.randn((B, N, 3 * Hkv, D), generator=gen, device=dev)
        qkv[:, :, Hkv:2 * Hkv] *= torch.exp(0.4 * torch.randn((Hkv, D), generator=gen, device=dev))
        qkv = qkv.to(dt)
        start = torch.randint(0, case["hi"], (B,), generator=gen, device=dev, dtype=torch.int32)
        M = (case["hi"] + N + PAGE - 1) // PAGE
        order = torch.randperm(B * M, generator=gen, device=dev).to(torch.int32)
        st.update(k=qkv[:, :, Hkv:2 * Hkv], v=qkv[:, :, 2 * Hkv:], start=start, table=order.view(B, M).contiguous(),
                  n_new=torch.tensor(_new_counts(case), dtype=torch.int32, device=dev),
                  pool=torch.zeros((B * M, Hkv, 68 * D), dtype=torch.uint8, device=dev))
        if own:
            import speculative_decoding_verification_target_gb300 as sv
            st["workspace"] = sv.new_pages_workspace(B, B * M, device=dev)
    elif op == "pages":
        S, M, P, N, F = case["S"], case["M"], case["P"], case["N"], case["forks"]
        cap = (M // 2) * PAGE - N
        lengths = torch.randint(0, max(1, cap), (S,), generator=gen, device=dev, dtype=torch.int32)
        perm = torch.randperm(S, generator=gen, device=dev).to(torch.int32)
        src, dst = perm[:F].contiguous(), perm[F:2 * F].contiguous()
        lengths[dst.long()] = 0
        counts = (lengths.long() + PAGE - 1) // PAGE
        held = torch.arange(M, device=dev)[None, :] < counts[:, None]
        order = torch.randperm(P, generator=gen, device=dev).to(torch.int32)
        table = torch.full((S, M), -1, dtype=torch.int32, device=dev)
        table[held] = order[:int(counts.sum())]
        refs = torch.zeros(P, dtype=torch.int32, device=dev)
        refs[order[:int(counts.sum())].long()] = 1
        st.update(table=table, lengths=lengths, refs=refs, src=src, dst=dst,
                  n_new=torch.full((S,), N, dtype=torch.int32, device=dev),
                  accept=torch.randint(0, N, (S,), generator=gen, device=dev, dtype=torch.int32),
                  pool=torch.randint(0, 256, (P, case["Hkv"], 68 * D), generator=gen, device=dev, dtype=torch.uint8))
        if own:
            import speculative_decoding_verification_target_gb300 as sv
            st["workspace"] = sv.new_pages_workspace(S, P, device=dev)
    else:
        S, M, P = case["S"], case["M"], case["P"]
        n = _used(case)
        order = torch.randperm(P, generator=gen, device=dev).to(torch.int32)
        slots = torch.randperm(S * M, generator=gen, device=dev)[:n]
        table = torch.full((S * M,), -1, dtype=torch.int32, device=dev)
        table[slots] = order[:n]
        refs = torch.zeros(P, dtype=torch.int32, device=dev)
        refs[order[:n].long()] = 1
        st.update(table=table.view(S, M), refs=refs,
                  pool=torch.randint(0, 256, (case["L"], P, case["Hkv"], 68 * D), generator=gen, device=dev,
                                     dtype=torch.uint8))
        if own:
            import speculative_decoding_verification_target_gb300 as sv
            st["workspace"] = sv.new_pages_workspace(S, P, device=dev)
    return st


def _used(case):
    return max(1, min(case["S"] * case["M"], int(case["used"] * case["P"])))


# --------------------------------------------------------------------------------------------------- plain forms
def _scale_bits(v):
    """Positive fp32 to the nearest 5-bit-exponent, 3-bit-mantissa value's bits (ties to even)."""
    bits = v.contiguous().view(torch.int32)
    normal = ((bits + 0x7FFFF + ((bits >> 20) & 1)) >> 20) - (112 << 3)
    small = torch.round(v * 131072.0).to(torch.int32)
    return torch.where(v < 2.0 ** -14, small, normal).clamp(max=SCALE_TOP)


def _scale_value(b):
    """The value of a scale's bits: those of a half, seven places up."""
    return (b.to(torch.int16) << 7).view(torch.float16).float()


def _codes(x):
    """x [..., D] in fp32 to codes + 8 [..., D] and scale bits [..., D / 32]."""
    g = x.unflatten(-1, (-1, GROUP))
    top = g.abs().amax(-1)
    b = _scale_bits(top / torch.full_like(top, 7.0))     # a tensor divisor: an exact quotient, rounded once
    s = _scale_value(b)[..., None]
    c = torch.where(s > 0, torch.round(g / s), torch.zeros_like(g)).clamp(-7, 7)
    return (c.to(torch.int32) + 8).flatten(-2).to(torch.uint8), b.to(torch.uint8)


def _pack(k, v):
    """Whole pages: k, v [P, 64, Hkv, D] fp32 to blocks [P, Hkv, 68 D]."""
    P, _, H, D = k.shape
    kc, ks = _codes(k)
    vc, vs = _codes(v)
    kb = (kc[..., 0::2] | (kc[..., 1::2] << 4)).view(P, PAGE, H, D // 32, 16).permute(0, 2, 3, 1, 4).reshape(P, H, 32 * D)
    vb = (vc[..., :D // 2] | (vc[..., D // 2:] << 4)).view(P, 4, 16, H, D // 2).permute(0, 3, 1, 4, 2).reshape(P, H, 32 * D)
    return torch.cat([kb, ks.permute(0, 2, 1, 3).reshape(P, H, 2 * D), vb, vs.permute(0, 2, 1, 3).reshape(P, H, 2 * D)], -1)


def _unpack(blocks):
    """Blocks [..., 68 D] to k, v [..., 64, D] fp32."""
    D = blocks.shape[-1] // 68
    G = D // GROUP
    kb, ks, vb, vs = blocks.split([32 * D, 2 * D, 32 * D, 2 * D], -1)
    kb = kb.unflatten(-1, (G, PAGE, 16)).transpose(-3, -2)
    k = torch.stack([kb & 15, kb >> 4], -1).flatten(-2).float() - 8.0               # [..., 64, G, 32]
    k = (k * _scale_value(ks.unflatten(-1, (PAGE, G)))[..., None]).flatten(-2)
    vb = vb.unflatten(-1, (4, D // 2, 16)).transpose(-2, -1)
    v = torch.cat([vb & 15, vb >> 4], -1).flatten(-3, -2).float() - 8.0             # [..., 64, D]
    v = (v.unflatten(-1, (G, GROUP)) * _scale_value(vs.unflatten(-1, (PAGE, G)))[..., None]).flatten(-2)
    return k, v


def _plain_attend(st):
    case, q, kv_len = st["case"], st["q"], st["kv_len"]
    B, N, Hq, D = q.shape
    H = case["Hkv"]
    G = Hq // H
    k, v = _unpack(st["pool"][st["table"].clamp(min=0).long()].transpose(1, 2))     # [B, H, M, 64, D]
    k, v = k.flatten(2, 3), v.flatten(2, 3)
    qq = q.float().unflatten(2, (H, G)).permute(0, 2, 1, 3, 4).reshape(B, H, N * G, D)
    s = (torch.matmul(qq, k.transpose(-1, -2)) * D ** -0.5).view(B, H, N, G, -1)
    at = torch.arange(s.shape[-1], device=q.device)[None, None, :]
    pos = (kv_len[:, None] - N + torch.arange(N, device=q.device))[:, :, None]
    seen = at <= pos
    if case["window"]:
        seen = seen & ((at > pos - case["window"]) | (at < case["sinks"]))
    s = torch.where(seen[:, None, :, None, :], s, torch.full_like(s, -math.inf))
    top = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e.view(B, H, N * G, -1), v).view(B, H, N, G, D) / torch.where(total > 0, total, torch.ones_like(total))
    out = {"out": o.permute(0, 2, 1, 3, 4).reshape(B, N, Hq, D).to(q.dtype)}
    if case["lse"]:
        out["lse"] = (top + torch.log(total)).squeeze(-1).permute(0, 2, 1, 3).reshape(B, N, Hq)
    return out


def _plain_norm_rope(st):
    case = st["case"]
    R = case["rot"]
    turn = st["positions"].double()[:, :, None, None] * st["inv_freq"]
    cos, sin = torch.cos(turn).float(), torch.sin(turn).float()

    def one(x, w):
        y = x.float()
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + 1e-6)
        if w is not None:
            y = y * w.float()
        r, rest = y[..., :R], y[..., R:]
        if case["interleaved"]:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = r[..., :R // 2], r[..., R // 2:]
            r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([r, rest], -1).to(x.dtype)

    return {"q": one(st["q"], st["q_weight"]), "k": one(st["k"], st["k_weight"])}


def _plain_append(st):
    """The new tokens into the pool's blocks, and the same tokens read back."""
    k, v, pool, table, start = st["k"], st["v"], st["pool"], st["table"], st["start"]
    B, N, H, D = k.shape
    dev = k.device
    G = D // GROUP
    i = torch.arange(N, device=dev)[None, :]
    pos = start[:, None].long() + i
    live = i < st["n_new"][:, None]
    page = torch.gather(table, 1, torch.clamp(pos // PAGE, max=table.shape[1] - 1)).long()
    kc, ks = _codes(k.float())
    vc, vs = _codes(v.float())
    t = (pos % PAGE)[live][:, None, None]                                   # [tokens, 1, 1]
    where = page[live][:, None, None]
    head = torch.arange(H, device=dev)[None, :, None]
    byte = torch.arange(D // 2, device=dev)[None, None, :]
    grp = torch.arange(G, device=dev)[None, None, :]
    pool[where, head, (byte // 16) * (PAGE * 16) + t * 16 + byte % 16] = (kc[..., 0::2] | (kc[..., 1::2] << 4))[live]
    pool[where, head, 32 * D + t * G + grp] = ks[live]
    pool[where, head, 34 * D + (t // 16) * (D * 8) + byte * 16 + t % 16] = (vc[..., :D // 2] | (vc[..., D // 2:] << 4))[live]
    pool[where, head, 66 * D + t * G + grp] = vs[live]
    zero = torch.zeros((B, N, H, D), dtype=k.dtype, device=dev)
    blocks = pool[page[live], :]                                            # [tokens, H, 68 D]
    kb = blocks[..., :32 * D].view(-1, H, G, PAGE, 16)
    kb = torch.gather(kb, 3, t[:, :, :, None, None].expand(-1, H, G, 1, 16)).squeeze(3)
    vb = blocks[..., 34 * D:66 * D].view(-1, H, 4, D // 2, 16).transpose(-1, -2).flatten(2, 3)
    vb = torch.gather(vb, 2, t[:, :, :, None].expand(-1, H, 1, D // 2)).squeeze(2)
    ks = torch.gather(blocks[..., 32 * D:34 * D].view(-1, H, PAGE, G), 2, t[:, :, :, None].expand(-1, H, 1, G)).squeeze(2)
    vs = torch.gather(blocks[..., 66 * D:].view(-1, H, PAGE, G), 2, t[:, :, :, None].expand(-1, H, 1, G)).squeeze(2)
    kk = (torch.stack([kb & 15, kb >> 4], -1).flatten(-2).float() - 8.0) * _scale_value(ks)[..., None]
    vv = (torch.cat([vb & 15, vb >> 4], -1).float() - 8.0).unflatten(-1, (G, GROUP)) * _scale_value(vs)[..., None]
    ok, ov = zero, zero.clone()
    ok[live] = kk.flatten(-2).to(k.dtype)
    ov[live] = vv.flatten(-2).to(k.dtype)
    return {"k": ok, "v": ov}


def _plain_pages(st):
    """Fork, reserve (with a copy of a shared last page) and commit, on copies of the bookkeeping."""
    case, pool = st["case"], st["pool"]
    table, lengths, refs = st["table"].clone(), st["lengths"].clone(), st["refs"].clone()
    S, M, P, N = case["S"], case["M"], case["P"], case["N"]
    dev = table.device
    j = torch.arange(M, device=dev)[None, :]
    src, dst = st["src"].long(), st["dst"].long()
    # fork: the destination's pages are dropped, the source's are shared
    old, new = table[dst], table[src]
    refs.index_add_(0, old[old >= 0].long(), torch.full_like(old[old >= 0], -1))
    refs.index_add_(0, new[new >= 0].long(), torch.ones_like(new[new >= 0]))
    table[dst], lengths[dst] = new, lengths[src]
    # reserve: the k-th page wanted, by sequence and position, is the k-th free one
    a, z = lengths[:, None] // PAGE, (lengths + st["n_new"] - 1)[:, None] // PAGE
    fits = (z < M) & (st["n_new"][:, None] > 0)
    held = table >= 0
    shared = held & (refs[table.clamp(min=0).long()] > 1)
    want = (j >= a) & (j <= z) & fits & (~held | shared)
    running = want.sum(1).cumsum(0)
    free = torch.nonzero(refs == 0).squeeze(1)
    served = ((running <= free.numel()) | (want.sum(1) == 0)) & (fits.squeeze(1) | (st["n_new"] <= 0))
    want = want & served[:, None]
    give = free[:int(want.sum())]
    was = table[want]
    copy = (want & held & (j == a) & (lengths % PAGE != 0)[:, None])[want]
    pool[give[copy]] = pool[was[copy].long()]
    refs.index_add_(0, was[was >= 0].long(), torch.full_like(was[was >= 0], -1))
    refs[give] = 1
    table[want] = give.to(torch.int32)
    # commit: the accepted tokens and the one before them stay; pages past the end, or out of every later view, go
    lengths = lengths + st["accept"] + 1
    gone = j >= (lengths[:, None] + PAGE - 1) // PAGE
    if case["window"]:
        gone = gone | ((j * PAGE >= case["sinks"]) & ((j + 1) * PAGE <= lengths[:, None] - case["window"] + 1))
    gone = gone & (table >= 0)
    refs.index_add_(0, table[gone].long(), torch.full_like(table[gone], -1))
    table = torch.where(gone, torch.full_like(table, -1), table)
    return {"table": table, "lengths": lengths, "refs": refs, "served": served.to(torch.int32), "pool": pool}


def _plain_compact(st):
    table, refs, pool = st["table"], st["refs"], st["pool"]
    used = refs > 0
    n = int(used.sum())
    ids = torch.arange(refs.numel(), device=refs.device)
    movers, holes = ids[used & (ids >= n)], ids[~used & (ids < n)]
    to = ids.clone()
    to[movers] = holes
    pool[:, holes] = pool[:, movers]
    new_refs = refs.clone()
    new_refs[holes] = refs[movers]
    new_refs[movers] = 0
    return {"table": torch.where(table >= 0, to[table.clamp(min=0).long()].to(torch.int32), table), "refs": new_refs,
            "used": used.sum().to(torch.int32).view(1), "pool": pool}


def run(st):
    case = st["case"]
    op = case["op"]
    if own:
        import speculative_decoding_verification_target_gb300 as sv
        if op == "attend":
            r = sv.cache_attention(st["q"], st["pool"], st["table"], st["kv_len"], window=case["window"],
                                   sinks=case["sinks"], want_lse=case["lse"], workspace=st["workspace"])
            return {"out": r["out"], "lse": r["lse"]} if case["lse"] else {"out": r["out"]}
        if op == "norm_rope":
            r = sv.qk_norm_rope(st["q"], st["k"], st["positions"], st["freqs"], q_weight=st["q_weight"],
                                k_weight=st["k_weight"], eps=1e-6, interleaved=case["interleaved"])
            return {"q": r["q"], "k": r["k"]}
        if op == "append":
            sv.cache_append(st["pool"], st["table"], st["start"], st["k"], st["v"], counts=st["n_new"],
                            workspace=st["workspace"])
            r = sv.cache_read(st["pool"], st["table"], st["start"], case["N"], counts=st["n_new"],
                              dtype=st["k"].dtype, workspace=st["workspace"])
            return {"k": r["k"], "v": r["v"]}
        if op == "pages":
            table, lengths, refs = st["table"].clone(), st["lengths"].clone(), st["refs"].clone()
            sv.pages_fork(table, lengths, refs, st["src"], st["dst"], workspace=st["workspace"])
            served = sv.pages_reserve(st["pool"], table, lengths, refs, st["n_new"], workspace=st["workspace"])
            sv.pages_commit(table, lengths, refs, st["accept"], extra=1, window=case["window"], sinks=case["sinks"],
                            workspace=st["workspace"])
            return {"table": table, "lengths": lengths, "refs": refs, "served": served, "pool": st["pool"]}
        table, refs = st["table"].clone(), st["refs"].clone()
        used = sv.pages_compact(st["pool"], table, refs, workspace=st["workspace"])
        return {"table": table, "refs": refs, "used": used, "pool": st["pool"]}
    return {"attend": _plain_attend, "norm_rope": _plain_norm_rope, "append": _plain_append, "pages": _plain_pages,
            "compact": _plain_compact}[op](st)


# --------------------------------------------------------------------------------------------------------- work
def work(case):
    op, D = case["op"], case["D"]
    if op == "attend":
        N, Hq, H = case["N"], case["Hq"], case["Hkv"]
        seen = sum(_visible(n, N, case["window"], case["sinks"]) for n in _lens(case))
        rows = case["B"] * N * Hq
        return {"bytes": seen * H * (D + D // 16) + 4 * rows * D + (4 * rows if case["lse"] else 0),
                "flops": 4 * seen * N * Hq * D}
    if op == "norm_rope":
        e = 4 if case["dtype"] == "fp32" else 2
        n = case["B"] * case["N"] * (case["Hq"] + case["Hkv"]) * D
        return {"bytes": 2 * e * n, "flops": 8 * n}
    if op == "append":
        n = sum(_new_counts(case)) * case["Hkv"] * D
        # 16 bits in and 4.25 out for each key and value, and back
        return {"bytes": 2 * n * (2 + 0.53125) + 2 * n * 0.53125 + 4 * case["B"] * case["N"] * case["Hkv"] * D,
                "flops": 12 * n}
    if op == "pages":
        S, M, P = case["S"], case["M"], case["P"]
        copies = 2 * case["forks"]
        return {"bytes": 8 * S * M + 8 * P + copies * 2 * case["Hkv"] * 68 * D, "flops": 4 * S * M + P}
    n, P = _used(case), case["P"]
    moved = n * (P - n) // P
    return {"bytes": 2 * moved * case["L"] * case["Hkv"] * 68 * D + 8 * case["S"] * case["M"] + 8 * P,
            "flops": P + case["S"] * case["M"]}


# ------------------------------------------------------------------------------------- the definitions in 64 bits
def _exact_table(dev):
    """The value in 64 bits of each of the 256 scale bytes, from its fields."""
    vals = [m * 2.0 ** -17 if e == 0 else (8 + m) * 2.0 ** (e - 18) for e in range(32) for m in range(8)]
    return torch.tensor(vals, dtype=torch.float64, device=dev)


def _exact_token_rows(pool, page, tok, h, D, scales):
    """Keys and values in 64 bits of the tokens (page, tok) of head h, channel by channel."""
    d = torch.arange(D, device=pool.device)[None, :]
    p, t = page[:, None], tok[:, None]
    kb = pool[p, h, (d // 32) * 1024 + t * 16 + (d % 32) // 2].long()
    kn = torch.where(d % 2 == 0, kb % 16, kb // 16)
    ks = scales[pool[p, h, 32 * D + t * (D // 32) + d // 32].long()]
    vb = pool[p, h, 34 * D + (t // 16) * (8 * D) + (d % (D // 2)) * 16 + t % 16].long()
    vn = torch.where(d < D // 2, vb % 16, vb // 16)
    vs = scales[pool[p, h, 66 * D + t * (D // 32) + d // 32].long()]
    return (kn - 8).double() * ks, (vn - 8).double() * vs


def _exact_attend(case, st):
    q, pool, table = st["q"].double(), st["pool"], st["table"].long()
    B, N, Hq, D = q.shape
    H = case["Hkv"]
    G = Hq // H
    scales = _exact_table(q.device)
    out = torch.zeros((B, N, Hq, D), dtype=torch.float64, device=q.device)
    lse = torch.full((B, N, Hq), -math.inf, dtype=torch.float64, device=q.device)
    for b, n in enumerate(_lens(case)):
        first = max(0, n - N - case["window"] + 1) if case["window"] else 0
        at = torch.arange(n, device=q.device)
        at = at[(at >= first) | (at < case["sinks"])] if case["window"] else at
        pos = n - N + torch.arange(N, device=q.device)[:, None]
        seen = at[None, :] <= pos
        if case["window"]:
            seen = seen & ((pos - at[None, :] < case["window"]) | (at[None, :] < case["sinks"]))
        hide = torch.zeros_like(seen, dtype=torch.float64).masked_fill(~seen, -math.inf)
        for h in range(H):
            k, v = _exact_token_rows(pool, table[b, at // PAGE], at % PAGE, h, D, scales)
            s = torch.einsum("ngd,ld->ngl", q[b, :, h * G:(h + 1) * G], k) / math.sqrt(D) + hide[:, None, :]
            z = torch.logsumexp(s, -1)
            w = torch.exp(s - torch.where(torch.isfinite(z), z, torch.zeros_like(z))[..., None])
            out[b, :, h * G:(h + 1) * G] = torch.einsum("ngl,ld->ngd", w, v)
            lse[b, :, h * G:(h + 1) * G] = z
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}


def _exact_norm_rope(case, st):
    R = case["rot"]
    theta = st["positions"].double()[..., None, None] * st["inv_freq"]
    spin = torch.polar(torch.ones_like(theta), theta)

    def one(x, w):
        y = x.double()
        y = y * torch.rsqrt(y.square().sum(-1, keepdim=True) / y.shape[-1] + 1e-6)
        y = y if w is None else y * w.double()
        if case["interleaved"]:
            z = torch.view_as_complex(y[..., :R].unflatten(-1, (R // 2, 2)).contiguous()) * spin
            y[..., :R] = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(y[..., :R // 2], y[..., R // 2:R]) * spin
            y[..., :R // 2], y[..., R // 2:R] = z.real, z.imag
        return y

    return {"q": one(st["q"], st["q_weight"]), "k": one(st["k"], st["k_weight"])}


def _exact_append(case, st):
    """Each value the nearest multiple (even on ties, at most seven) of the representable scale nearest to a
    seventh of its group's largest magnitude."""
    grid = _exact_table(st["k"].device)[:SCALE_TOP + 1]
    live = torch.arange(case["N"], device=grid.device)[None, :] < st["n_new"][:, None]

    def one(x):
        g = x.double().unflatten(-1, (-1, 32))
        v = g.abs().amax(-1, keepdim=True) / 7
        hi = torch.searchsorted(grid, v.contiguous()).clamp(max=SCALE_TOP)
        lo = (hi - 1).clamp(min=0)
        up, down = (grid[hi] - v).abs(), (v - grid[lo]).abs()
        s = grid[torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)]
        c = torch.where(s > 0, torch.round(g / torch.where(s > 0, s, torch.ones_like(s))), torch.zeros_like(g))
        return torch.where(live[..., None, None], (c.clamp(-7, 7) * s).flatten(-2), torch.zeros((), dtype=torch.float64,
                                                                                              device=x.device))

    return {"k": one(st["k"]), "v": one(st["v"])}


def exact(case, seed):
    op = case["op"]
    if op in ("pages", "compact"):
        return None             # whole numbers: compared for equality
    st = prepare(case, seed)
    if op == "attend":
        return _exact_attend(case, st)
    return _exact_norm_rope(case, st) if op == "norm_rope" else _exact_append(case, st)
