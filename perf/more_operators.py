"""The operators between the target's last layer and a verification, as cases to be measured.

A verification takes the target's logits as they are sampled from. Before that, a serving loop runs four operators:

- norm: the residual's addition and the root-mean-square norm of each token, x + residual = r and
  v = r w / sqrt(mean(r^2) + eps), with v in the activations' type or in 8-bit integers with a scale per token;
- quantize: a token's values in 8-bit integers with a scale, without a norm;
- matmul: the product of 8-bit integers with scales for each token and each output channel;
- logits: biases, penalties for repeated tokens and grammar masks on the logits of the tokens to be verified.

Formats. r is rounded to the activations' type T, as it is kept; the norm is taken from r. In 8 bits: p = r w rounded to
fp32 (exact where T has 16 bits; r alone without a weight), m the row's largest |p|, code = the integer nearest to
127 p / m (even on ties; 0 where m = 0), scale = m / 127, times 1 / sqrt(mean(r^2) + eps) with a norm. The codes do not depend on
the mean, so they are decided without any rounding, and come out as the whole numbers that they are, beside their scales.

The product: out[m, n] = T(sum_k a[m, k] w[n, k] a_scale[m] w_scale[n] + bias[n]).

The logits of row j of a sequence stand after its history and the drafts before j. With n the times that a token is among
the history's output part and those drafts: y = x + bias; if the token is in the history or those drafts, y / rep where
y > 0, else y rep; minus frequency n, minus presence where n > 0; -inf where the row's mask (32 tokens a word, lowest bit first) has a 0.
"""
import math

import torch

own = False

EPS = 1e-6


# ------------------------------------------------------------------------------------------------------ the cases
def _norm(name, rows, D, dtype="bf16", codes=True, residual=True, weight=True):
    return dict(name=name, op="norm", rows=rows, D=D, dtype=dtype, codes=codes, residual=residual, weight=weight)


def _quantize(name, rows, D, dtype="bf16"):
    return dict(name=name, op="quantize", rows=rows, D=D, dtype=dtype)


def _matmul(name, M, N, K, dtype="bf16", bias=False):
    return dict(name=name, op="matmul", M=M, N=N, K=K, dtype=dtype, bias=bias)


def _logits(name, B, R, V, L, dtype="bf16", biases=0, mask=False):
    return dict(name=name, op="logits", B=B, R=R, V=V, L=L, dtype=dtype, biases=biases, mask=mask)


def listed():
    return [
        # one token of one user: latency
        _norm("norm_one", 1, 4096),
        # the last token and K = 5 drafts of 64 sequences, in 8 bits for the product behind it
        _norm("norm_chain", 384, 8192),
        # prompts' tokens: bandwidth
        _norm("norm_prompt", 16384, 4096),
        # an odd width, 16-bit outputs, as in front of a product in 16 bits
        _norm("norm_odd_fp16", 5001, 2050 + 1, dtype="fp16", codes=False),
        # the attention's output of a draft chain, in front of its projection
        _quantize("quantize_chain", 384, 4096),
        # the inner values of a prompt's feed-forward part
        _quantize("quantize_prompt", 8192, 14336),
        # one token's projection: the weights' bytes
        _matmul("matmul_one", 1, 4096, 4096),
        # the vocabulary's product for the standard chain workload, 64 sequences of 6 tokens
        _matmul("matmul_head_chain", 384, 128256, 4096),
        # a prompt's feed-forward product
        _matmul("matmul_prompt", 8192, 14336, 4096),
        # one row at the Llama-3 vocabulary with penalties, as a drafter's step has: latency
        _logits("logits_one", 1, 1, 128256, 2000),
        # the standard chain workload under grammars and with biases
        _logits("logits_chain", 64, 6, 128256, 8192, biases=64, mask=True),
        # the target's rows of the longest chain workload at the Qwen vocabulary, long histories
        _logits("logits_long_chain", 128, 21, 151936, 32768),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "quantize", "matmul", "matmul", "matmul", "logits", "logits"])
    dt = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op in ("norm", "quantize"):
        D = _log(rng, 16, 16384)
        if rng.random() < 0.6:
            D = max(16, D // 16 * 16)
        rows = _log(rng, 1, max(1, min(16384, (1 << 25) // D)))
        if op == "quantize":
            return dict(op=op, rows=rows, D=D, dtype=dt)
        return dict(op=op, rows=rows, D=D, dtype=dt, codes=rng.random() < 0.6, residual=rng.random() < 0.7,
                    weight=rng.random() < 0.8)
    if op == "matmul":
        K = 16 * _log(rng, 1, 1024)
        N = _log(rng, 1, min(128256, int(5.2e8 / K)))
        top = min(8192, int(1e8 / K), int(2e8 / N), int(2e11 / (N * K)))
        if rng.random() < 0.2:          # a width that is no multiple of 16 bytes
            K, top = K - rng.randint(1, 15), max(1, top // 16)
        return dict(op=op, M=_log(rng, 1, max(1, top)), N=N, K=K, dtype=dt, bias=rng.random() < 0.3)
    V = _log(rng, 1000, 262144)
    if rng.random() < 0.5:
        V = V // 64 * 64
    R = rng.randint(1, 21)
    B = _log(rng, 1, max(1, min(128, int(2e8 / (V * R)))))
    return dict(op=op, B=B, R=R, V=V, L=_log(rng, 1, 32768), dtype=rng.choice(["bf16", "fp32"]),
                biases=rng.choice([0, 0, _log(rng, 1, 300)]), mask=rng.random() < 0.5)


# ------------------------------------------------------------------------------------------------ inputs and sizes
def _type(name):
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[name]


def _lengths(case):
    """Ragged history lengths and prompt parts that depend on the case alone, so that its work does."""
    B, L = case["B"], case["L"]
    full = [L if b == 0 else L // 8 + int((L - L // 8) * ((b * 0.6180339887498949) % 1.0)) for b in range(B)]
    return full, [int(n * (0.2 + 0.6 * ((b * 0.7548776662466927) % 1.0))) for b, n in enumerate(full)]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    op, st = case["op"], dict(case=case)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    def rand(*shape):
        return torch.rand(shape, generator=gen, device=dev)

    if op in ("norm", "quantize"):
        rows, D, dt = case["rows"], case["D"], _type(case["dtype"])
        gain = torch.exp(0.7 * randn(D))         # some channels are larger than others, as a residual stream's are
        st.update(x=(randn(rows, D) * gain).to(dt), residual=None, weight=None)
        if op == "norm" and case["residual"]:
            st["residual"] = (3.0 * randn(rows, D) * gain).to(dt)
        if op == "norm" and case["weight"]:
            st["weight"] = (1 + 0.2 * randn(D)).to(dt)
    elif op == "matmul":
        M, N, K = case["M"], case["N"], case["K"]

        def codes(rows, sigma):
            return torch.round(sigma * randn(rows, K)).clamp_(-127, 127).to(torch.int8)

        st.update(a=codes(M, 32.0), a_scale=0.02 * (0.5 + rand(M)), w=codes(N, 36.0),
                  w_scale=(0.5 + rand(N)) / (36.0 * math.sqrt(K)), bias=randn(N) if case["bias"] else None)
        if own:
            import speculative_decoding_verification_target_gb300 as sv
            st["workspace"] = sv.new_matmul_workspace(M, N, K)
    else:
        B, R, V, L = case["B"], case["R"], case["V"], case["L"]
        x = 3.0 * randn(B, R, V)
        at = torch.randint(0, V, (B, R, 20), generator=gen, device=dev)
        x.scatter_(-1, at, x.gather(-1, at) + 8.0)

        def text(n):      # few tokens often, many seldom
            return (rand(B, n).pow(3) * V).long().clamp_(max=V - 1).to(torch.int32)

        full, prompt = (torch.tensor(v, dtype=torch.int32, device=dev) for v in _lengths(case))
        history = text(L)
        history[torch.arange(L, device=dev)[None, :] >= full[:, None]] = -1
        on = rand(3, B) < 0.8                    # some sequences leave a penalty out
        st.update(logits=x.to(_type(case["dtype"])), tokens=text(R), history=history, lengths=full, prompt=prompt,
                  repetition=torch.where(on[0], 1.0 + 0.5 * rand(B), torch.ones(B, device=dev)),
                  frequency=torch.where(on[1], rand(B), torch.zeros(B, device=dev)),
                  presence=torch.where(on[2], rand(B), torch.zeros(B, device=dev)), bias_tokens=None, bias=None, mask=None)
        n = case["biases"]
        if n:             # tokens of their own, some entries unused
            step = V // n
            ids = (torch.arange(n, device=dev) * step + torch.randint(0, step, (B, n), generator=gen, device=dev)).to(torch.int32)
            ids[rand(B, n) < 0.1] = -1
            st.update(bias_tokens=ids, bias=4.0 * randn(B, n))
        if case["mask"]:  # a grammar allows everything, about half of the tokens, or a few
            W = (V + 31) // 32
            words = torch.randint(-2 ** 31, 2 ** 31, (B, R, W), generator=gen, device=dev)
            few = torch.where(rand(B, R, W) < 0.02, words, torch.zeros_like(words))
            few[..., 0] |= 1
            kind = rand(B, R, 1)
            st["mask"] = torch.where(kind < 0.3, torch.full_like(words, -1), torch.where(kind < 0.6, words, few)).to(torch.int32)
    return st


# --------------------------------------------------------------------------------------------------- plain forms
def _codes(p):
    """fp32 rows to codes and the scale's m / 127; the quotients in 64 bits, since a border decides a whole number."""
    m = p.abs().amax(-1, keepdim=True)
    q = torch.round(127.0 * p.double() / torch.where(m > 0, m, torch.ones_like(m)).double())
    return q.to(torch.int8), m[..., 0] / 127.0


def _plain_norm(st):
    case, x = st["case"], st["x"]
    r = x if st["residual"] is None else (x.float() + st["residual"].float()).to(x.dtype)
    f = r.float()
    p = f if st["weight"] is None else f * st["weight"].float()
    inv = torch.rsqrt(f.square().mean(-1) + EPS)
    out = {} if st["residual"] is None else {"residual": r}
    if case["codes"]:
        q, s = _codes(p)
        return {"out": q, "scale": s * inv, **out}
    return {"out": (p * inv[:, None]).to(x.dtype), **out}


def _plain_quantize(st):
    q, s = _codes(st["x"].float())
    return {"out": q, "scale": s}


def _plain_matmul(st):
    y = torch.matmul(st["a"].float(), st["w"].float().t()) * (st["a_scale"][:, None] * st["w_scale"])
    if st["bias"] is not None:
        y = y + st["bias"]
    return {"out": y.to(_type(st["case"]["dtype"]))}


def _plain_logits(st):
    x = st["logits"]
    B, R, V = x.shape
    dev = x.device
    at = torch.arange(st["history"].shape[1], device=dev)[None, :]
    ids = st["history"].long()
    known = (at < st["lengths"][:, None]) & (ids >= 0) & (ids < V)
    ids = torch.where(known, ids, torch.full_like(ids, V))
    made = (at >= st["prompt"][:, None]).int()
    seen = torch.zeros((B, V + 1), dtype=torch.int32, device=dev).scatter_add_(1, ids, torch.ones_like(made))
    count = torch.zeros((B, V + 1), dtype=torch.int32, device=dev).scatter_add_(1, ids, made)
    drafts = torch.zeros((B, R, V), dtype=torch.int32, device=dev)
    if R > 1:
        drafts[:, 1:].scatter_(2, st["tokens"][:, :R - 1].long()[..., None], 1)
        drafts = drafts.cumsum(1, dtype=torch.int32)
    count = count[:, None, :V] + drafts
    seen = (seen[:, None, :V] + drafts) > 0
    y = x.float()
    if st["bias_tokens"] is not None:
        t = st["bias_tokens"].long()
        t = torch.where(t >= 0, t, torch.full_like(t, V))
        y = y + torch.zeros((B, V + 1), device=dev).scatter_(1, t, st["bias"])[:, None, :V]
    rep = st["repetition"][:, None, None]
    y = torch.where(seen, torch.where(y > 0, y / rep, y * rep), y)
    y = y - st["frequency"][:, None, None] * count - st["presence"][:, None, None] * (count > 0)
    if st["mask"] is not None:
        v = torch.arange(V, device=dev)
        y = torch.where((st["mask"][..., v // 32] >> (v % 32)) & 1 > 0, y, torch.full_like(y, -math.inf))
    return {"out": y.to(x.dtype)}


# ----------------------------------------------------------------------------------------------------- one pass
def run(state):
    st, op = state, state["case"]["op"]
    if own:
        import speculative_decoding_verification_target_gb300 as sv
        if op == "norm":
            r = sv.residual_norm(st["x"], st["residual"], st["weight"], EPS, quantize=st["case"]["codes"])
            return {k: v for k, v in r.items() if v is not None}
        if op == "quantize":
            return sv.quantize_rows(st["x"])
        if op == "matmul":
            return {"out": sv.int8_matmul(st["a"], st["a_scale"], st["w"], st["w_scale"], bias=st["bias"],
                                          dtype=_type(st["case"]["dtype"]), workspace=st["workspace"])["out"]}
        return sv.process_logits(st["logits"], tokens=st["tokens"], history=st["history"], lengths=st["lengths"],
                                 prompt=st["prompt"], repetition=st["repetition"], frequency=st["frequency"],
                                 presence=st["presence"], bias_tokens=st["bias_tokens"], bias=st["bias"], mask=st["mask"])
    return {"norm": _plain_norm, "quantize": _plain_quantize, "matmul": _plain_matmul, "logits": _plain_logits}[op](st)


# --------------------------------------------------------------------------------------------------------- work
def work(case):
    op, e = case["op"], 4 if case["dtype"] == "fp32" else 2
    if op in ("norm", "quantize"):
        n, rows = case["rows"] * case["D"], case["rows"]
        if op == "quantize":
            return {"bytes": (e + 1) * n + 4 * rows, "flops": 3 * n}
        out = n + 4 * rows if case["codes"] else e * n
        return {"bytes": e * n * (3 if case["residual"] else 1) + out + (e * case["D"] if case["weight"] else 0), "flops": 6 * n}
    if op == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": M * K + N * K + e * M * N + 4 * (M + N) + (4 * N if case["bias"] else 0), "flops": 2 * M * N * K}
    n = case["B"] * case["R"] * case["V"]
    words = case["B"] * case["R"] * ((case["V"] + 31) // 32) if case["mask"] else 0
    return {"bytes": 2 * e * n + 4 * words + 4 * sum(_lengths(case)[0]) + 4 * case["B"] * (case["R"] + 5 + 2 * case["biases"]),
            "flops": 4 * n}


# ------------------------------------------------------------------------------------- the definitions in 64 bits
def _exact_rows(case, st):
    """Norm and quantisation: each code is the integer c with |127 p - c m| smallest, the even one of two."""
    x = st["x"].double()
    D = x.shape[1]
    r, out = x, {}
    if st["residual"] is not None:
        out["residual"] = x + st["residual"].double()
        r = out["residual"].to(st["x"].dtype).double()
    p = r if st["weight"] is None else (r * st["weight"].double()).float().double()
    inv = (r.pow(2).sum(1) / D + EPS).pow(-0.5) if case["op"] == "norm" else torch.ones_like(x[:, 0])
    if case["op"] == "norm" and not case["codes"]:
        w = 1.0 if st["weight"] is None else st["weight"].double()
        return {"out": r * w * inv[:, None], **out}
    m = p.abs().max(1).values
    c = torch.floor(127.0 * p / m.clamp(min=1e-300)[:, None])
    twice = 254.0 * p - (2.0 * c + 1.0) * m[:, None]            # sign: above or below the middle of c and c + 1
    c = c + ((twice > 0) | ((twice == 0) & (c % 2 != 0))).double()
    return {"out": torch.where(m[:, None] > 0, c, torch.zeros_like(c)).to(torch.int8), "scale": m / 127.0 * inv, **out}


def _exact_matmul(case, st):
    w, s = st["w"], st["w_scale"].double()
    out = torch.empty((case["M"], case["N"]), dtype=torch.float64, device=w.device)
    for i in range(0, case["N"], 8192):
        n = slice(i, min(i + 8192, case["N"]))
        out[:, n] = torch.einsum("mk,nk->mn", st["a"].double(), w[n].double()) * s[n]
    out = out * st["a_scale"].double()[:, None]
    return {"out": out if st["bias"] is None else out + st["bias"].double()}


def _exact_logits(case, st):
    B, R, V = case["B"], case["R"], case["V"]
    dev = st["logits"].device
    out = torch.empty((B, R, V), dtype=torch.float64, device=dev)
    shift = torch.arange(32, device=dev)
    full, prompt = _lengths(case)
    for b in range(B):
        h = st["history"][b].long()
        asked, said = h[:prompt[b]], h[prompt[b]:full[b]]
        rep, freq, pres = (float(st[k][b]) for k in ("repetition", "frequency", "presence"))
        add = torch.zeros(V, dtype=torch.float64, device=dev)
        if st["bias_tokens"] is not None:
            used = st["bias_tokens"][b] >= 0
            add[st["bias_tokens"][b][used].long()] = st["bias"][b][used].double()
        in_prompt = torch.bincount(asked, minlength=V) > 0
        for j in range(R):
            n = torch.bincount(torch.cat([said, st["tokens"][b, :j].long()]), minlength=V)
            y = st["logits"][b, j].double() + add
            hit = in_prompt | (n > 0)
            y[hit] = torch.where(y[hit] > 0, y[hit] / rep, y[hit] * rep)
            y = y - freq * n.double() - pres * (n > 0).double()
            if st["mask"] is not None:
                allowed = ((st["mask"][b, j].long()[:, None] >> shift) % 2 != 0).flatten()[:V]
                y[~allowed] = -math.inf
            out[b, j] = y
    return {"out": out}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("norm", "quantize"):
        return _exact_rows(case, st)
    return _exact_matmul(case, st) if case["op"] == "matmul" else _exact_logits(case, st)
