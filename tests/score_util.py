"""Plain forms in 64 bits of the operators between the last layer and a verification, and how far fp32 arithmetic may be off."""
import torch


def exact_codes(p):
    """p [rows, D] in fp32: the integers nearest to 127 p / m, even on ties, by comparing whole products."""
    p = p.double()
    m = p.abs().amax(1, keepdim=True)
    c = torch.floor(127.0 * p / torch.where(m > 0, m, torch.ones_like(m)))
    twice = 254.0 * p - (2.0 * c + 1.0) * m
    c = c + ((twice > 0) | ((twice == 0) & (c % 2 != 0))).double()
    return torch.where(m > 0, c, torch.zeros_like(c)).to(torch.int8), m[:, 0] / 127.0


def norm(x, residual, weight, eps):
    """r in x's type, p in fp32 values, 1 / sqrt(mean(r^2) + eps), v in 64 bits."""
    r = x if residual is None else (x.double() + residual.double()).to(x.dtype)
    d = r.double()
    w = torch.ones_like(d[0]) if weight is None else weight.double()
    inv = (d.square().mean(1) + eps).rsqrt()
    return r, (d * w).float(), inv, d * w * inv[:, None]


def inv_tol(D):
    """1 / sqrt of a sum of D squares in fp32, relative: a lane adds at most D / 32 of them in a row and sixteen partial sums behind
    that, each addition half a step of 2^-23, of which the root leaves half; eight more for the mean, eps, root and products."""
    return ((D / 32 + 16) / 2 + 8) * 2.0 ** -24


def half_step(y, dtype):
    """Half a step of dtype at y, subnormal ones too."""
    return torch.finfo(dtype).eps / 2 * y.abs() + torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def logits(x, tokens=None, history=None, lengths=None, prompt=None, repetition=None, frequency=None, presence=None,
           bias_tokens=None, bias=None, mask=None):
    """[B, R, V] in 64 bits, what fp32 may be off by, and where the logits are as they were."""
    B, R, V = x.shape
    out, tol, same = x.double().clone(), torch.zeros(B, R, V, dtype=torch.float64), torch.ones(B, R, V, dtype=torch.bool)
    for b in range(B):
        asked, said, add = set(), {}, {}
        if history is not None:
            n = min(max(int(lengths[b]), 0), history.shape[1])
            for i, t in enumerate(history[b, :n].tolist()):
                if 0 <= t < V:
                    if prompt is not None and i < int(prompt[b]):
                        asked.add(t)
                    else:
                        said[t] = said.get(t, 0) + 1
        if bias_tokens is not None:
            add = {t: float(v) for t, v in zip(bias_tokens[b].tolist(), bias[b].tolist()) if 0 <= t < V}
        rep = 1.0 if repetition is None else float(repetition[b])
        freq = 0.0 if frequency is None else float(frequency[b])
        pres = 0.0 if presence is None else float(presence[b])
        for j in range(R):
            if j and tokens is not None and 0 <= int(tokens[b, j - 1]) < V:
                said[int(tokens[b, j - 1])] = said.get(int(tokens[b, j - 1]), 0) + 1
            for t in set(add) | asked | set(said):
                y = float(x[b, j, t]) + add.get(t, 0.0)
                mag = abs(float(x[b, j, t])) + abs(add.get(t, 0.0))
                if t in asked or t in said:
                    y = y / rep if y > 0 else y * rep
                    mag *= max(rep, 1 / rep)
                if t in said:
                    y -= freq * said[t] + pres
                    mag += freq * said[t] + pres
                # five operations of fp32, none on more than mag
                out[b, j, t], tol[b, j, t], same[b, j, t] = y, 5 * 2.0 ** -24 * mag, False
            if mask is not None:
                bits = torch.tensor([(w >> i) & 1 for w in mask[b, j].tolist() for i in range(32)], dtype=torch.bool)[:V]
                out[b, j][~bits] = -torch.inf
                same[b, j][~bits] = False
    return out, tol, same
