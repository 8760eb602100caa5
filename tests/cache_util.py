"""Plain 64-bit forms of the 4-bit cache's operators for the tests: numpy, one token or page at a time, written from the
definitions in include/speccache.h."""
import numpy as np

PAGE = 64


def scale_grid():
    """The 199 representable scales, ascending: byte b is the half with bits b << 7."""
    return (np.arange(199, dtype=np.uint16) << 7).view(np.float16).astype(np.float64)


def quantise(x):
    """x [..., D] (float64) to codes + 8 and scale bytes, by search over the representable scales."""
    grid = scale_grid()
    g = np.nan_to_num(x, nan=0.0, posinf=1e30, neginf=-1e30).reshape(x.shape[:-1] + (-1, 32))
    v = np.minimum(np.abs(g).max(-1) / 7.0, 1e30)
    hi = np.clip(np.searchsorted(grid, v), 0, 198)
    lo = np.maximum(hi - 1, 0)
    up, down = np.abs(grid[hi] - v), np.abs(v - grid[lo])
    b = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    s = grid[b][..., None]
    c = np.where(s > 0, np.rint(g / np.where(s > 0, s, 1.0)), 0.0)
    c = np.where(np.isnan(x.reshape(g.shape)), 0.0, np.clip(c, -7, 7))
    return (c.reshape(x.shape) + 8).astype(np.uint8), b.astype(np.uint8)


def write_token(pool, page, h, t, kc, kb, vc, vb):
    """One token's codes and scale bytes into pool[page, h] (uint8)."""
    D = kc.shape[0]
    blk = pool[page, h]
    for d in range(0, D, 2):
        blk[(d // 32) * 1024 + t * 16 + (d % 32) // 2] = kc[d] | (kc[d + 1] << 4)
    for r in range(D // 2):
        blk[34 * D + (t // 16) * 8 * D + r * 16 + t % 16] = vc[r] | (vc[r + D // 2] << 4)
    n = D // 32
    blk[32 * D + t * n:32 * D + (t + 1) * n] = kb
    blk[66 * D + t * n:66 * D + (t + 1) * n] = vb


def block_values(blk):
    """A block's keys and values [64, D] in float64 (scale bytes past the grid are read as the half they are)."""
    D = blk.shape[0] // 68
    n = D // 32
    val = lambda b: (b.astype(np.uint16) << 7).view(np.float16).astype(np.float64)  # noqa: E731
    kb = blk[:32 * D].reshape(n, 64, 16).transpose(1, 0, 2)
    k = np.stack([kb & 15, kb >> 4], -1).reshape(64, D).astype(np.float64) - 8
    vb = blk[34 * D:66 * D].reshape(4, D // 2, 16).transpose(0, 2, 1).reshape(64, D // 2)
    v = np.concatenate([vb & 15, vb >> 4], -1).astype(np.float64) - 8
    ks, vs = val(blk[32 * D:34 * D].reshape(64, n)), val(blk[66 * D:].reshape(64, n))
    return k * np.repeat(ks, 32, 1), v * np.repeat(vs, 32, 1)


def attention(q, pool, table, kv_len, q_len, scale, window=0, sinks=0):
    """out, lse, and per output the bound's parts: sum p |v|, the largest sum |q k| scale among visible tokens, sum |v|."""
    B, N, Hq, D = q.shape
    P, H = pool.shape[:2]
    G = Hq // H
    out = np.zeros((B, N, Hq, D))
    mass = np.zeros((B, N, Hq, D))
    total = np.zeros((B, N, Hq, D))
    big = np.zeros((B, N, Hq))
    lse = np.full((B, N, Hq), -np.inf)
    for b in range(B):
        n = min(max(int(kv_len[b]), 0), table.shape[1] * PAGE)
        ql = min(max(int(q_len[b]), 0), N)
        for h in range(H):
            k, v, held = np.zeros((n, D)), np.zeros((n, D)), np.zeros(n, bool)
            for j in range((n + PAGE - 1) // PAGE):
                page = table[b, j]
                if 0 <= page < P:
                    kk, vv = block_values(pool[page, h])
                    m = min(PAGE, n - j * PAGE)
                    k[j * PAGE:j * PAGE + m], v[j * PAGE:j * PAGE + m] = kk[:m], vv[:m]
                    held[j * PAGE:j * PAGE + m] = True
            at = np.arange(n)
            for i in range(ql):
                pos = n - ql + i
                see = held & (at <= pos)
                if window:
                    see &= (at > pos - window) | (at < sinks)
                if not see.any():
                    continue
                for g in range(G):
                    x = q[b, i, h * G + g]
                    s = k[see] @ x * scale
                    m = s.max()
                    e = np.exp(s - m)
                    p = e / e.sum()
                    out[b, i, h * G + g] = p @ v[see]
                    mass[b, i, h * G + g] = p @ np.abs(v[see])
                    total[b, i, h * G + g] = np.abs(v[see]).sum(0)
                    big[b, i, h * G + g] = (np.abs(k[see]) @ np.abs(x)).max() * abs(scale)
                    lse[b, i, h * G + g] = m + np.log(e.sum())
    return out, lse, mass, big, total


def fork(table, lengths, refs, src, dst):
    S = table.shape[0]
    bad = 0
    for f in range(len(src)):
        if not (0 <= src[f] < S and 0 <= dst[f] < S) or dst[f] in src or dst[f] in dst[:f]:
            bad = 32
            continue
        for p in table[dst[f]]:
            if p >= 0:
                refs[p] -= 1
        table[dst[f]] = table[src[f]]
        for p in table[dst[f]]:
            if p >= 0:
                refs[p] += 1
        lengths[dst[f]] = lengths[src[f]]
    return bad


def reserve(pool, table, lengths, refs, n_new):
    """pool [layers, pages, ...]. Returns served and the status bits."""
    S, M = table.shape
    was = refs.copy()
    free = [p for p in range(len(refs)) if refs[p] <= 0]
    served, status, asked = np.zeros(S, np.int32), 0, 0
    for s in range(S):
        if n_new[s] <= 0:
            served[s] = 1
            continue
        end = int(lengths[s]) + int(n_new[s])
        if lengths[s] < 0 or end > M * PAGE:
            status |= 8
            continue
        want = [j for j in range(lengths[s] // PAGE, (end - 1) // PAGE + 1) if table[s, j] < 0 or was[table[s, j]] > 1]
        first = asked
        asked += len(want)
        if want and asked > len(free):
            status |= 16
            continue
        served[s] = 1
        for j, p in zip(want, free[first:asked]):
            old = table[s, j]
            if old >= 0:
                refs[old] -= 1
                if j == lengths[s] // PAGE and lengths[s] % PAGE:
                    pool[:, p] = pool[:, old]
            refs[p] = 1
            table[s, j] = p
    return served, status


def commit(table, lengths, refs, advance, extra, window, sinks):
    S, M = table.shape
    status = 0
    for s in range(S):
        raw = int(lengths[s]) + int(advance[s]) + extra
        n = min(max(raw, 0), M * PAGE)
        status |= 8 if n != raw else 0
        lengths[s] = n
        for j in range(M):
            gone = j * PAGE >= n or (window and j * PAGE >= sinks and j * PAGE + 63 < n - window + 1)
            if gone and table[s, j] >= 0:
                refs[table[s, j]] -= 1
                table[s, j] = -1
    return status


def compact(pool, table, refs):
    """pool [layers, pages, ...]. Returns the number of pages in use."""
    n = int((refs > 0).sum())
    movers = [p for p in range(n, len(refs)) if refs[p] > 0]
    holes = [p for p in range(n) if refs[p] <= 0]
    for a, z in zip(movers, holes):
        pool[:, z] = pool[:, a]
        refs[z], refs[a] = refs[a], 0
        table[table == a] = z
    return n
