"""Plain 64-bit forms of rotary positions, of attention with a mask, and of forked and freed
pages, written from their formulas."""
import numpy as np


def angles(turns, positions):
    """Radians of each position and pair, from whole numbers of 2^-64ths of a turn, without rounding but the last."""
    frac = [[(int(p) * int(t)) % 2 ** 64 / 2 ** 64 for t in turns] for p in positions]
    return 2 * np.pi * np.array(frac, np.float64).reshape(len(positions), len(turns))


def rotate(x, angle, rot, interleaved, gain=1.0, inverse=False):
    """float64 x [tokens, heads, 128] -> (turned, per element gain (|a| + |b|) of its pair, 0 where nothing turns)."""
    i = np.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    c, s = gain * np.cos(angle)[:, None], gain * np.sin(angle)[:, None] * (-1 if inverse else 1)
    y, size = x.copy(), np.zeros_like(x)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    size[..., a] = size[..., b] = abs(gain) * (np.abs(x[..., a]) + np.abs(x[..., b]))
    return y, size


def attention(q, k, v, scale, seen):
    """float64 q [n, Hq, 128], k, v [kv, H, 128], seen [n, kv] -> (o, lse [n, Hq], a, s): a = sum p |v| / sum p and
    s = the largest scale sum |q_d k_d| of the row, for error bounds.  A hidden key takes no part, whatever it holds."""
    n, Hq, _ = q.shape
    H = k.shape[1]
    G = Hq // H
    o, a = np.zeros((n, Hq, 128)), np.zeros((n, Hq, 128))
    lse, s = np.full((n, Hq), -np.inf), np.zeros((n, Hq))
    for i in range(n):
        j = np.flatnonzero(seen[i])
        if not len(j):
            continue
        for h in range(H):
            hs = slice(h * G, (h + 1) * G)
            with np.errstate(invalid="ignore"):
                x = scale * q[i, hs] @ k[j, h].T
                top = x.max(-1, keepdims=True)
                p = np.exp(x - top)
                t = p.sum(-1, keepdims=True)
                lse[i, hs] = (top + np.log(t))[:, 0]
                o[i, hs] = p @ v[j, h] / t
                a[i, hs] = p @ np.abs(v[j, h]) / t
                s[i, hs] = (scale * np.abs(q[i, hs]) @ np.abs(k[j, h]).T).max(-1)
    return o, lse, a, s


def window_mask(n, kv, window, sinks):
    p, j = kv - n + np.arange(n)[:, None], np.arange(kv)
    return (j <= p) & ((j > p - window) | (j < sinks))


def fork(table, src, dst, lens, refs, ring, head, tail, page):
    """Fork by fork; table and refs are updated -> (from, to, lens, state)."""
    a, b, kept, want = [], [], [], 0
    for s, d, n in zip(src, dst, lens):
        whole = n // page
        for j in range(whole):
            table[d][j] = table[s][j]
            refs[table[s][j]] += 1
        pair = (-1, -1)
        if n % page:
            if want < tail - head:
                pair = (table[s][whole], ring[(head + want) % len(ring)])
            else:
                n = whole * page
            want += 1
            table[d][whole] = pair[1]
        a.append(pair[0])
        b.append(pair[1])
        kept.append(n)
    took = min(want, tail - head)
    return a, b, kept, [head + took, tail, want - took]


def free(table, rows, first, end, refs, ring, head, tail, lacked):
    """Row by row; refs and ring are updated -> state."""
    for r, f, e in zip(rows, first, end):
        for j in range(f, e):
            if table[r][j] >= 0:
                refs[table[r][j]] -= 1
    gone = [b for b, n in enumerate(refs) if n < 0]
    for i, b in enumerate(gone):
        refs[b] = 0
        ring[(tail + i) % len(ring)] = b
    return [head, tail + len(gone), lacked]
