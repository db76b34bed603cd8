"""Plain 64-bit forms of the 4-bit cache's operators, written from their formulas:
quantization by nearest value, attention over dequantized rows, and the step
plan as a loop over requests."""

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([(c & 7) * 2.0 ** -9 if c < 8 else (8 + (c & 7)) * 2.0 ** ((c >> 3) - 10) for c in range(127)])


def nearest(y, grid):
    """Index of the value of the ascending grid nearest to each y >= 0, ties to the even index."""
    mid = (grid[1:] + grid[:-1]) / 2
    i = np.searchsorted(mid, y, side="left")
    tie = (i < len(mid)) & (y == mid[np.minimum(i, len(mid) - 1)])
    return np.where(tie & (i % 2 == 1), i + 1, i)


def f32(a):
    with np.errstate(over="ignore"):
        return np.asarray(a, np.float32).astype(np.float64)


def quantize(x, fmt, st=1.0):
    """float64 x[..., 128] -> (codes u8 [..., 64], scale bytes u8, values float64)."""
    nb = 4 if fmt == 0 else 8
    b = x.reshape(*x.shape[:-1], nb, 128 // nb)
    bad = ~np.isfinite(b).all(-1, keepdims=True)
    b = np.where(bad, 0.0, b)
    amax = np.abs(b).max(-1, keepdims=True)
    if fmt == 0:
        e = np.where(amax > 0, np.floor(np.log2(np.maximum(amax, 1e-300))) - 2, -23)
        e = np.clip(e, -23, 13)
        sf = np.where(bad, 255, e + 127).astype(np.uint8)
        unit, div, st = 2.0 ** e, 2.0 ** e, 1.0
    else:
        i = nearest(f32(amax / f32(6.0 * st)), E4M3)
        sf = np.where(bad, 127, i).astype(np.uint8)
        unit = E4M3[i]
        div = f32(unit * st)
    y = np.where(div > 0, f32(np.abs(b) / np.where(div > 0, div, 1.0)), 0.0)
    c = nearest(y, E2M1)
    val = np.where(bad, np.nan, np.sign(b) * E2M1[c] * unit * st).reshape(x.shape)
    neg = np.signbit(b) & (div > 0)
    code = (c + 8 * neg).astype(np.uint8).reshape(x.shape)
    return code[..., 0::2] | (code[..., 1::2] << 4), sf[..., 0], val


def dequantize(codes, sf, fmt, st=1.0):
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], 128)
    v = np.where(c & 8, -1.0, 1.0) * E2M1[c & 7]
    if fmt == 0:
        s = np.where(sf == 255, np.nan, 2.0 ** (sf.astype(np.float64) - 127))
    else:
        s = np.concatenate([E4M3, [np.nan]])[sf & 127] * np.where(sf & 128, -1.0, 1.0) * st
    return v * np.repeat(s, 128 // sf.shape[-1], -1)


def attention(q, k, v, scale, causal):
    """float64 q [n, Hq, 128], k, v [kv, H, 128] -> (o, lse [n, Hq], a, s): a = sum p |v| / sum p and
    s = the largest scale sum |q_d k_d| of the row, for error bounds.  A key that a row does not see
    takes no part, whatever it holds."""
    n, Hq, _ = q.shape
    kv, H = k.shape[0], k.shape[1]
    G = Hq // H
    o, a = np.zeros((n, Hq, 128)), np.zeros((n, Hq, 128))
    lse, s = np.full((n, Hq), -np.inf), np.zeros((n, Hq))
    for h in range(H):
        kh, vh = k[:, h], v[:, h]
        hs = slice(h * G, (h + 1) * G)
        x_all = scale * np.einsum("igd,jd->igj", q[:, hs], kh)
        s_all = scale * np.einsum("igd,jd->igj", np.abs(q[:, hs]), np.abs(kh))
        for i in range(n):
            m = min(kv, kv - n + i + 1) if causal else kv
            if m <= 0:
                continue
            x = x_all[i, :, :m]
            top = x.max(-1, keepdims=True)
            with np.errstate(invalid="ignore"):
                p = np.exp(x - top)
                t = p.sum(-1, keepdims=True)
                lse[i, hs] = (top + np.log(t))[:, 0]
                o[i, hs] = p @ vh[:m] / t
                a[i, hs] = p @ np.abs(vh[:m]) / t
            s[i, hs] = s_all[i, :, :m].max(-1)
    return o, lse, a, s


def plan(ctx, new, table, ring, head, tail, page, tokens):
    """The step plan, request by request; table and ring are updated."""
    cu, kv, slots, pos, back, want, first = [0], [], [], [], [], 0, head
    n = len(ring)
    for r, (c, a) in enumerate(zip(ctx, new)):
        have = -(-c // page)
        if a < 0:
            back += [int(b) for b in table[r][:have]]
            kv.append(0)
            cu.append(cu[-1])
            continue
        grow = -(-(c + a) // page) - have
        want += grow
        fits = grow == 0 or want <= tail - head
        if fits:
            for j in range(grow):
                table[r][have + j] = ring[first % n]
                first += 1
        for p in range(c, c + a):
            pos.append(p)
            slots.append(int(table[r][p // page]) * page + p % page if fits else -1)
        cu.append(cu[-1] + a)
        kv.append(c + a if fits else c)
    for i, b in enumerate(back):
        ring[(tail + i) % n] = b
    pad = tokens - len(slots)
    return cu, kv, slots + [-1] * pad, pos + [-1] * pad, [first, tail + len(back), want - (first - head)]
