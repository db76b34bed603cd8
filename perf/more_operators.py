"""Measured cases of what a serving and training step needs around attention: rotary positions,
attention with a sliding window and sinks, attention of requests that share a prefix, and
forked and freed pages of the 4-bit key/value cache.

A cache holds keys and values of 128 channels a head in pages: payload u8
[blocks][heads][page][64], two E2M1 codes a byte (the even channel in the low nibble), and
block scales u8 [blocks][heads][page][4 or 8]:
  format 0 (MXFP4)  1x32 blocks, E8M0 byte X + 127, X = floor(log2 amax) - 2 in [-23, 13]
  format 1 (NVFP4)  1x16 blocks, E4M3 scale E4M3(amax / (6 st)) under an fp32 scale st of the
                    whole K or V cache
A slot is block * page + row; -1 marks a token that is not in the cache.

Rotary: channels i and i + rot / 2 (half layout) or 2 i and 2 i + 1 (interleaved) of the first rot
channels turn by the angle position * freq[i], times a gain; the others stay.
"""
import math
import random
from fractions import Fraction

import numpy as np
import torch

own = False

D = 128
DEV = "cuda"
MAX_BYTES = 6.0e8        # of cache that an attention case reads at most
MAX_SCORES = 1.5e9       # padded scores of an attention case at most
MAX_ELEMENTS = 1.7e8     # of a rotated tensor at most
MAX_ENTRIES = 4.0e5      # table entries of a fork case at most
TWO_PI = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494459")


# ------------------------------------------------------------------------------ cases
def listed():
    attn = dict(causal=True, kv_min=1)
    return [
        # one decoding step: q and k of 64 requests turned, k and v stored
        dict(name="rope_step", op="append", fmt=0, tokens=64, hq=32, heads=8, page=16, pad=3, far=30000, rot=128, inter=False, base=10000.0, factor=1.0),
        # an odd chunk of prompts far into a long context: half of the head turned, scaled frequencies
        dict(name="rope_odd", op="append", fmt=1, tokens=1531, hq=20, heads=5, page=32, pad=0, far=900000, rot=64, inter=True, base=10000.0, factor=32.0),
        # the tokens of a batch of prompts
        dict(name="rope_prompts", op="append", fmt=0, tokens=16384, hq=32, heads=8, page=64, pad=100, far=0, rot=128, inter=False, base=500000.0, factor=8.0),
        # q and k of the training benchmark's dense batch, next to each other in a fused projection
        dict(name="rope_train", op="rope", back=False, seqs=2, longest=8192, ragged=False, heads=32, extra=16, rot=128, inter=False, base=10000.0, factor=1.0),
        # gradients of a jagged batch of 64 sequences turned back
        dict(name="rope_grad", op="rope", back=True, seqs=64, longest=2048, ragged=True, heads=16, extra=0, rot=96, inter=True, base=10000.0, factor=1.0),
        # the least call: one request, one token, a window inside a longer context
        dict(attn, name="window_one", op="window", fmt=0, requests=1, q_max=1, kv_max=4099, heads=2, group=8, page=16, mix=1, window=500, sinks=4),
        # a decoding batch of long ragged contexts
        dict(attn, name="window_batch", op="window", fmt=0, requests=16, q_max=1, kv_max=32768, heads=8, group=4, page=16, mix=2, window=4096, sinks=4),
        # prompt chunks over earlier context
        dict(attn, name="window_prompt", op="window", fmt=1, requests=2, q_max=2048, kv_max=8192, heads=8, group=4, page=64, mix=3, window=1024, sinks=64, kv_min=4096),
        # a decoding batch behind one long system prompt
        dict(name="shared_batch", op="shared", fmt=0, groups=1, members=64, q_max=1, prefix=8192, tail=1024, heads=8, group=4, page=64, mix=4),
        # drafted tokens of a few small groups, prefixes of many lengths
        dict(name="shared_groups", op="shared", fmt=1, groups=6, members=5, q_max=5, prefix=3000, tail=300, heads=5, group=3, page=16, mix=5),
        # four continuations of one request, then dropped
        dict(name="pages_few", op="pages", fmt=0, sources=1, forks=4, longest=1000, heads=8, page=16, spare=40, done=1, mix=6),
        # parallel sampling over a server's long contexts
        dict(name="pages_many", op="pages", fmt=0, sources=16, forks=256, longest=20000, heads=8, page=16, spare=200, done=5, mix=7),
    ]


def _spread(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_rotation(rng):
    return dict(rot=rng.choice([16, 32, 64, 96, 112, 128, 128]), inter=rng.random() < 0.5, base=rng.choice([10000.0, 500000.0, 1.0e6]), factor=rng.choice([1.0, 1.0, 4.0, 32.0]))


def draw(rng):
    op = rng.choice(["append", "rope", "window", "window", "shared", "shared", "pages"])
    page = rng.choice([16, 32, 64, 128])
    fmt = rng.randint(0, 1)
    mix = rng.randint(0, 10**6)
    if op == "append":
        heads = rng.choice([1, 2, 3, 4, 5, 8, 16])
        hq = heads * rng.choice([1, 2, 3, 4, 5, 8])
        tokens = _spread(rng, 1, min(16384, int(MAX_ELEMENTS / 2 / D / max(8, hq + heads))))
        return dict(op=op, fmt=fmt, tokens=tokens, hq=hq, heads=heads, page=page, pad=rng.randint(0, tokens // 8), far=rng.choice([0, 4000, 1000000]), **_draw_rotation(rng))
    if op == "rope":
        heads = rng.choice([1, 2, 3, 4, 5, 8, 16, 20, 32, 40])
        seqs = _spread(rng, 1, 64)
        longest = _spread(rng, 1, 32768)
        while longest > 1 and seqs * longest * heads * D > 0.4 * MAX_ELEMENTS:
            longest //= 2
        return dict(op=op, back=rng.random() < 0.5, seqs=seqs, longest=longest, ragged=rng.random() < 0.6, heads=heads, extra=rng.choice([0, 0, 2, 7]), **_draw_rotation(rng))
    heads = rng.choice([1, 2, 4, 5, 8, 16])
    if op == "pages":
        forks = _spread(rng, 1, 256)
        sources = rng.randint(1, min(forks, 32))
        longest = _spread(rng, 1, 32768)
        while longest > 1 and (forks + sources) * longest / page > MAX_ENTRIES or sources * longest * heads * 144 > MAX_BYTES:
            longest //= 2
        return dict(op=op, fmt=fmt, sources=sources, forks=forks, longest=longest, heads=heads, page=page, spare=rng.randint(0, 2 * forks), done=rng.randint(0, sources), mix=mix)
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
    kind = rng.choice(["decode", "decode", "verify", "prompt"])
    if op == "shared":
        q_max = 1 if kind == "decode" else _spread(rng, 2, 8) if kind == "verify" else _spread(rng, 16, 200)
        groups, members = _spread(rng, 1, 12), _spread(rng, 1, 64)
        prefix, tail = _spread(rng, 1, 16384), _spread(rng, q_max, max(q_max, 2048))
        while groups * members * (prefix + tail) * heads * max(144, 2 * group * q_max) > MAX_BYTES:
            groups, members, prefix, tail = max(1, groups - 1), max(1, members * 2 // 3), max(1, prefix * 3 // 4), max(q_max, tail * 3 // 4)
        return dict(op=op, fmt=fmt, groups=groups, members=members, q_max=q_max, prefix=prefix, tail=tail, heads=heads, group=group, page=page, mix=mix)
    q_max = 1 if kind == "decode" else _spread(rng, 2, 8) if kind == "verify" else _spread(rng, 16, 2048)
    kv_max = _spread(rng, max(q_max, 64), 131072 if kind == "decode" else 32768 if kind == "verify" else 8192)
    n = _spread(rng, 1, 64)
    while n > 1 and (n * kv_max * heads * 144 > MAX_BYTES or n * kv_max * heads * group * q_max > 0.5 * MAX_SCORES):
        n //= 2
    if kv_max * heads * group * q_max > 0.5 * MAX_SCORES:
        kv_max = max(q_max, int(0.5 * MAX_SCORES / (heads * group * q_max)))
    return dict(op=op, fmt=fmt, requests=n, q_max=q_max, kv_max=kv_max, kv_min=1, heads=heads, group=group, page=page, causal=True, mix=mix,
                window=_spread(rng, 1, 8192), sinks=rng.choice([0, 1, 4, 4, 16, 64, 200]))


def _lengths(case):
    """(new tokens, keys, prefix) of each request of an attention case; the keys include the new tokens."""
    rng = random.Random(case["mix"])
    q, kv, pre = [], [], []
    if case["op"] == "shared":
        for g in range(case["groups"]):
            p = case["prefix"] if g == 0 else rng.randint(0, case["prefix"])
            p -= p % case["page"]
            for m in range(case["members"]):
                n = case["q_max"] if m == 0 else rng.randint(max(1, case["q_max"] // 2), case["q_max"])
                q.append(n)
                kv.append(p + rng.randint(n, max(n, case["tail"])))
                pre.append(p)
        return q, kv, pre
    for r in range(case["requests"]):
        n = case["q_max"] if r == 0 else rng.randint(max(1, case["q_max"] // 2), case["q_max"])
        lo = max(n, case["kv_min"])
        q.append(n)
        kv.append(max(lo, case["kv_max"]) if r == 0 else rng.randint(lo, max(lo, case["kv_max"])))
        pre.append(0)
    return q, kv, pre


def _fork_lengths(case):
    """(tokens of each source, source of each fork, tokens of each fork, spare blocks)"""
    rng = random.Random(case["mix"])
    ctx = [case["longest"] if s == 0 else rng.randint(0, case["longest"]) for s in range(case["sources"])]
    src = [rng.randrange(case["sources"]) for _ in range(case["forks"])]
    return ctx, src, [ctx[s] if rng.random() < 0.7 else rng.randint(0, ctx[s]) for s in src]


def _sequence_lengths(case):
    rng = random.Random(1000 * case["seqs"] + case["longest"])
    return [rng.randint(max(1, case["longest"] // 32), case["longest"]) if case["ragged"] else case["longest"] for _ in range(case["seqs"])]


def _freqs(case):
    """Radians a position of each pair: base^(-2 i / rot), and for a context `factor` times the usual one the slow half of the pairs slowed down by it."""
    half = case["rot"] // 2
    f = [case["base"] ** (-i / half) for i in range(half)]
    keep = [min(1.0, max(0.0, 2.0 - 4.0 * i / half)) for i in range(half)]
    return [x * (k + (1.0 - k) / case["factor"]) for x, k in zip(f, keep)]


def _gain(case):
    return 0.1 * math.log(case["factor"]) + 1.0


# ----------------------------------------------------------------------------- inputs
def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32)


def _random_cache(fmt, blocks, heads, page, gen):
    """A cache of normal keys (some channels larger) and values, every row filled."""
    sf = 4 if fmt == 0 else 8
    cache = dict(fmt=fmt, page=page)
    for name, scale in (("k", 24.0 / 2688), ("v", 24.0 / 2688)):
        st = torch.tensor([scale], dtype=torch.float32, device=DEV)
        cache[name] = torch.empty((blocks, heads, page, 64), dtype=torch.uint8, device=DEV)
        cache[name + "_sf"] = torch.empty((blocks, heads, page, sf), dtype=torch.uint8, device=DEV)
        cache[name + "_scale"] = st if fmt == 1 else None
        step = max(1, (1 << 26) // (heads * page * D))
        for b in range(0, blocks, step):
            x = _normal(gen, min(step, blocks - b), heads, page, D)
            if name == "k":
                x[..., 5::29] *= 3.0
            c, s = _encode(x.bfloat16(), fmt, st)
            cache[name][b: b + step], cache[name + "_sf"][b: b + step] = c, s
    return cache


def _rotation(case):
    """The plan of a rotation: radians a position in 64 bits, and the same as 2^-64ths of a turn, wrapped around."""
    f = _freqs(case)
    turns = [round(Fraction(x) / TWO_PI * 2**64) % 2**64 for x in f]
    return dict(freqs=torch.tensor(f, dtype=torch.float64, device=DEV),
                turns=torch.tensor([t - 2**64 if t >= 2**63 else t for t in turns], dtype=torch.int64, device=DEV), gain=_gain(case))


def _tables(pages, shared, order):
    """Block tables int32 [requests][width]: row r has pages[r] blocks of `order`, the first shared[r][1] of them those of row shared[r][0]."""
    width = max(1, max(pages))
    table = np.full((len(pages), width), -1, np.int32)
    order, at = order.cpu().numpy(), 0
    for r, (n, (first, p)) in enumerate(zip(pages, shared)):
        p = 0 if first == r else min(p, n)
        table[r, :p] = table[first, :p]
        table[r, p:n] = order[at: at + n - p]
        at += n - p
    return torch.from_numpy(table).to(DEV), at


def _inputs(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    i32 = dict(dtype=torch.int32, device=DEV)
    if case["op"] == "rope":
        lens = _sequence_lengths(case)
        pos = torch.cat([torch.arange(n, **i32) for n in lens])
        x = _normal(gen, pos.numel(), case["heads"] + case["extra"], D).bfloat16()
        return dict(_rotation(case), x=x[:, : case["heads"]], positions=pos)
    page = case["page"]
    if case["op"] == "append":
        n, h, hq = case["tokens"] - case["pad"], case["heads"], case["hq"]
        blocks = -(-n // page) + 3
        order = torch.randperm(blocks - 1, generator=gen, device=DEV)
        at = (order[:, None] * page + torch.arange(page, device=DEV)).reshape(-1)[:n]
        slots = torch.cat([at, at.new_full((case["pad"],), -1)])
        rng = random.Random(seed)
        pos, t = [], 0
        while t < n:  # runs of tokens, each somewhere in its request
            run = min(n - t, 1 if case["tokens"] <= 256 else rng.randint(1, 4096))
            pos.append(torch.arange(run, **i32) + rng.randint(0, case["far"]))
            t += run
        pos = torch.cat(pos + [torch.full((case["pad"],), -1, **i32)])
        x = _normal(gen, case["tokens"], hq + 2 * h, D)
        x[:, :, ::17] *= 6.0
        return dict(_rotation(case), cache=_random_cache(case["fmt"], blocks, h, page, gen), qkv=x.reshape(case["tokens"], -1).bfloat16(), slots=slots, positions=pos,
                    turned=torch.zeros((case["tokens"], hq, D), dtype=torch.bfloat16, device=DEV))
    if case["op"] == "pages":
        ctx, src, lens = _fork_lengths(case)
        have = [-(-c // page) for c in ctx]
        blocks = sum(have) + case["spare"] + 1
        order = torch.randperm(blocks, generator=gen, device=DEV).to(torch.int32)
        rows, _ = _tables(have, [(r, 0) for r in range(len(have))], order)
        table = torch.full((case["sources"] + case["forks"], rows.shape[1]), -1, **i32)
        table[: case["sources"]] = rows
        head = 3 * blocks - case["spare"] // 2  # the ring of free blocks, at some place of its life
        ring = torch.full((blocks,), -7, **i32)
        ring[(head + torch.arange(case["spare"], device=DEV)) % blocks] = order[sum(have): sum(have) + case["spare"]]
        dst = list(range(case["sources"], case["sources"] + case["forks"]))
        free = dst + list(range(case["done"]))
        ends = [-(-n // page) for n in lens] + have[: case["done"]]
        return dict(cache=_random_cache(case["fmt"], blocks, case["heads"], page, gen), table=table, refs=torch.zeros(blocks, **i32), ring=ring,
                    state=torch.tensor([head, head + case["spare"], 0], dtype=torch.int64, device=DEV), unused=order[-1],
                    src=torch.tensor(src, **i32), dst=torch.tensor(dst, **i32), lens=torch.tensor(lens, **i32),
                    free=torch.tensor(free, **i32), first=torch.zeros(len(free), **i32), end=torch.tensor(ends, **i32))
    q, kv, pre = _lengths(case)
    h, g = case["heads"], case["group"]
    m = case["members"] if case["op"] == "shared" else 1
    pages = [-(-k // page) for k in kv]
    blocks = sum(pages) + 2
    order = torch.randperm(blocks, generator=gen, device=DEV).to(torch.int32)
    table, used = _tables(pages, [(r // m * m, p // page) for r, p in enumerate(pre)], order)
    cu = [0]
    for n in q:
        cu.append(cu[-1] + n)
    fused = _normal(gen, cu[-1], h * (g + 2) * D).bfloat16()
    s = dict(cache=_random_cache(case["fmt"], blocks, h, page, gen), table=table, q=fused[:, : h * g * D].unflatten(1, (h * g, D)),
             cu_q=torch.tensor(cu, **i32), kv_lens=torch.tensor(kv, **i32))
    if case["op"] == "shared":
        starts = list(range(0, len(q) + 1, m))
        s.update(starts=torch.tensor(starts, **i32), prefix_lens=torch.tensor(pre[::m], **i32), most=max(cu[b] - cu[a] for a, b in zip(starts, starts[1:])))
    return s


def prepare(case, seed):
    return dict(case, **_inputs(case, seed))


# ------------------------------------------------------------------------- plain forms
def _round_e2m1(y):
    """The E2M1 value nearest to y >= 0, ties to the even code, at most 6."""
    step = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0))
    return (torch.round(y / step) * step).clamp(max=6.0)


def _encode(x, fmt, st):
    """bf16 [..., 128] -> (packed codes u8 [..., 64], block scales u8 [..., 4 or 8])."""
    x = x.float().unflatten(-1, (4, 32) if fmt == 0 else (8, 16))
    amax = x.abs().amax(-1, keepdim=True)
    if fmt == 0:
        e = torch.where(amax > 0, torch.frexp(amax).exponent - 3, -23).clamp(-23, 13)
        sf = (e + 127).to(torch.uint8)
        y = x * ((127 - e) << 23).view(torch.float32)
    else:
        e4 = (amax / (6.0 * st)).clamp(max=448.0).to(torch.float8_e4m3fn)
        sf = e4.view(torch.uint8)
        unit = e4.float() * st
        y = torch.where(unit > 0, x / unit, 0.0)
    v = _round_e2m1(y.abs())
    code = torch.where(v < 2, 2 * v, torch.where(v < 4, v + 2, v / 2 + 4)).to(torch.uint8)
    code = (code + torch.where(y < 0, 8, 0).to(torch.uint8)).flatten(-2)
    return code[..., 0::2] + code[..., 1::2] * 16, sf.squeeze(-1)


def _decode(codes, sf, fmt, st):
    """Packed codes and block scales -> fp32 [..., 128]."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    m = (c & 7).float()
    v = torch.where(m < 4, m * 0.5, torch.where(m < 6, m - 2.0, 2.0 * m - 8.0))
    v = torch.where(c >= 8, -v, v)
    s = (sf.to(torch.int32) << 23).view(torch.float32) if fmt == 0 else sf.view(torch.float8_e4m3fn).float()
    v = (v.unflatten(-1, (sf.shape[-1], -1)) * s[..., None]).flatten(-2)
    return v if fmt == 0 else v * st


def _turn(x, s, back):
    """x bf16 [tokens, heads, 128] turned by its tokens' positions, or back; angles in 64 bits."""
    rot, half = s["rot"], s["rot"] // 2
    angle = s["positions"].double()[:, None] * s["freqs"]
    c, w = (torch.cos(angle) * s["gain"]).float()[:, None], (torch.sin(angle) * s["gain"]).float()[:, None]
    w = -w if back else w
    x = x.float()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if s["inter"] else (x[..., :half], x[..., half:rot])
    turned = (a * c - b * w, b * c + a * w)
    turned = torch.stack(turned, -1).flatten(-2) if s["inter"] else torch.cat(turned, -1)
    return torch.cat([turned, x[..., rot:]], -1).bfloat16()


def _plain_rope(s):
    return dict(y=_turn(s["x"], s, s["back"]))


def _split(s):
    h, hq = s["heads"], s["hq"]
    return (x.unflatten(1, (-1, D)) for x in s["qkv"].split([hq * D, h * D, h * D], 1))


def _plain_load(s, slots):
    cache, fmt, page = s["cache"], s["fmt"], s["page"]
    at = slots.clamp(min=0)
    block, row = at // page, at % page
    gone = (slots < 0)[:, None, None]
    k = _decode(cache["k"][block, :, row], cache["k_sf"][block, :, row], fmt, cache["k_scale"])
    v = _decode(cache["v"][block, :, row], cache["v_sf"][block, :, row], fmt, cache["v_scale"])
    return dict(k=torch.where(gone, 0.0, k).bfloat16(), v=torch.where(gone, 0.0, v).bfloat16())


def _plain_append(s):
    cache, fmt, page = s["cache"], s["fmt"], s["page"]
    q, k, v = _split(s)
    live = s["positions"] >= 0
    s["turned"].copy_(torch.where(live[:, None, None], _turn(q, s, False), s["turned"]))
    spare = cache["k"].shape[0] * page - 1
    at = torch.where(s["slots"] < 0, spare, s["slots"])
    (ck, sk), (cv, sv) = _encode(_turn(k, s, False), fmt, cache["k_scale"]), _encode(v, fmt, cache["v_scale"])
    block, row = at // page, at % page
    cache["k"][block, :, row] = ck
    cache["v"][block, :, row] = cv
    cache["k_sf"][block, :, row] = sk
    cache["v_sf"][block, :, row] = sv
    return dict(_plain_load(s, s["slots"]), q=s["turned"])


def _plain_attn(s):
    cache, fmt, page = s["cache"], s["fmt"], s["page"]
    h, g, most = s["heads"], s["group"], s["q_max"]
    table, cu, kv = s["table"].clamp(min=0), s["cu_q"].long(), s["kv_lens"].long()
    n, keys = table.shape[0], table.shape[1] * page
    k = _decode(cache["k"][table], cache["k_sf"][table], fmt, cache["k_scale"]).transpose(1, 2).reshape(n, h, keys, D)
    v = _decode(cache["v"][table], cache["v_sf"][table], fmt, cache["v_scale"]).transpose(1, 2).reshape(n, h, keys, D)
    i = torch.arange(most, device=table.device)
    ql = cu[1:] - cu[:-1]
    q = s["q"][(cu[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)].float()
    q = q.reshape(n, most, h, g, D).permute(0, 2, 1, 3, 4).reshape(n, h, most * g, D)
    score = (q @ k.transpose(-1, -2)).view(n, h, most, g, keys) * (D ** -0.5)
    at = ((kv - ql)[:, None] + i).clamp(max=kv[:, None] - 1)[:, :, None]  # a query's own position
    j = torch.arange(keys, device=table.device)
    seen = j <= at
    if s["op"] == "window":
        seen = seen & ((j > at - s["window"]) | (j < s["sinks"]))
    score = torch.where(seen[:, None, :, None, :], score, -torch.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -torch.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    lse = (top + torch.log(total)).squeeze(-1)
    o = (p.view(n, h, most * g, keys) @ v).view(n, h, most, g, D) / torch.where(total > 0, total, 1.0)
    t = torch.arange(s["q"].shape[0], device=table.device)
    r = (torch.searchsorted(cu, t, right=True) - 1).clamp(max=n - 1)
    at = t - cu[r]
    return dict(o=o[r, :, at].reshape(-1, h * g, D).bfloat16(), lse=lse[r, :, at].reshape(-1, h * g).t().contiguous())


def _copied_rows(s, to):
    """Slots of the rows of the copied blocks."""
    page = s["page"]
    return torch.where(to[:, None] < 0, -1, to.long()[:, None] * page + torch.arange(page, device=to.device)).reshape(-1)


def _plain_pages(s):
    page, table, refs, ring, cache = s["page"], s["table"], s["refs"], s["ring"], s["cache"]
    src, dst, lens = s["src"].long(), s["dst"].long(), s["lens"].long()
    head, tail = s["state"][0], s["state"][1]
    whole, part = lens // page, lens % page > 0
    j = torch.arange(table.shape[1], device=table.device)
    # whole pages are shared; the last one, where it is not full, goes into a block of its own
    rows = table[src]
    shared = j < whole[:, None]
    refs += torch.bincount(torch.where(shared, rows + 1, 0).reshape(-1), minlength=refs.numel() + 1)[1:].int()
    rank = part.long().cumsum(0) - 1
    served = part & (rank < tail - head)
    fresh = ring[(head + rank.clamp(min=0)) % ring.numel()]
    old = rows.gather(1, whole.clamp(max=table.shape[1] - 1)[:, None])[:, 0]
    at, to = torch.where(served, old, -1), torch.where(served, fresh, -1)
    mine = torch.where(shared, rows, table[dst])
    table[dst] = torch.where((j == whole[:, None]) & part[:, None], torch.where(served, fresh, -1)[:, None], mine)
    kept = torch.where(part & ~served, whole * page, lens)
    taken = torch.minimum(part.sum(), (tail - head).clamp(min=0))
    a, b = (torch.where(x < 0, s["unused"], x).long() for x in (at, to))
    cache["k"][b] = cache["k"][a]
    cache["v"][b] = cache["v"][a]
    cache["k_sf"][b] = cache["k_sf"][a]
    cache["v_sf"][b] = cache["v_sf"][a]
    # pages given up: one owner fewer each; those of none go to the ring, the lowest first
    up = (j >= s["first"][:, None]) & (j < s["end"][:, None])
    given = torch.where(up, table[s["free"].long()] + 1, 0)
    refs -= torch.bincount(given.reshape(-1), minlength=refs.numel() + 1)[1:].int()
    gone = refs < 0
    count = gone.sum()
    place = torch.where(gone, (tail + gone.long().cumsum(0) - 1) % ring.numel(), ring.numel())
    block = torch.arange(refs.numel(), dtype=torch.int32, device=table.device)
    ring.copy_(torch.cat([ring, ring[:1]]).index_copy_(0, place, block)[: ring.numel()])
    refs.clamp_(min=0)
    state = torch.stack([head + taken, tail + count, part.sum() - taken])
    return dict(_plain_load(s, _copied_rows(s, to)), table=table, refs=refs, ring=ring, at=at, to=to, kept=kept.int(), state=state)


def run(s):
    if own:
        return _own(s)
    return {"rope": _plain_rope, "append": _plain_append, "window": _plain_attn, "shared": _plain_attn, "pages": _plain_pages}[s["op"]](s)


def _own(s):
    import mxfp8_block_scaled_fa_gb300 as mx
    if s["op"] == "rope":
        rp = mx.Rope(s["turns"], s["inter"], s["gain"])
        return dict(y=(mx.rope_bwd if s["back"] else mx.rope)(s["x"], rp, s["positions"]))
    c = s["cache"]
    cache = mx.KvCache(c["k"], c["v"], c["k_sf"], c["v_sf"], c["fmt"], c["k_scale"], c["v_scale"])
    if s["op"] == "append":
        rp = mx.Rope(s["turns"], s["inter"], s["gain"])
        q, k, v = _split(s)
        mx.kv_append_rope(cache, q, k, v, rp, s["positions"], s["slots"], out=s["turned"])
        k, v = mx.kv_load(cache, s["slots"])
        return dict(q=s["turned"], k=k, v=v)
    if s["op"] == "window":
        o, lse = mx.kv_attention(s["q"], cache, s["cu_q"], s["kv_lens"], s["table"], s["q_max"], D ** -0.5, window=s["window"], sinks=s["sinks"])
        return dict(o=o, lse=lse)
    if s["op"] == "shared":
        o, lse = mx.kv_attention_shared(s["q"], cache, s["cu_q"], s["kv_lens"], s["table"], s["starts"], s["prefix_lens"], s["q_max"], s["most"], D ** -0.5)
        return dict(o=o, lse=lse)
    f = mx.kv_fork(s["table"], s["src"], s["dst"], s["lens"], s["refs"], s["ring"], s["state"], s["page"])
    mx.kv_copy_blocks(cache, f.from_blocks, f.to_blocks)
    k, v = mx.kv_load(cache, _copied_rows(s, f.to_blocks))
    state = mx.kv_free(s["table"], s["free"], s["first"], s["end"], s["refs"], s["ring"], f.ring_state)
    return dict(k=k, v=v, table=s["table"], refs=s["refs"], ring=s["ring"], at=f.from_blocks, to=f.to_blocks, kept=f.lens, state=state)


# ---------------------------------------------------------------------- work and values
def work(case):
    if case["op"] == "rope":
        n = sum(_sequence_lengths(case))
        return dict(bytes=n * (case["heads"] * D * 4 + 4), flops=n * case["heads"] * case["rot"] * 3)
    row = 64 + (4 if case["fmt"] == 0 else 8)
    if case["op"] == "append":
        n, h = case["tokens"] - case["pad"], case["heads"]
        # q in and out, k and v in, codes and scales out; then read back for comparison
        return dict(bytes=n * (case["hq"] * D * 4 + 2 * h * (2 * D + row) + 12) + n * 2 * h * row + case["tokens"] * (2 * h * 2 * D + 8), flops=n * (case["hq"] + h) * case["rot"] * 3)
    if case["op"] == "pages":
        ctx, src, lens = _fork_lengths(case)
        page = case["page"]
        copied = min(case["spare"], sum(n % page > 0 for n in lens))
        shared = sum(n // page for n in lens)
        given = sum(-(-n // page) for n in lens) + sum(-(-n // page) for n in ctx[: case["done"]])
        blocks = sum(-(-n // page) for n in ctx) + case["spare"] + 1
        # an entry shared: read, written, its count read and written; an entry given up: read, its count read and written;
        # counts looked at; blocks copied, and read back for comparison
        return dict(bytes=16 * shared + 12 * given + 4 * blocks + copied * case["heads"] * page * 2 * (3 * row + 2 * D), flops=0)
    q, kv, pre = _lengths(case)
    h, g, page = case["heads"], case["group"], case["page"]
    if case["op"] == "shared":
        m = case["members"]
        cells = sum(n * (k - n) + n * (n + 1) // 2 for n, k in zip(q, kv))
        keys = sum(k - p for k, p in zip(kv, pre)) + sum(pre[::m])
    else:
        w, sk = case["window"], case["sinks"]
        cells = keys = 0
        for n, k in zip(q, kv):
            for p in range(k - n, k):
                lo = max(0, p - w + 1)
                cells += p + 1 - lo + min(sk, lo)
            lo = max(0, k - n - w + 1)
            keys += k - lo + min(sk, lo)
    size = 2 * keys * h * row + 4 * -(-keys // page) + sum(q) * h * g * (4 * D + 4) + 8 * len(q)
    return dict(bytes=size, flops=4 * D * h * g * cells)


_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _values(codes, sf, fmt, st):
    """Packed codes and scales -> float64 by tables."""
    tab = torch.tensor(_E2M1 + [-x for x in _E2M1], dtype=torch.float64, device=codes.device)
    both = tab[torch.stack([(codes % 16).long(), (codes // 16).long()], -1)].flatten(-2)
    if fmt == 0:
        scale = torch.tensor([2.0 ** (b - 127) for b in range(255)] + [math.nan], dtype=torch.float64, device=codes.device)[sf.long()]
    else:
        e4 = [(b & 7) * 2.0 ** -9 if b & 120 == 0 else math.nan if b & 127 == 127 else (8 + (b & 7)) * 2.0 ** ((b >> 3 & 15) - 10) for b in range(256)]
        scale = torch.tensor([-x if b & 128 else x for b, x in enumerate(e4)], dtype=torch.float64, device=codes.device)[sf.long()] * st.double()
    return both * scale.repeat_interleave(D // sf.shape[-1], -1)


def _nearest(y, grid, most):
    """y >= 0 (float64) rounded to the ascending grid, ties to the even index, at most grid[most]."""
    i = np.clip(np.searchsorted(grid, y, side="right") - 1, 0, len(grid) - 2)
    low, high = y - grid[i], grid[i + 1] - y
    up = (high < low) | ((high == low) & (i % 2 == 1))
    return grid[np.minimum(i + up, most)]


def _stored(x, fmt, st):
    """What the cache holds for bf16 x[..., 128], in float64: the definition's fp32 steps rounded one by one."""
    x = x.double().cpu().numpy()
    st = np.float64(st.item()) if st is not None else 1.0
    codes = np.array(_E2M1 + [8.0])
    if fmt == 0:
        b = x.reshape(*x.shape[:-1], 4, 32)
        amax = np.abs(b).max(-1, keepdims=True)
        unit = 2.0 ** np.clip(np.floor(np.log2(np.maximum(amax, 1e-300))) - 2, -23, 13)
        val = np.sign(b) * _nearest(np.abs(b) / unit, codes, 7) * unit
    else:
        e4 = np.array([(c & 7) * 2.0 ** -9 if c < 8 else (8 + (c & 7)) * 2.0 ** ((c >> 3) - 10) for c in range(128)])
        f32 = lambda a: np.asarray(a, np.float32).astype(np.float64)  # noqa: E731
        b = x.reshape(*x.shape[:-1], 8, 16)
        amax = np.abs(b).max(-1, keepdims=True)
        sb = _nearest(f32(amax / f32(6.0 * st)), e4, 126)
        unit = f32(sb * st)
        val = np.sign(b) * np.where(unit > 0, _nearest(f32(np.abs(b) / np.where(unit > 0, unit, 1.0)), codes, 7), 0.0) * (sb * st)
    return torch.from_numpy(val.reshape(x.shape))


def _rotated(x, case, positions, back):
    """The rotation as a product of complex numbers, in 64 bits."""
    rot = case["rot"]
    angle = positions.double().cpu().numpy()[:, None] * np.array(_freqs(case))
    z = torch.from_numpy(_gain(case) * np.exp((-1j if back else 1j) * angle)).to(x.device)[:, None]
    x = x.double()
    if case["inter"]:
        y = torch.view_as_complex(x[..., :rot].unflatten(-1, (rot // 2, 2)).contiguous())
        y = torch.view_as_real(y * z).flatten(-2)
    else:
        y = torch.complex(x[..., : rot // 2].contiguous(), x[..., rot // 2: rot].contiguous()) * z
        y = torch.cat([y.real, y.imag], -1)
    return torch.cat([y, x[..., rot:]], -1)


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "rope":
        return dict(y=_rotated(s["x"], case, s["positions"], case["back"]))
    c, page, fmt = s["cache"], case["page"], case["fmt"]
    h = case["heads"]
    if case["op"] == "append":
        if case["tokens"] * h > 40000:
            return None
        q, k, v = _split(dict(case, **s))
        y = _rotated(q, case, s["positions"], False)
        y[s["positions"] < 0] = 0.0
        k = _stored(_rotated(k, case, s["positions"], False).float().bfloat16(), fmt, c["k_scale"]).to(DEV)
        v = _stored(v, fmt, c["v_scale"]).to(DEV)
        k[s["slots"] < 0] = 0.0
        v[s["slots"] < 0] = 0.0
        return dict(q=y, k=k, v=v)
    if case["op"] == "pages":
        ctx, src, lens = _fork_lengths(case)
        table, ring, n = s["table"].tolist(), s["ring"].tolist(), 0
        out = dict(k=[], v=[])
        for a, m in zip(src, lens):
            took = m % page > 0 and n < case["spare"]
            n += m % page > 0
            for x in "kv":
                b = table[a][m // page] if took else 0
                val = _values(c[x][b], c[x + "_sf"][b], fmt, c[x + "_scale"]).transpose(0, 1)
                out[x].append(val if took else torch.zeros_like(val))
        return dict(k=torch.cat(out["k"]), v=torch.cat(out["v"]), table=None, refs=None, ring=None, at=None, to=None, kept=None, state=None)
    q, kv, _ = _lengths(case)
    if sum(n * k for n, k in zip(q, kv)) * h * case["group"] > 1.2e9:
        return None
    g = case["group"]
    o = torch.zeros(sum(q), h * g, D, dtype=torch.float64, device=DEV)
    lse = torch.full((h * g, sum(q)), -math.inf, dtype=torch.float64, device=DEV)
    t = 0
    for r, (n, k) in enumerate(zip(q, kv)):
        pages = s["table"][r, : -(-k // page)].long()
        hidden = torch.ones(n, k, dtype=torch.bool, device=DEV).triu(k - n + 1)
        if case["op"] == "window":
            outside = torch.ones(n, k, dtype=torch.bool, device=DEV).tril(k - n - case["window"])
            outside[:, : case["sinks"]] = False
            hidden |= outside
        for a in range(h):
            key, val = (_values(c[x][pages, a].reshape(-1, 64)[:k], c[x + "_sf"][pages, a].flatten(0, 1)[:k], fmt, c[x + "_scale"]) for x in "kv")
            x = s["q"][t: t + n, a * g: (a + 1) * g].double().transpose(0, 1)
            score = (torch.matmul(x, key.t()) / math.sqrt(D)).masked_fill(hidden, -math.inf)
            w = torch.logsumexp(score, -1)
            o[t: t + n, a * g: (a + 1) * g] = torch.matmul(torch.exp(score - w[..., None]), val).transpose(0, 1)
            lse[a * g: (a + 1) * g, t: t + n] = w
        t += n
    return dict(o=o, lse=lse)
