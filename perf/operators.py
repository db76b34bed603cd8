"""Measured cases of the 4-bit key/value cache: the plan of a step, the store and the load
of tokens, and the attention that reads the cache.

A cache holds keys and values of 128 channels a head in pages: payload u8
[blocks][heads][page][64], two E2M1 codes a byte (the even channel in the low nibble), and
block scales u8 [blocks][heads][page][4 or 8]:
  format 0 (MXFP4)  1x32 blocks, E8M0 byte X + 127, X = floor(log2 amax) - 2 in [-23, 13]
  format 1 (NVFP4)  1x16 blocks, E4M3 scale E4M3(amax / (6 st)) under an fp32 scale st of the
                    whole K or V cache
A slot is block * page + row; -1 marks a token that is not in the cache.
"""
import math
import random

import numpy as np
import torch

own = False

D = 128
DEV = "cuda"
MAX_BYTES = 6.0e8        # of cache that an attention case reads at most
MAX_SCORES = 1.5e9       # padded scores of an attention case at most
MAX_PAIRS = 7.0e8        # (query row, key) pairs of an attention case at most


# ------------------------------------------------------------------------------ cases
def listed():
    attn = dict(op="attn", causal=True, empties=False, kv_min=1)
    return [
        # one decoding step of a small server: every request asks for one more slot
        dict(name="plan_step", op="plan", requests=16, page=16, width=256, tokens=16, prompts=0, done=0, spare=64, mix=1),
        # a busy server's step: decoding requests, prompts of thousands of tokens, finished requests
        dict(name="plan_mixed", op="plan", requests=1024, page=16, width=2048, tokens=131072, prompts=24, done=37, spare=20000, mix=2),
        # the new tokens of one decoding step, K and V as slices of a fused projection
        dict(name="append_step", op="append", fmt=0, tokens=64, heads=8, page=16, pad=3),
        # an odd chunk of prompts in the finer format
        dict(name="append_odd", op="append", fmt=1, tokens=1531, heads=5, page=32, pad=0),
        # the tokens of a batch of prompts
        dict(name="append_prompts", op="append", fmt=0, tokens=32768, heads=8, page=64, pad=100),
        # a short prefix read back for inspection
        dict(name="load_prefix", op="load", fmt=1, tokens=777, heads=8, page=16, pad=7),
        # requests moved out of the cache
        dict(name="load_swap", op="load", fmt=0, tokens=49152, heads=8, page=64, pad=0),
        # the least call: one request, one token, a short context
        dict(attn, name="attn_one", fmt=0, requests=1, q_max=1, kv_max=201, heads=2, group=8, page=16, mix=3),
        # a decoding batch of ragged contexts, some requests idle
        dict(attn, name="attn_batch", fmt=0, requests=64, q_max=1, kv_max=8192, heads=8, group=4, page=16, mix=4, empties=True),
        # few long contexts, where the keys have to be split
        dict(attn, name="attn_long", fmt=1, requests=3, q_max=1, kv_max=130001, heads=8, group=8, page=64, mix=5),
        # drafted tokens verified a few at a time, causal among themselves
        dict(attn, name="attn_verify", fmt=0, requests=24, q_max=6, kv_max=12288, heads=8, group=8, page=128, mix=6),
        # prompt chunks over earlier context
        dict(attn, name="attn_prompt", fmt=1, requests=2, q_max=2048, kv_max=8192, heads=8, group=4, page=64, mix=7, kv_min=4096),
    ]


def _spread(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "load", "attn", "attn", "attn"])
    page = rng.choice([16, 32, 64, 128])
    if op == "plan":
        n = _spread(rng, 1, 1024)
        most = _spread(rng, 128, 32768)
        return dict(op=op, requests=n, page=page, width=-(-most // page) + 1, tokens=_spread(rng, n, 131072),
                    prompts=rng.randint(0, min(n, 24)), done=rng.randint(0, n // 4), spare=_spread(rng, 1, 20000), mix=rng.randint(0, 10**6))
    fmt = rng.randint(0, 1)
    if op in ("append", "load"):
        heads = rng.choice([1, 2, 3, 4, 5, 8, 16])
        tokens = _spread(rng, 1, 32768 * 8 // max(8, heads))
        return dict(op=op, fmt=fmt, tokens=tokens, heads=heads, page=page, pad=rng.randint(0, tokens // 8))
    heads = rng.choice([1, 2, 4, 5, 8, 16])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
    kind = rng.choice(["decode", "decode", "verify", "prompt"])
    q_max = 1 if kind == "decode" else _spread(rng, 2, 8) if kind == "verify" else _spread(rng, 16, 2048)
    kv_max = _spread(rng, max(q_max, 64), 131072 if kind == "decode" else 32768 if kind == "verify" else 8192)
    n = _spread(rng, 1, 128)
    while n > 1 and (n * kv_max * heads * 144 > MAX_BYTES or n * kv_max * heads * group * q_max > min(MAX_SCORES, MAX_PAIRS)):
        n //= 2
    if kv_max * heads * group * q_max > min(MAX_SCORES, MAX_PAIRS):
        kv_max = max(q_max, int(min(MAX_SCORES, MAX_PAIRS) / (heads * group * q_max)))
    return dict(op=op, fmt=fmt, requests=n, q_max=q_max, kv_max=kv_max, kv_min=1, heads=heads, group=group, page=page,
                causal=rng.random() < 0.8, empties=n > 2 and rng.random() < 0.5, mix=rng.randint(0, 10**6))


def _lengths(case):
    """(new tokens, keys) of each request of an attention case; the keys include the new tokens."""
    rng = random.Random(case["mix"])
    q, kv = [], []
    for r in range(case["requests"]):
        n = case["q_max"] if r == 0 else rng.randint(max(1, case["q_max"] // 2), case["q_max"])
        lo = max(n, case["kv_min"])
        k = max(lo, case["kv_max"]) if r == 0 else _spread(rng, lo, max(lo, case["kv_max"])) if case["kv_max"] < 1024 else rng.randint(lo, max(lo, case["kv_max"]))
        if case["empties"] and r % 7 == 1:
            n, k = (0, k) if r % 2 else (n, 0)
        q.append(n)
        kv.append(k)
    return q, kv


def _plan_lengths(case):
    """(tokens before the step, new tokens) of each request of a plan; -1 new tokens: the request is done."""
    rng = random.Random(case["mix"])
    n, most = case["requests"], case["width"] * case["page"]
    new = [1] * n
    order = list(range(n))
    rng.shuffle(order)
    left = case["tokens"] - n
    for r in order[: case["prompts"]]:
        c = rng.randint(0, max(0, min(left, 2 * left // max(1, case["prompts"]), most - 1)))
        new[r] += c
        left -= c
    for r in order[case["prompts"]: case["prompts"] + case["done"]]:
        new[r] = -1
    for r in order[case["prompts"] + case["done"]:]:
        if rng.random() < 0.05:
            new[r] = 0
    ctx = [rng.randint(0, max(0, most - max(0, c))) if rng.random() < 0.8 else 0 for c in new]
    return ctx, new


# ----------------------------------------------------------------------------- inputs
def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32)


def _tokens(case, gen):
    """The fused projection [tokens][(4 + 2) heads * 128] bf16 whose last parts are K and V: a few channels are larger than the others."""
    h = case["heads"]
    x = _normal(gen, case["tokens"], 6 * h, D)
    x[:, :, ::17] *= 6.0
    return x.reshape(case["tokens"], 6 * h * D).bfloat16()


def _slots(case, gen):
    """Slots of the tokens, whole pages in a random order; the last `pad` tokens have none. One block is left over."""
    page, n = case["page"], case["tokens"] - case["pad"]
    blocks = -(-n // page) + 3
    order = torch.randperm(blocks - 1, generator=gen, device=DEV)
    s = (order[:, None] * page + torch.arange(page, device=DEV)).reshape(-1)[:n]
    return torch.cat([s, s.new_full((case["pad"],), -1)]), blocks


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


def _inputs(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    i32 = dict(dtype=torch.int32, device=DEV)
    if case["op"] == "plan":
        ctx, new = _plan_lengths(case)
        page, width = case["page"], case["width"]
        have = [-(-c // page) for c in ctx]
        blocks = sum(have) + case["spare"]
        order = torch.randperm(blocks, generator=gen, device=DEV).to(torch.int32)
        at = torch.tensor([0] + have, device=DEV).cumsum(0)
        j = torch.arange(width, device=DEV)
        table = torch.where(j < (at[1:] - at[:-1])[:, None], order[(at[:-1, None] + j).clamp(max=blocks - 1)], torch.full((), -1, **i32))
        # the ring of free blocks, at some place of its life: `spare` entries from `head` on
        head = 3 * blocks - case["spare"] // 2
        ring = torch.full((blocks,), -7, **i32)
        ring[(head + torch.arange(case["spare"], device=DEV)) % blocks] = order[sum(have):]
        return dict(ctx=torch.tensor(ctx, **i32), new=torch.tensor(new, **i32), table=table.contiguous(), ring=ring,
                    state=torch.tensor([head, head + case["spare"], 0], dtype=torch.int64, device=DEV))
    if case["op"] in ("append", "load"):
        slots, blocks = _slots(case, gen)
        cache = _random_cache(case["fmt"], blocks, case["heads"], case["page"], gen)
        s = dict(slots=slots, cache=cache)
        if case["op"] == "append":
            s["qkv"] = _tokens(case, gen)
        return s
    q, kv = _lengths(case)
    page, h, g = case["page"], case["heads"], case["group"]
    pages = [-(-k // page) for k in kv]
    blocks = sum(pages) + 2
    order = torch.randperm(blocks, generator=gen, device=DEV).to(torch.int32)
    width = max(1, max(pages))
    at = torch.tensor([0] + pages, device=DEV).cumsum(0)
    j = torch.arange(width, device=DEV)
    table = torch.where(j < (at[1:] - at[:-1])[:, None], order[(at[:-1, None] + j).clamp(max=blocks - 1)], torch.full((), -1, **i32))
    cu = [0]
    for n in q:
        cu.append(cu[-1] + n)
    fused = _normal(gen, cu[-1], h * (g + 2) * D).bfloat16()
    return dict(cache=_random_cache(case["fmt"], blocks, h, page, gen), table=table.contiguous(), q=fused[:, : h * g * D].unflatten(1, (h * g, D)),
                cu_q=torch.tensor(cu, **i32), kv_lens=torch.tensor(kv, **i32))


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
    bad = ~torch.isfinite(amax)
    x = torch.where(bad, 0.0, x)
    amax = torch.where(bad, 0.0, amax)
    if fmt == 0:
        e = torch.where(amax > 0, torch.frexp(amax).exponent - 3, -23).clamp(-23, 13)
        sf = torch.where(bad, 255, e + 127).to(torch.uint8)
        y = x * ((127 - e) << 23).view(torch.float32)
    else:
        e4 = (amax / (6.0 * st)).clamp(max=448.0).to(torch.float8_e4m3fn)
        sf = torch.where(bad, 127, e4.view(torch.uint8)).to(torch.uint8)
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
    if fmt == 0:
        s = torch.where(sf == 255, torch.nan, (sf.to(torch.int32) << 23).view(torch.float32))
    else:
        s = sf.view(torch.float8_e4m3fn).float()
    v = (v.unflatten(-1, (sf.shape[-1], -1)) * s[..., None]).flatten(-2)
    return v if fmt == 0 else v * st


def _plain_plan(s):
    page, width, tokens = s["page"], s["width"], s["tokens"]
    ctx, new, table, ring = s["ctx"].long(), s["new"].long(), s["table"], s["ring"]
    head, tail = s["state"][0], s["state"][1]
    done = new < 0
    q = new.clamp(min=0)
    zero = torch.zeros(1, dtype=torch.int64, device=ctx.device)
    cu = torch.cat([zero, q.cumsum(0)])
    have = (ctx + page - 1) // page
    need = torch.where(done, 0, (ctx + q + page - 1) // page)
    grow = (need - have).clamp(min=0)
    whole = grow.cumsum(0)
    fits = (whole <= tail - head) | (grow == 0)
    kv = torch.where(done, 0, torch.where(fits, ctx + q, ctx))
    j = torch.arange(width, device=ctx.device)
    rank = (whole - grow)[:, None] + j - have[:, None]
    fresh = (j >= have[:, None]) & (j < need[:, None]) & fits[:, None]
    table = torch.where(fresh, ring[(head + rank.clamp(min=0)) % ring.numel()], table)
    back = torch.where(done, have, 0)
    entry = torch.arange(ring.numel(), device=ctx.device)
    upto = back.cumsum(0)
    who = torch.searchsorted(upto, entry, right=True).clamp(max=ctx.numel() - 1)
    block = table[who, (entry - (upto - back)[who]).clamp(0, width - 1)]
    place = (tail + entry) % ring.numel()
    ring = ring.scatter(0, place, torch.where(entry < upto[-1], block, ring[place]))
    t = torch.arange(tokens, device=ctx.device)
    r = (torch.searchsorted(cu, t, right=True) - 1).clamp(max=ctx.numel() - 1)
    live = t < cu[-1]
    pos = ctx[r] + t - cu[r]
    block = table[r, (pos // page).clamp(max=width - 1)].long()
    slots = torch.where(live & fits[r], block * page + pos % page, -1)
    taken = torch.where(whole <= tail - head, whole, 0).amax()
    state = torch.stack([head + taken, tail + upto[-1], whole[-1] - taken])
    return dict(cu_q=cu.int(), kv_lens=kv.int(), slots=slots, positions=torch.where(live, pos, -1).int(), table=table, ring=ring, state=state)


def _plain_append(s):
    cache, fmt, page, h = s["cache"], s["fmt"], s["page"], s["heads"]
    k, v = (x.unflatten(1, (h, D)) for x in s["qkv"].split([4 * h * D, h * D, h * D], 1)[1:])
    spare = cache["k"].shape[0] * page - 1
    at = torch.where(s["slots"] < 0, spare, s["slots"])
    (ck, sk), (cv, sv) = _encode(k, fmt, cache["k_scale"]), _encode(v, fmt, cache["v_scale"])
    block, row = at // page, at % page
    cache["k"][block, :, row] = ck
    cache["v"][block, :, row] = cv
    cache["k_sf"][block, :, row] = sk
    cache["v_sf"][block, :, row] = sv
    return _plain_load(s)


def _plain_load(s):
    cache, fmt, page = s["cache"], s["fmt"], s["page"]
    at = s["slots"].clamp(min=0)
    block, row = at // page, at % page
    gone = (s["slots"] < 0)[:, None, None]
    k = _decode(cache["k"][block, :, row], cache["k_sf"][block, :, row], fmt, cache["k_scale"])
    v = _decode(cache["v"][block, :, row], cache["v_sf"][block, :, row], fmt, cache["v_scale"])
    return dict(k=torch.where(gone, 0.0, k).bfloat16(), v=torch.where(gone, 0.0, v).bfloat16())


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
    last = (kv - ql)[:, None] + 1 + i if s["causal"] else kv[:, None].expand(n, most)
    j = torch.arange(keys, device=table.device)
    seen = (j < torch.minimum(last, kv[:, None])[:, :, None])[:, None, :, None, :]
    score = torch.where(seen, score, -torch.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -torch.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    lse = (top + torch.log(total)).squeeze(-1)
    o = (p.view(n, h, most * g, keys) @ v).view(n, h, most, g, D) / torch.where(total > 0, total, 1.0)
    t = torch.arange(s["q"].shape[0], device=table.device)
    r = (torch.searchsorted(cu, t, right=True) - 1).clamp(max=n - 1)
    at = t - cu[r]
    return dict(o=o[r, :, at].reshape(-1, h * g, D).bfloat16(), lse=lse[r, :, at].reshape(-1, h * g).t().contiguous())


def run(s):
    if own:
        return _own(s)
    return {"plan": _plain_plan, "append": _plain_append, "load": _plain_load, "attn": _plain_attn}[s["op"]](s)


def _own(s):
    import mxfp8_block_scaled_fa_gb300 as mx
    if s["op"] == "plan":
        step = mx.kv_plan(s["ctx"], s["new"], s["table"], s["ring"], s["state"], s["page"], s["tokens"])
        return dict(cu_q=step.cu_q, kv_lens=step.kv_lens, slots=step.slots, positions=step.positions, table=s["table"], ring=s["ring"], state=step.ring_state)
    c = s["cache"]
    cache = mx.KvCache(c["k"], c["v"], c["k_sf"], c["v_sf"], c["fmt"], c["k_scale"], c["v_scale"])
    if s["op"] == "attn":
        o, lse = mx.kv_attention(s["q"], cache, s["cu_q"], s["kv_lens"], s["table"], s["q_max"], D ** -0.5, causal=s["causal"])
        return dict(o=o, lse=lse)
    if s["op"] == "append":
        h = s["heads"]
        k, v = (x.unflatten(1, (h, D)) for x in s["qkv"].split([4 * h * D, h * D, h * D], 1)[1:])
        mx.kv_append(cache, k, v, s["slots"])
    k, v = mx.kv_load(cache, s["slots"])
    return dict(k=k, v=v)


# ---------------------------------------------------------------------- work and values
def work(case):
    if case["op"] == "plan":
        ctx, new = _plan_lengths(case)
        page = case["page"]
        moved = sum(-(-c // page) if n < 0 else -(-(c + n) // page) - -(-c // page) for c, n in zip(ctx, new))
        # lengths in, offsets and lengths out; ring entry read and table entry written, or the other way; slot, position and block of each token
        return dict(bytes=16 * case["requests"] + 8 * moved + 12 * case["tokens"] + 4 * sum(-(-max(0, n) // page) for n in new) + 48, flops=0)
    row = 64 + (4 if case["fmt"] == 0 else 8)
    if case["op"] in ("append", "load"):
        n = (case["tokens"] - case["pad"]) * case["heads"] * 2
        both = n * row + case["tokens"] * case["heads"] * 2 * D * 2 + 8 * case["tokens"]
        return dict(bytes=both if case["op"] == "load" else both + n * (row + 2 * D), flops=0)
    q, kv = _lengths(case)
    h, g = case["heads"], case["group"]
    cells = sum(sum(max(0, min(k, k - n + i + 1)) for i in range(n)) if case["causal"] else n * k for n, k in zip(q, kv))
    size = sum(2 * k * h * row + 4 * -(-k // case["page"]) for n, k in zip(q, kv) if n) + sum(q) * h * g * (4 * D + 4) + 8 * len(q)
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


def exact(case, seed):
    if case["op"] == "plan":
        return None
    s = _inputs(case, seed)
    c, page, fmt = s["cache"], case["page"], case["fmt"]
    h = case["heads"]
    if case["op"] in ("append", "load"):
        at = s["slots"].clamp(min=0)
        out = {}
        for i, name in enumerate("kv"):
            if case["op"] == "append":
                if case["tokens"] * h > 40000:
                    return None
                x = s["qkv"].reshape(case["tokens"], 6, h, D)[:, 4 + i]
                val = _stored(x, fmt, c[name + "_scale"]).to(DEV)
            else:
                val = _values(c[name][at // page, :, at % page], c[name + "_sf"][at // page, :, at % page], fmt, c[name + "_scale"])
            val[s["slots"] < 0] = 0.0
            out[name] = val
        return out
    q, kv = _lengths(case)
    if sum(n * k for n, k in zip(q, kv)) * h * case["group"] > 1.2e9:
        return None
    g = case["group"]
    o = torch.zeros(sum(q), h * g, D, dtype=torch.float64, device=DEV)
    lse = torch.full((h * g, sum(q)), -math.inf, dtype=torch.float64, device=DEV)
    t = 0
    for r, (n, k) in enumerate(zip(q, kv)):
        pages = s["table"][r, : -(-k // page)].long()
        for a in range(h if n and k else 0):
            key, val = (_values(c[x][pages, a].reshape(-1, 64)[:k], c[x + "_sf"][pages, a].flatten(0, 1)[:k], fmt, c[x + "_scale"]) for x in "kv")
            x = s["q"][t: t + n, a * g: (a + 1) * g].double().transpose(0, 1)
            score = torch.matmul(x, key.t()) / math.sqrt(D)
            if case["causal"]:
                score = score.masked_fill(torch.ones(n, k, dtype=torch.bool, device=DEV).triu(k - n + 1), -math.inf)
            w = torch.logsumexp(score, -1)
            p = torch.exp(score - torch.where(torch.isinf(w), 0.0, w)[..., None])
            o[t: t + n, a * g: (a + 1) * g] = torch.matmul(p, val).transpose(0, 1)
            lse[a * g: (a + 1) * g, t: t + n] = w
        t += n
    return dict(o=o, lse=lse)
