"""Rotary positions, windowed and shared-prefix attention and shared pages on the GPU against
plain 64-bit forms.

Rotation's bound, per element, with z = gain (|a| + |b|) of its pair:
  2^-8 |y|      y rounded to bf16 (half a step)
  2^-20 z       the angle: 2^-32 of a turn cut off and half a step of fp32 of at most pi
                (2^-29.3 + 2^-22.3 radians), sine and cosine 2 steps (2^-22), gain and products
                2^-23, together below 2^-20
  2^-134        half the smallest bf16
The attention's bounds are those of the other attention tests: a prefix's (m, l, O) joins in fp32."""
import numpy as np
import pytest

from tests import kv_ref, more_ref
from tests.helpers import host
from tests.test_gpu_kv import bf16, cached, f64, new_cache, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    import torch
    from mxfp8_block_scaled_fa_gb300 import build, mxfa
    build.build()
    assert torch.cuda.is_available()
    assert mxfa.device_status() == 0
    return mxfa


def dev(x, dtype=np.int32):
    import torch
    return torch.from_numpy(np.asarray(x, dtype)).cuda()


# ------------------------------------------------------------------------------- rotation
def make_rope(mx, rot, inter, gain, rng):
    f = 10000.0 ** (-np.arange(rot // 2) / (rot // 2)) * rng.uniform(0.9, 1.1, rot // 2)
    f[-1] = -3.0 * f[-1]                                     # a turn of more than half a turn, modulo one
    return mx.Rope.from_freqs(f.tolist(), inter, gain)


def check_rotation(y, x, positions, rp, inverse=False):
    import torch
    x, y, pos = f64(x), f64(y), np.asarray(host(positions), np.int64)
    rot = 2 * rp.turns.numel()
    angle = more_ref.angles([int(t) for t in host(rp.turns)], pos)
    want, z = more_ref.rotate(x, angle, rot, rp.interleaved, rp.gain, inverse)
    err = np.abs(y - want) - (2.0 ** -8 * np.abs(want) + 2.0 ** -20 * z + 2.0 ** -134)
    assert err.max() <= 0, (float(err.max()), np.unravel_index(err.argmax(), err.shape))
    np.testing.assert_array_equal(y[..., rot:], x[..., rot:])
    # step by step in fp32, as an elementwise form has it; a cosine or sine may be one step off (2^-23 of it at most)
    f32 = kv_ref.f32
    c, s = f32(rp.gain * np.cos(angle))[:, None], f32(rp.gain * np.sin(angle))[:, None] * (-1 if inverse else 1)
    i = np.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if rp.interleaved else (i, i + rot // 2)
    v = x.copy()
    with np.errstate(over="ignore", under="ignore"):
        v[..., a] = f32(f32(x[..., a] * c) - f32(x[..., b] * s))
        v[..., b] = f32(f32(x[..., b] * c) + f32(x[..., a] * s))
    to_bf16 = lambda w: torch.from_numpy(w.astype(np.float32)).bfloat16().double().numpy()
    low, mid, high = (to_bf16(v + d * z) for d in (-2.0 ** -23, 0.0, 2.0 ** -23))
    assert ((low <= y) & (y <= high)).all()
    assert (y != mid).mean() <= 1e-5 + 1.0 / y.size


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("T,H,rot,inter,gain", [
    (1, 1, 128, False, 1.0), (1, 5, 128, True, 1.0), (7, 3, 16, False, 1.0), (7, 2, 16, True, 1.25), (33, 8, 64, False, 0.7),
    (130, 17, 96, False, 1.0), (129, 16, 112, True, 1.3), (2051, 33, 128, False, 1.0), (1500, 40, 48, True, 1.0)])
def test_rope(mx, T, H, rot, inter, gain, inverse):
    import torch
    rng = np.random.default_rng(T + rot)
    rp = make_rope(mx, rot, inter, gain, rng)
    fused = bf16(rng, T, H + 3, 128, scale=3.0).cuda()
    fused[0, 1, :20] = torch.tensor([1e30, -2e-38, 0.0, -0.0, 1e-40] * 4, device="cuda").bfloat16()
    x = fused[:, 1: 1 + H]                                  # strided tokens
    pos = rng.integers(0, 2 ** 31, T)
    pos[: min(T, 5)] = [0, 2 ** 31 - 1, 1, 131071, 2 ** 30][: min(T, 5)]
    p = dev(pos)
    call = mx.rope_bwd if inverse else mx.rope
    y = call(x, rp, p)
    check_rotation(y, x, p, rp, inverse)
    before = fused.clone()
    assert call(x, rp, p, out=x) is x                       # in place, its neighbours as they were
    assert torch.equal(x.view(torch.int16), y.view(torch.int16))
    assert torch.equal(fused[:, 0].view(torch.int16), before[:, 0].view(torch.int16))
    assert torch.equal(fused[:, 1 + H:].view(torch.int16), before[:, 1 + H:].view(torch.int16))
    assert mx.device_status() == 0


def test_rope_leaves_tokens_out(mx):
    import torch
    rng = np.random.default_rng(2)
    rp = mx.Rope.make(64)
    x, pos = bf16(rng, 9, 4, 128).cuda(), dev([3, -1, 5, 0, -2147483648, 1, 2, -1, -1])
    out = torch.full((9, 4, 128), 77.0, dtype=torch.bfloat16, device="cuda")
    mx.rope(x, rp, pos, out=out)
    live = host(pos) >= 0
    check_rotation(out[dev(live, bool)], x[dev(live, bool)], pos[dev(live, bool)], rp)
    assert (host(out.float())[~live] == 77.0).all()
    assert mx.rope(x[:0], rp, pos[:0]).shape == (0, 4, 128)


def test_rope_nan_and_infinity_stay_in_their_pair(mx):
    import torch
    x = torch.ones(2, 2, 128, dtype=torch.bfloat16, device="cuda")
    x[0, 0, 3], x[0, 0, 100], x[1, 1, 70] = float("nan"), float("inf"), float("-inf")
    y = mx.rope(x, mx.Rope.make(64), dev([5, 5]))
    bad = ~torch.isfinite(y.float())
    want = torch.zeros_like(bad)
    want[0, 0, [3, 35, 100]] = True
    want[1, 1, 70] = True
    assert torch.equal(bad, want) and y[0, 0, 100] == float("inf") and y[1, 1, 70] == float("-inf")


def test_rope_gradient(mx):
    """<dy, rope(x)> = <rope_bwd(dy), x>, and the step of the result along each input, by differences."""
    import torch
    rng = np.random.default_rng(4)
    for inter in (False, True):
        rp = mx.Rope.make(96, interleaved=inter, scaling="yarn", factor=8.0)
        pos = dev(rng.integers(0, 100000, 50))
        x, dy = bf16(rng, 50, 3, 128).cuda(), bf16(rng, 50, 3, 128).cuda()
        y, dx = mx.rope(x, rp, pos), mx.rope_bwd(dy, rp, pos)
        a, b = (f64(dy) * f64(y)).sum(), (f64(dx) * f64(x)).sum()
        size = np.abs(f64(dy) * f64(y)).sum() + np.abs(f64(dx) * f64(x)).sum()
        assert abs(a - b) <= 2.0 ** -8 * 1.01 * size        # each element's rounding
        for c in (0, 5, 48, 95, 96, 127):
            e = torch.zeros_like(x)
            e[..., c] = 1.0
            step = f64(mx.rope(e, rp, pos)) - f64(mx.rope(-e, rp, pos))  # twice the derivative
            want = (step * f64(dy)).sum(-1) / 2
            # two products of bf16 values, each off by half a step, and dx by half of its own
            bound = 2.0 ** -8 * (np.abs(step * f64(dy)).sum(-1) / 2 + np.abs(f64(dx)[..., c])) * 1.01
            assert (np.abs(want - f64(dx)[..., c]) <= bound + 2.0 ** -18).all()


@pytest.mark.parametrize("lengths", [None, [129, 0, 70, 256]])
def test_rope_in_a_training_step(mx, lengths):
    """q and k turned, quantized, attended; the gradients turned back: those of the unturned q and k."""
    import torch
    rng = np.random.default_rng(6)
    seqs = mx.Seqs.dense(2, 192) if lengths is None else mx.Seqs.varlen(lengths, "cuda")
    T, H = seqs.total, 2
    rp, pos = mx.Rope.make(128), mx.rope_positions(seqs)
    q, k, v, do = (bf16(rng, T, H, 128).cuda() for _ in range(4))
    qr, kr = mx.rope(q, rp, pos), mx.rope(k, rp, pos)
    check_rotation(qr, q, pos, rp)
    scale = 128 ** -0.5
    quant = lambda x, b: mx.quantize(x, b, seqs)
    o, lse = mx.attention_fwd(quant(qr, mx.ROW), quant(kr, mx.ROW), quant(v, mx.COL), seqs, seqs, scale, causal=True)
    dq, dk, dv = mx.attention_bwd(quant(qr, mx.SQ), quant(kr, mx.SQ), quant(v, mx.ROW), quant(do, mx.SQ), o, do, lse, seqs, seqs, scale, causal=True)
    gq, gk = mx.rope_bwd(dq, rp, pos), mx.rope_bwd(dk, rp, pos)
    check_rotation(gq, dq, pos, rp, inverse=True)
    check_rotation(gk, dk, pos, rp, inverse=True)
    # against differences of the unquantized loss <do, o>: MXFP8's own bar for a gradient's direction
    n = 192 if lengths is None else 129
    angle = more_ref.angles([int(t) for t in host(rp.turns)], range(n))

    def loss(x, y):
        xr, yr = (more_ref.rotate(z, angle, 128, False)[0] for z in (x, y))
        w = np.einsum("ihd,jhd->hij", xr, yr) * scale
        w = np.where(np.tril(np.ones((n, n), bool)), w, -np.inf)
        p = np.exp(w - w.max(-1, keepdims=True))
        p /= p.sum(-1, keepdims=True)
        return (np.einsum("hij,jhd->ihd", p, f64(v)[:n]) * f64(do)[:n]).sum()
    x, y = f64(q)[:n], f64(k)[:n]
    for g, which in ((f64(gq)[:n], 0), (f64(gk)[:n], 1)):
        along = g / np.linalg.norm(g)
        args = [x, y]
        step = []
        for h in (1e-3, -1e-3):
            moved = list(args)
            moved[which] = args[which] + h * along
            step.append(loss(*moved))
        slope = (step[0] - step[1]) / 2e-3
        assert abs(slope - np.linalg.norm(g)) <= 0.1 * np.linalg.norm(g)   # 20 dB, as for the gradients themselves
    assert mx.device_status() == 0


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("T,Hq,H,page,rot,inter", [
    (1, 1, 1, 16, 128, False), (3, 6, 3, 16, 64, True), (61, 32, 8, 16, 128, False), (257, 10, 5, 32, 96, False),
    (700, 16, 1, 64, 16, True), (1200, 40, 8, 128, 128, True)])
def test_append_rope_is_rope_and_append(mx, fmt, T, Hq, H, page, rot, inter):
    import torch
    rng = np.random.default_rng(T + Hq)
    rp = make_rope(mx, rot, inter, 1.1, rng)
    blocks = -(-T // page) + 3
    fused = bf16(rng, T, Hq + 2 * H + 1, 128, scale=2.0).cuda()
    fused[0, Hq, 5] = float("nan")
    q, k, v = fused[:, :Hq], fused[:, Hq: Hq + H], fused[:, Hq + H: Hq + 2 * H]
    slots = rng.permutation(blocks * page)[:T].astype(np.int64)
    pos = rng.integers(0, 2 ** 20, T)
    if T > 4:
        slots[[1, 2]] = -1                                  # no slot: q alone
        pos[[2, T - 1]] = -1                                # no token
    slots, pos = dev(slots, np.int64), dev(pos)
    one, two = (new_cache(mx, blocks, H, page, fmt, fill=0x5A) for _ in range(2))
    got = torch.full((T, Hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    assert mx.kv_append_rope(one, q, k, v, rp, pos, slots, out=got) is got
    want = torch.full((T, Hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    mx.rope(q, rp, pos, out=want)
    mx.kv_append(two, mx.rope(k, rp, pos), v, torch.where(pos < 0, -1, slots))
    bits = lambda t: t.view(torch.uint8) if t.dtype is torch.uint8 else t.view(torch.int16)
    for a, b in ((got, want), (one.k, two.k), (one.v, two.v), (one.k_sf, two.k_sf), (one.v_sf, two.v_sf)):
        assert torch.equal(bits(a.contiguous()), bits(b.contiguous()))
    check_rotation(got[dev(host(pos) >= 0, bool)], q[dev(host(pos) >= 0, bool)], pos[pos >= 0], rp)
    # in place, within the projection that k and v are parts of
    kept = fused[:, Hq:].clone()
    mx.kv_append_rope(one, q, k, v, rp, pos, slots, out=q)
    live = dev(host(pos) >= 0, bool)
    assert torch.equal(bits(q[live].contiguous()), bits(want[live])) and torch.equal(bits(fused[:, Hq:].contiguous()), bits(kept))
    assert torch.equal(one.k, two.k) and torch.equal(one.v_sf, two.v_sf)
    assert mx.device_status() == 0
    mx.kv_append_rope(one, q, k, v, rp, pos, torch.full_like(slots, blocks * page))
    assert mx.device_status() == 7 and torch.equal(one.k, two.k)      # past the cache


# ------------------------------------------------------------------------------ attention
def build(mx, rng, fmt, page, H, G, q_lens, kv_lens, groups=None, hidden=None, extra=2):
    """A cache of the requests' keys in random pages (other rows hold NaN blocks) and q.  groups: (requests, prefix)
    whose first `prefix` keys are those of the first of them; hidden(r, key): keys of no page."""
    import torch
    pages = [-(-k // page) for k in kv_lens]
    blocks = sum(pages) + extra
    width = max(pages + [1]) + 1
    perm = rng.permutation(blocks)
    table, at, slots = np.full((len(kv_lens), width), -1, np.int32), 0, []
    for r, n in enumerate(pages):
        table[r, :n] = perm[at: at + n]
        at += n
    for members, prefix in groups or []:
        for r in members:                                   # whole pages shared; a part of a page is each one's own
            table[r, : prefix // page] = table[members[0], : prefix // page]
    for r, k in enumerate(kv_lens):
        p = np.arange(k)
        slots.append(table[r, p // page].astype(np.int64) * page + p % page)
    c = new_cache(mx, blocks, H, page, fmt, fill=0xFF)
    everything = np.unique(np.concatenate(slots + [np.zeros(0, np.int64)]))
    if len(everything):
        k, v = bf16(rng, len(everything), H, 128), bf16(rng, len(everything), H, 128)
        mx.kv_append(c, k.cuda(), v.cuda(), torch.from_numpy(everything).cuda())
    for members, prefix in groups or []:                    # the part of a page that the first request has
        for r in members:
            slots[r][:prefix] = slots[members[0]][:prefix]
    if hidden is not None:
        for r in range(len(kv_lens)):
            for j in range(pages[r]):
                if all(hidden(r, key) for key in range(j * page, min(kv_lens[r], (j + 1) * page))):
                    table[r, j] = -1 if j % 2 else 1 << 30
    nq = sum(q_lens)
    fused = bf16(rng, nq + 3, H * G + 2, 128).cuda()
    cu = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    return c, fused[:, 1: 1 + H * G], dev(cu), dev(kv_lens), dev(table), slots


def compare(c, q, cu, slots, o, lse, mask, rows=None, scale=128 ** -0.5):
    """Each request's rows within the bounds; mask(r, n, kv) [n, kv]."""
    cu, q64, go, gl = host(cu), f64(q), f64(o), host(lse).astype(np.float64).T
    for r, sl in enumerate(slots):
        a, b = cu[r], cu[r + 1]
        if a == b or (rows is not None and r not in rows):
            continue
        k, v = cached(c, sl) if len(sl) else (np.zeros((0, c.pages.H, 128)),) * 2
        seen = mask(r, b - a, len(sl))
        vmax = np.abs(np.where(np.isfinite(v), v, 0.0)).max(initial=0.0)
        within(go[a:b], gl[a:b], more_ref.attention(q64[a:b], k, v, scale, seen), max(len(sl), 1), vmax)


def results(q):
    import torch
    T, Hq, _ = q.shape
    return (torch.full((T, Hq, 128), 77.0, dtype=torch.bfloat16, device="cuda"),
            torch.full((Hq, T), 77.0, dtype=torch.float32, device="cuda"))


WINDOWS = [
    # few rows: decoding, short and long contexts, windows inside a tile, on its edges, over several
    (0, 16, 2, 8, [1], [201], 50, 4), (1, 16, 1, 1, [1, 1, 1], [1, 2, 700], 1, 0), (0, 32, 2, 4, [1] * 5, [128, 129, 256, 1000, 3], 128, 1),
    (1, 64, 3, 3, [1, 0, 1], [5000, 17, 4097], 1000, 200), (0, 128, 1, 16, [1, 1], [9000, 20], 300, 0), (0, 16, 8, 4, [1] * 9, [3000] * 9, 2047, 130),
    # drafted tokens: several positions in a block of rows, more rows than one block
    (0, 16, 2, 8, [3, 6, 1], [300, 1500, 40], 100, 4), (1, 32, 1, 7, [5, 2], [2000, 700], 37, 129), (0, 64, 2, 6, [8, 7, 0, 8], [9, 1300, 50, 640], 3, 2),
    (0, 16, 1, 12, [4, 4], [6000, 100], 1, 128),
    # prompts
    (0, 64, 2, 4, [150, 3], [700, 300], 100, 5), (1, 16, 1, 8, [257], [257], 64, 0), (0, 128, 1, 2, [300, 65, 1], [1500, 65, 900], 129, 257),
    (1, 32, 2, 3, [90, 0, 40], [1000, 0, 40], 1, 1), (0, 16, 1, 40, [7, 20], [500, 1300], 256, 128),
    # no key in sight: more tokens than keys, none at all
    (0, 16, 2, 4, [5, 3, 1], [2, 0, 0], 4, 1), (1, 64, 1, 8, [100, 60], [30, 0], 7, 3)]


@pytest.mark.parametrize("fmt,page,H,G,q_lens,kv_lens,window,sinks", WINDOWS)
def test_window(mx, fmt, page, H, G, q_lens, kv_lens, window, sinks):
    import torch
    rng = np.random.default_rng(sum(kv_lens) + window)
    unseen = lambda r, key: q_lens[r] == 0 or (key >= sinks and key < kv_lens[r] - q_lens[r] - window + 1)
    c, q, cu, kv, table, slots = build(mx, rng, fmt, page, H, G, q_lens, kv_lens, hidden=unseen)
    o, lse = results(q)
    mx.kv_attention(q, c, cu, kv, table, max(q_lens), 128 ** -0.5, out=(o, lse), window=window, sinks=sinks)
    torch.cuda.synchronize()
    assert mx.device_status() == 0                          # pages out of sight are not looked at
    compare(c, q, cu, slots, o, lse, lambda r, n, k: more_ref.window_mask(n, k, window, sinks))
    rest = sum(q_lens)
    assert (o[rest:].float() == 77.0).all() and (lse[:, rest:] == 77.0).all()
    # every length of table is allowed, and new buffers
    o2, lse2 = mx.kv_attention(q, c, cu, kv, table, max(q_lens), 128 ** -0.5, window=window, sinks=sinks)
    assert torch.equal(o2[:rest].view(torch.int16), o[:rest].view(torch.int16)) and torch.equal(lse2[:, :rest], lse[:, :rest])


@pytest.mark.parametrize("q_lens,kv_lens,G", [([1, 1, 1], [2000, 5, 700], 4), ([4, 6], [3000, 900], 8), ([120, 1], [1500, 64], 4)])
def test_window_over_everything_is_attention(mx, q_lens, kv_lens, G):
    import torch
    rng = np.random.default_rng(9)
    c, q, cu, kv, table, _ = build(mx, rng, 0, 16, 2, G, q_lens, kv_lens)
    want = mx.kv_attention(q, c, cu, kv, table, max(q_lens), 0.09)
    n = sum(q_lens)
    for window, sinks in ((1 << 31, 0), (2 ** 31 - 1, 7), (5000, 0), (1, 1 << 30), (1, 2 ** 31 - 1), (700, 2400)):
        if window >= 1 << 31:
            with pytest.raises(Exception):
                mx.kv_attention(q, c, cu, kv, table, max(q_lens), 0.09, window=window, sinks=sinks)
            continue
        o, lse = mx.kv_attention(q, c, cu, kv, table, max(q_lens), 0.09, window=window, sinks=sinks)
        assert torch.equal(o[:n].view(torch.int16), want[0][:n].view(torch.int16)) and torch.equal(lse[:, :n], want[1][:, :n])


def test_window_nan_blocks(mx):
    """A NaN block of K or V reaches the rows that see its key, and no others."""
    import torch
    rng = np.random.default_rng(11)
    for q_lens, G in (([6], 4), ([100], 2)):
        n = q_lens[0]
        c, q, cu, kv, table, slots = build(mx, rng, 0, 16, 1, G, q_lens, [400])
        key = 400 - n - 20                                  # seen by the first rows alone
        s = int(slots[0][key])
        c.v_sf[s // 16, 0, s % 16, 1] = 0xFF
        c.v[s // 16, 0, s % 16, 16:32] = 0
        s = int(slots[0][2])                                # a sink
        window, sinks = 22, 2
        c.k_sf[s // 16, 0, s % 16, 0] = 0xFF                # key 2: in no row's sight
        c.k[s // 16, 0, s % 16, :16] = 0
        o, lse = results(q)
        mx.kv_attention(q, c, cu, kv, table, n, 0.09, out=(o, lse), window=window, sinks=sinks)
        bad = torch.isnan(o[:n].float())
        assert bad[:2, :, 32:64].all() and not bad[2:].any() and not bad[..., :32].any() and not bad[..., 64:].any()
        compare(c, q, cu, slots, o, lse, lambda r, n, k: more_ref.window_mask(n, k, window, sinks), scale=0.09)
        assert mx.device_status() == 0
        c2, key = table.clone(), 0
        c2[0, 0] = -1                                       # a sink's page that is not there is recorded, its keys left out
        mx.kv_attention(q, c, cu, kv, c2, n, 0.09, out=(o, lse), window=window, sinks=sinks)
        assert mx.device_status() == 7
        compare(c, q, cu, slots, o, lse, lambda r, n, k: more_ref.window_mask(n, k, window, 0), scale=0.09)


SHARED = [
    # (fmt, page, H, G, [(members' new tokens, prefix, members' own keys)], ungrouped requests (new, keys) before and behind)
    (0, 16, 2, 4, [([1, 1, 1], 160, [1, 20, 300])], [], []),
    (1, 64, 1, 8, [([1] * 9, 1024, [1, 5, 64, 65, 200, 900, 1, 2, 3])], [(1, 70)], [(1, 1), (0, 0)]),
    (0, 32, 3, 2, [([1, 1], 33, [1, 90]), ([1], 500, [10]), ([1, 1, 1, 1], 0, [1, 2, 3, 700])], [], []),
    (0, 16, 2, 3, [([4, 6, 1], 1000, [4, 100, 1]), ([2, 0, 5], 17, [9, 0, 129])], [(3, 200)], [(2, 2)]),
    (1, 128, 1, 16, [([2, 3], 129, [128, 3]), ([1, 1], 3000, [1, 129])], [], []),
    # more rows in a group than a request: the prefix goes by the prompts' kernel
    (0, 64, 2, 4, [([1] * 30, 2000, list(range(1, 31)))], [], []),
    (1, 16, 1, 8, [([5] * 12, 777, list(range(5, 17))), ([1] * 3, 100, [1, 1, 1])], [(6, 300)], []),
    (0, 32, 2, 40, [([1, 1, 2], 300, [1, 40, 2])], [], [(1, 600)]),
    # prompts behind a prefix
    (0, 16, 2, 4, [([100, 20, 1], 700, [100, 150, 1])], [], [(1, 90)]),
    (1, 64, 1, 6, [([70, 260], 130, [70, 700]), ([300], 64, [300])], [(33, 33)], []),
    # a group none of whose requests has queries
    (0, 16, 1, 4, [([0, 0], 50, [0, 4]), ([1, 2], 60, [1, 2])], [], [])]


def shared_case(mx, rng, fmt, page, H, G, groups, ahead, behind, **kw):
    q_lens, kv_lens = [n for n, _ in ahead], [k for _, k in ahead]
    starts, named = [len(ahead)], []
    for new, prefix, tails in groups:
        members = list(range(len(q_lens), len(q_lens) + len(new)))
        q_lens += new
        kv_lens += [prefix + t if n or t else 0 for n, t in zip(new, tails)]
        kv_lens[members[0]] = max(kv_lens[members[0]], prefix)
        named.append((members, prefix))
        starts.append(len(q_lens))
    q_lens += [n for n, _ in behind]
    kv_lens += [k for _, k in behind]
    most = max(sum(new) for new, _, _ in groups)
    named = [([r for r in m if kv_lens[r] >= p], p) for m, p in named]
    c, q, cu, kv, table, slots = build(mx, rng, fmt, page, H, G, q_lens, kv_lens, groups=named, **kw)
    for m, p in named:                                      # the first one's row alone is read for the prefix
        for r in m[1:]:
            table[r, : p // page] = -1 if r % 2 else 1 << 30
    return c, q, cu, kv, table, slots, dev(starts), dev([p for _, p, _ in groups]), max(max(q_lens), 1), most, q_lens, kv_lens


@pytest.mark.parametrize("share", [True, False, None])
@pytest.mark.parametrize("case", SHARED)
def test_shared(mx, case, share):
    import torch
    rng = np.random.default_rng(len(case[4]) + case[3])
    c, q, cu, kv, table, slots, starts, pre, max_q, most, q_lens, _ = shared_case(mx, rng, *case)
    o, lse = results(q)
    mx.kv_attention_shared(q, c, cu, kv, table, starts, pre, max_q, most, 128 ** -0.5, out=(o, lse), share=share)
    torch.cuda.synchronize()
    assert mx.device_status() == 0
    compare(c, q, cu, slots, o, lse, lambda r, n, k: more_ref.window_mask(n, k, 1 << 30, 0))
    rest = sum(q_lens)
    assert (o[rest:].float() == 77.0).all() and (lse[:, rest:] == 77.0).all()
    o2, lse2 = mx.kv_attention_shared(q, c, cu, kv, table, starts, pre, max_q, most, 128 ** -0.5, share=share)
    assert torch.equal(o2[:rest].view(torch.int16), o[:rest].view(torch.int16)) and torch.equal(lse2[:, :rest], lse[:, :rest])


def test_shared_without_groups(mx):
    import torch
    rng = np.random.default_rng(1)
    c, q, cu, kv, table, _ = build(mx, rng, 1, 16, 2, 4, [1, 2], [300, 40])
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    got = mx.kv_attention_shared(q, c, cu, kv, table, dev([0]), none, 2, 0, 0.1)
    want = mx.kv_attention(q, c, cu, kv, table, 2, 0.1)
    assert torch.equal(got[0][:3].view(torch.int16), want[0][:3].view(torch.int16)) and torch.equal(got[1][:, :3], want[1][:, :3])


@pytest.mark.parametrize("share", [True, False])
@pytest.mark.parametrize("rows", [2, 30])
def test_shared_nan_in_the_prefix(mx, rows, share):
    import torch
    rng = np.random.default_rng(3)
    c, q, cu, kv, table, slots, starts, pre, max_q, most, _, _ = shared_case(mx, rng, 0, 16, 1, 4, [([1] * rows, 300, [1] * rows)], [(1, 50)], [])
    s = int(slots[1][123])
    c.v_sf[s // 16, 0, s % 16, 3] = 0xFF
    c.v[s // 16, 0, s % 16, 48:] = 0
    o, lse = results(q)
    mx.kv_attention_shared(q, c, cu, kv, table, starts, pre, max_q, most, 0.1, out=(o, lse), share=share)
    bad = torch.isnan(o[: rows + 1].float())
    assert not bad[0].any() and bad[1:, :, 96:].all() and not bad[1:, :, :96].any() and mx.device_status() == 0
    q[1, 2, 7] = float("inf")                                # an infinite query: its row alone
    mx.kv_attention_shared(q, c, cu, kv, table, starts, pre, max_q, most, 0.1, out=(o, lse), share=share)
    bad = torch.isnan(o[: rows + 1].float()).all(-1)
    assert bad[1, 2] and bad.sum() == 1


@pytest.mark.parametrize("share", [True, False])
def test_shared_outside_its_bounds(mx, share):
    """Groups and requests that are not as documented are left out and recorded; the others are computed."""
    import torch
    rng = np.random.default_rng(8)
    args = (0, 16, 2, 4, [([1, 1], 64, [1, 9]), ([1, 1], 100, [1, 50]), ([1], 40, [5])], [], [])
    for starts, pre, kv_of, lost in (
            (None, [64, 100, 1 << 20], None, {4}), (None, [64, -1, 40], None, {2, 3}), ([0, 2, 4, 99], None, None, {4}),
            ([-3, 2, 4, 5], None, None, {0, 1}), (None, None, {3: 100}, {3}), (None, None, {1: 3}, {1}), ([0, 2, 1, 5], None, None, None)):
        c, q, cu, kv, table, slots, st, p, max_q, most, q_lens, kv_lens = shared_case(mx, rng, *args)
        st = st if starts is None else dev(starts)
        p = p if pre is None else dev(pre)
        for r, n in (kv_of or {}).items():
            kv[r] = n
        o, lse = results(q)
        mx.kv_attention_shared(q, c, cu, kv, table, st, p, max_q, most, 0.1, out=(o, lse), share=share)
        torch.cuda.synchronize()
        assert mx.device_status() == 7
        if lost is None:
            continue
        compare(c, q, cu, slots, o, lse, lambda r, n, k: more_ref.window_mask(n, k, 1 << 30, 0), rows=set(range(5)) - lost, scale=0.1)
        for r in lost:
            assert (o[r].float() == 77.0).all(), (r, starts, pre, kv_of)
    c, q, cu, kv, table, slots, st, p, _, _, _, _ = shared_case(mx, rng, *args)
    o, lse = results(q)
    mx.kv_attention_shared(q, c, cu, kv, table, st, p, 1, 1, 0.1, out=(o, lse), share=share)  # groups of 2 tokens, 1 allowed
    assert mx.device_status() == 7 and (o[:4].float() == 77.0).all()


# ---------------------------------------------------------------------------------- pages
def random_pages(rng, R, page, width, spare):
    ctx = [int(rng.integers(0, width * page + 1)) if rng.random() < 0.8 else 0 for _ in range(R)]
    have = [-(-c // page) for c in ctx]
    blocks = sum(have) + spare + 2
    perm = rng.permutation(blocks)
    table, at = np.full((R, width), -1), 0
    for r in range(R):
        table[r, :have[r]] = perm[at: at + have[r]]
        at += have[r]
    head = int(rng.integers(0, 5 * blocks))
    ring = np.full(blocks, -9)
    ring[(head + np.arange(spare)) % blocks] = perm[at: at + spare]
    return ctx, table, ring, head, head + spare, blocks


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("R,F,page,width,spare", [(2, 1, 16, 3, 1), (9, 5, 32, 7, 2), (40, 30, 16, 3000, 40), (700, 600, 128, 5, 300), (3, 0, 16, 4, 2),
                                                  (17, 16, 64, 1, 16)])
def test_fork_and_free(mx, R, F, page, width, spare, inplace):
    import torch
    for seed in range(3):
        rng = np.random.default_rng(100 * R + seed)
        ctx, table, ring, head, tail, blocks = random_pages(rng, R - F, page, width, spare)
        table = np.concatenate([table, np.full((F, width), -5)])
        order = rng.permutation(R)                          # rows in any order
        place = np.argsort(order)
        table = table[order]
        src = place[rng.integers(0, R - F, F)] if F else np.zeros(0, int)
        dst = place[R - F:]
        lens = np.array([rng.integers(0, ctx[order[s]] + 1) if rng.random() < 0.5 else ctx[order[s]] for s in src], int)
        t, f, refs = dev(table), dev(ring), mx.kv_refs(blocks)
        state = dev([head, tail, -5], np.int64)
        out = None
        if inplace:
            e = lambda: torch.full((F,), -77, dtype=torch.int32, device="cuda")
            out = mx.KvFork(e(), e(), e(), state)
        got = mx.kv_fork(t, dev(src), dev(dst), dev(lens), refs, f, state, page, out=out)
        wt, wr, wf = table.tolist(), [0] * blocks, ring.tolist()
        want = more_ref.fork(wt, src.tolist(), dst.tolist(), lens.tolist(), wr, wf, head, tail, page)
        for g, w in zip((got.from_blocks, got.to_blocks, got.lens, got.ring_state), want):
            assert host(g).tolist() == w
        assert host(t).tolist() == wt and host(refs).tolist() == wr and host(f).tolist() == wf
        # some forks and some sources are given up, in parts, in two calls
        rows = np.concatenate([dst, place[: R - F]])
        ends = np.concatenate([-(-lens // page), [-(-n // page) for n in ctx]]).astype(int)
        some = rng.random(R) < 0.7
        mid = np.where(rng.random(R) < 0.5, 0, rng.integers(0, ends + 1))
        s = got.ring_state
        for first, end in ((mid, ends), (np.zeros(R, int), mid)):
            w = more_ref.free(wt, rows[some].tolist(), first[some].tolist(), end[some].tolist(), wr, wf, *want[3])
            s = mx.kv_free(t, dev(rows[some]), dev(first[some]), dev(end[some]), refs, f, s, out=s if inplace else None)
            want = (None, None, None, w)
            assert host(s).tolist() == w and host(refs).tolist() == wr and host(f).tolist() == wf
        assert host(t).tolist() == wt and mx.device_status() == 0


def test_free_many_blocks(mx):
    rng = np.random.default_rng(7)
    for blocks, width in ((1, 1), (31, 31), (8192, 4000), (70001, 40000)):
        table = rng.permutation(blocks)[: 1 * width].reshape(1, width)
        refs, ring = rng.integers(0, 2, blocks), np.zeros(blocks, int)
        t, r, f = dev(table), dev(refs), dev(ring)
        end = width - width // 3
        s = mx.kv_free(t, dev([0, 0]), dev([0, width // 2]), dev([end, width // 2]), r, f, dev([5, 9, 3], np.int64))
        wr, wf = refs.tolist(), ring.tolist()
        want = more_ref.free(table.tolist(), [0], [0], [end], wr, wf, 5, 9, 3)
        assert host(s).tolist() == want and host(r).tolist() == wr and host(f).tolist() == wf and mx.device_status() == 0


def test_pages_outside_their_bounds(mx):
    table = [[1, 2, 99, -1], [3, 4, 5, 6], [-1] * 4, [-1] * 4]
    t, refs, ring = dev(table), mx.kv_refs(8), dev([0, 7, 50, 0, 0, 0, 0, 0])
    f = mx.kv_fork(t, dev([0, 1, -1, 1, 1, 4]), dev([2, 3, 2, 1, 9, 2]), dev([48, 65, 5, 5, 5, 5]), refs, ring, dev([0, 3, 0], np.int64), 16)
    assert mx.device_status() == 7
    assert host(t).tolist() == [[1, 2, 99, -1], [3, 4, 5, 6], [1, 2, -1, -1], [-1] * 4]   # 99 is no block; 65 tokens are too many
    assert host(refs).tolist() == [0, 1, 1, 0, 0, 0, 0, 0] and host(f.lens).tolist() == [48, 0, 0, 0, 0, 0]
    assert host(f.ring_state).tolist() == [0, 3, 0]
    f = mx.kv_fork(t, dev([1, 1, 1]), dev([2, 3, 0]), dev([17, 1, 1]), refs, ring, dev([0, 3, 0], np.int64), 16)
    assert mx.device_status() == 7                           # the ring's third entry is no block
    assert host(f.to_blocks).tolist() == [0, 7, -1] and host(f.lens).tolist() == [17, 1, 0] and host(t)[0, 0] == -1
    s = mx.kv_free(dev([[9, -1, 3, -1]]), dev([0, 1, 0, 0]), dev([0, 0, -1, 0]), dev([4, 1, 1, 5]), mx.kv_refs(8), ring, dev([2, 3, 0], np.int64))
    assert mx.device_status() == 7 and host(s).tolist() == [2, 4, 0] and host(ring)[3] == 3
    s = mx.kv_free(dev([[3, 3]]), dev([0]), dev([0]), dev([2]), refs.zero_(), ring, dev([2, 3, 0], np.int64))
    assert mx.device_status() == 7 and host(s).tolist() == [2, 4, 0] and not refs.any()    # given up twice: freed once


@pytest.mark.parametrize("fmt,H,page,blocks", [(0, 1, 16, 5), (1, 3, 16, 9), (0, 8, 128, 6), (1, 5, 64, 40), (0, 2, 16, 8192), (1, 1, 32, 3000), (0, 3, 16, 300)])
def test_copy_blocks(mx, fmt, H, page, blocks):
    import torch
    rng = np.random.default_rng(blocks)
    c = new_cache(mx, blocks, H, page, fmt)
    for t in (c.k, c.v, c.k_sf, c.v_sf):
        t.copy_(torch.from_numpy(rng.integers(0, 256, tuple(t.shape), np.uint8)))
    want = [host(t).copy() for t in (c.k, c.v, c.k_sf, c.v_sf)]
    a, b = [0, 0, -1, 3, 2, 1], [4, 1, 2, -1, 2, blocks]
    for x, y in ((0, 4), (0, 1)):
        for w in want:
            w[y] = w[x]
    mx.kv_copy_blocks(c, dev(a), dev(b))
    for t, w in zip((c.k, c.v, c.k_sf, c.v_sf), want):
        np.testing.assert_array_equal(host(t), w)
    assert mx.device_status() == 7                           # block `blocks` is past the cache
    # moves: a block that is read is written too, in a ring and along a line, more of them than a CTA has threads
    for n in (blocks - 1, blocks):
        before = [host(t).copy() for t in (c.k, c.v, c.k_sf, c.v_sf)]
        order = rng.permutation(blocks)[:n]
        mx.kv_copy_blocks(c, dev(order), dev(np.roll(order, 1)))
        for t, w in zip((c.k, c.v, c.k_sf, c.v_sf), before):
            w[np.roll(order, 1)] = w[order]
            np.testing.assert_array_equal(host(t), w)
    # blocks written by several pairs: the last one's stays
    a, b = (rng.integers(-1, blocks, blocks) for _ in range(2))
    b[: blocks // 2] = b[blocks - blocks // 2:]
    before = [host(t).copy() for t in (c.k, c.v, c.k_sf, c.v_sf)]
    mx.kv_copy_blocks(c, dev(a), dev(b))
    for t, old in zip((c.k, c.v, c.k_sf, c.v_sf), before):
        w = old.copy()
        for x, y in zip(a, b):
            if x >= 0 and y >= 0:
                w[y] = old[x]
        np.testing.assert_array_equal(host(t), w)
    mx.kv_copy_blocks(c, dev([]), dev([]))
    assert mx.device_status() == 0


# ------------------------------------------------------------------------------- together
class Server:
    """Requests served step by step with every operator, beside a plain record of their keys and values."""

    def __init__(self, mx, rng, fmt, page, H, G, R, width, blocks):
        import torch
        self.mx, self.rng, self.page, self.H, self.G, self.R = mx, rng, page, H, G, R
        self.c = new_cache(mx, blocks, H, page, fmt, fill=0xFF)
        self.rp = mx.Rope.make(64, interleaved=True, scaling="yarn", factor=2.0)
        self.ring, self.state = mx.kv_ring(blocks)
        self.refs = mx.kv_refs(blocks)
        self.table = torch.full((R, width), -1, dtype=torch.int32, device="cuda")
        self.ctx = [0] * R
        self.slots = [[] for _ in range(R)]                  # of each request's tokens

    def tokens(self, new):
        T = sum(new)
        fused = bf16(self.rng, T, self.H * (self.G + 2), 128).cuda()
        Hq = self.H * self.G
        return fused[:, :Hq], fused[:, Hq: Hq + self.H], fused[:, Hq + self.H:]

    def step(self, new, attend):
        mx, (q, k, v) = self.mx, self.tokens(new)
        plan = mx.kv_plan(dev(self.ctx), dev(new), self.table, self.ring, self.state, self.page, sum(new))
        self.state = plan.ring_state
        qr = mx.kv_append_rope(self.c, q, k, v, self.rp, plan.positions, plan.slots)
        at, s = 0, host(plan.slots)
        for r, n in enumerate(new):
            self.slots[r] = self.slots[r][: self.ctx[r]] + s[at: at + n].tolist()
            self.ctx[r] += n
            at += n
        assert host(plan.kv_lens).tolist() == self.ctx and (s >= 0).all()
        kr = mx.rope(k, self.rp, plan.positions)
        gk, _ = mx.kv_load(self.c, plan.slots)
        bound = np.abs(f64(kr)).reshape(*kr.shape[:2], -1, 32).max(-1, keepdims=True).repeat(32, -1).reshape(kr.shape)
        assert (np.abs(f64(gk) - f64(kr)) <= bound * 0.26 + 1e-6).all()   # half of E2M1's widest step, 1 of 4, and saturation
        o, lse = attend(qr, plan)
        return qr, plan, o, lse

    def check(self, qr, plan, o, lse, window=1 << 30, sinks=0):
        compare(self.c, qr, plan.cu_q, [np.array(s[: c], np.int64) for s, c in zip(self.slots, self.ctx)], o, lse,
                lambda r, n, k: more_ref.window_mask(n, k, window, sinks))
        assert self.mx.device_status() == 0


@pytest.mark.parametrize("fmt,page,stream", [(0, 16, False), (1, 64, True)])
def test_serving(mx, fmt, page, stream):
    """A prompt, forked, continued by each fork over the shared prefix, drafted tokens in a window, forks dropped."""
    import torch
    rng = np.random.default_rng(page)
    with torch.cuda.stream(torch.cuda.Stream() if stream else torch.cuda.default_stream()):
        s = Server(mx, rng, fmt, page, 2, 4, 6, 2 + 900 // page, 400)
        scale = 128 ** -0.5
        all_of = lambda qr, p: mx.kv_attention(qr, s.c, p.cu_q, p.kv_lens, s.table, 300, scale)
        s.check(*s.step([261, 0, 0, 0, 40, 0], all_of))
        free0 = host(s.state).tolist()
        f = mx.kv_fork(s.table, dev([0, 0, 0]), dev([1, 2, 3]), dev([261, 261, 261]), s.refs, s.ring, s.state, page)
        mx.kv_copy_blocks(s.c, f.from_blocks, f.to_blocks)
        s.state = f.ring_state
        for r in (1, 2, 3):
            s.ctx[r] = 261
            to = host(s.table)[r]
            s.slots[r] = [int(to[p // page]) * page + p % page for p in range(261)]
        prefix = 261 // page * page
        shared = lambda qr, p: mx.kv_attention_shared(qr, s.c, p.cu_q, p.kv_lens, s.table, dev([0, 4]), dev([prefix]), 8, 32, scale, share=fmt == 0)
        for new in ([1, 1, 1, 1, 1, 5], [1, 3, 0, 8, 2, 1], [2, 2, 2, 2, 0, 1]):
            s.check(*s.step(new, shared))
        for window, sinks in ((50, 4), (1, 0), (1000, 3)):
            inside = lambda qr, p: mx.kv_attention(qr, s.c, p.cu_q, p.kv_lens, s.table, 8, scale, window=window, sinks=sinks)
            s.check(*s.step([1, 4, 1, 0, 3, 1], inside), window, sinks)
        # everything is given up: the ring holds every block again, once
        used = [-(-c // page) for c in s.ctx]
        s.state = mx.kv_free(s.table, dev(range(6)), dev([0] * 6), dev(used), s.refs, s.ring, s.state)
        head, tail, _ = host(s.state).tolist()
        assert tail - head == 400 and not s.refs.any()
        ring = host(s.ring)
        assert sorted(ring[(head + np.arange(400)) % 400].tolist()) == list(range(400)) and free0[2] == 0


def test_captured_and_replayed(mx):
    """A decoding step of every operator captured once and replayed with new inputs, workspaces and counters in place."""
    import torch
    rng = np.random.default_rng(21)
    R, page, H, G, width, blocks = 5, 16, 2, 4, 40, 300
    s = Server(mx, rng, 0, page, H, G, R, width, blocks)
    s.step([200, 0, 0, 0, 30], lambda qr, p: (None, None))
    f = mx.kv_fork(s.table, dev([0, 0, 0]), dev([1, 2, 3]), dev([200] * 3), s.refs, s.ring, s.state, page)
    mx.kv_copy_blocks(s.c, f.from_blocks, f.to_blocks)
    for r in (1, 2, 3):
        s.ctx[r] = 200
        s.slots[r] = [int(host(s.table)[r][p // page]) * page + p % page for p in range(200)]
    ctx, state = dev(s.ctx), f.ring_state.clone()
    ones = dev([1] * R)
    i32 = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")
    step = mx.KvStep(i32(R + 1), ctx, torch.empty(R, dtype=torch.int64, device="cuda"), i32(R), state)
    Hq = H * G
    fused = torch.zeros(R, Hq + 2 * H, 128, dtype=torch.bfloat16, device="cuda")
    q, k, v = fused[:, :Hq], fused[:, Hq: Hq + H], fused[:, Hq + H:]
    starts, pre, turned = dev([0, 4]), dev([192]), torch.empty(R, Hq, 128, dtype=torch.bfloat16, device="cuda")

    def one():
        mx.kv_plan(ctx, ones, s.table, s.ring, state, page, R, out=step)
        mx.kv_append_rope(s.c, q, k, v, s.rp, step.positions, step.slots, out=turned)
        a = mx.kv_attention_shared(turned, s.c, step.cu_q, step.kv_lens, s.table, starts, pre, 1, 4, 0.09, share=True)
        b = mx.kv_attention(turned, s.c, step.cu_q, step.kv_lens, s.table, 1, 0.09, window=70, sinks=2)
        return a, b
    side = torch.cuda.Stream()
    keep = [t.clone() for t in (ctx, s.table, s.ring, state, s.c.k, s.c.v, s.c.k_sf, s.c.v_sf)]
    with torch.cuda.stream(side):
        one()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a, b = one()
    for t, w in zip((ctx, s.table, s.ring, state, s.c.k, s.c.v, s.c.k_sf, s.c.v_sf), keep):
        t.copy_(w)
    for i in range(20):
        fused.copy_(bf16(rng, *fused.shape))
        g.replay()
        torch.cuda.synchronize()
        for r in range(R):
            s.slots[r].append(int(step.slots[r]))
            s.ctx[r] += 1
        assert host(ctx).tolist() == s.ctx
        sl = [np.array(x, np.int64) for x in s.slots]
        compare(s.c, turned, step.cu_q, sl, *a, lambda r, n, k: more_ref.window_mask(n, k, 1 << 30, 0), scale=0.09)
        compare(s.c, turned, step.cu_q, sl, *b, lambda r, n, k: more_ref.window_mask(n, k, 70, 2), scale=0.09)
    assert mx.device_status() == 0
    # the same step's page calls, captured, with the ring's counters in place
    src, dst, lens = dev([1, 2]), dev([3, 0]), dev([90, 33])
    out = mx.KvFork(i32(2), i32(2), i32(2), state)
    rows, first, end = dev([3, 0]), dev([0, 0]), dev([6, 3])
    refs = s.refs.clone()
    g2 = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g2):
        mx.kv_fork(s.table, src, dst, lens, refs, s.ring, state, page, out=out)
        mx.kv_copy_blocks(s.c, out.from_blocks, out.to_blocks)
        mx.kv_free(s.table, rows, first, end, refs, s.ring, state, out=state)
    wt, wr, wf, (head, tail, _) = host(s.table).tolist(), host(refs).tolist(), host(s.ring).tolist(), host(state).tolist()
    for i in range(3):
        g2.replay()
        torch.cuda.synchronize()
        w = more_ref.fork(wt, [1, 2], [3, 0], [90, 33], wr, wf, head, tail, page)
        head, tail, _ = more_ref.free(wt, [3, 0], [0, 0], [6, 3], wr, wf, *w[3])
        assert host(out.to_blocks).tolist() == w[1] and host(state).tolist()[:2] == [head, tail]
        assert host(s.table).tolist() == wt and host(refs).tolist() == wr and host(s.ring).tolist() == wf
        a, b = (int(x[0]) for x in (out.from_blocks, out.to_blocks))
        assert torch.equal(s.c.k[a], s.c.k[b]) and torch.equal(s.c.v_sf[a], s.c.v_sf[b])
    assert mx.device_status() == 0


def test_two_streams_at_once(mx):
    import torch
    rng = np.random.default_rng(31)
    shared = shared_case(mx, rng, 0, 16, 2, 4, [([1] * 20, 600, list(range(1, 21)))], [], [])
    c, q, cu, kv, table, slots = build(mx, rng, 1, 32, 2, 4, [3, 200, 1], [700, 900, 300])
    st = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for _ in range(10):
        a = mx.kv_attention_shared(shared[1], shared[0], *shared[2:5], *shared[6:10], 0.1, stream=st[0], share=True)
        b = mx.kv_attention(q, c, cu, kv, table, 200, 0.1, stream=st[1], window=333, sinks=5)
        outs.append((a, b))
    torch.cuda.synchronize()
    for a, b in outs:
        n, m = int(shared[2][-1]), int(cu[-1])
        assert torch.equal(a[0][:n], outs[0][0][0][:n]) and torch.equal(b[0][:m], outs[0][1][0][:m])
    compare(shared[0], shared[1], shared[2], shared[5], *outs[0][0], lambda r, n, k: more_ref.window_mask(n, k, 1 << 30, 0), scale=0.1)
    compare(c, q, cu, slots, *outs[0][1], lambda r, n, k: more_ref.window_mask(n, k, 333, 5), scale=0.1)
    assert mx.device_status() == 0


def test_calls_on_a_given_stream(mx):
    """With stream= the work and the memory of the results belong to that stream, behind what it already holds."""
    import torch
    rng = np.random.default_rng(51)
    side = torch.cuda.Stream()
    rp, pos = mx.Rope.make(32), dev(np.arange(3000))
    x = bf16(rng, 3000, 8, 128).cuda()
    want = mx.rope(x, rp, pos)
    late = torch.empty_like(x)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        big = torch.randn(4096, 4096, device="cuda")
        for _ in range(3):
            big = big @ big * 1e-4                           # keeps the stream busy
        late.copy_(x)
    got = mx.rope(late, rp, pos, stream=side)
    back = mx.rope_bwd(got, rp, pos, stream=side)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(back, mx.rope_bwd(want, rp, pos))
    c = new_cache(mx, 9, 2, 16, 0)
    q, k, v = (bf16(rng, 5, n, 128).cuda() for n in (4, 2, 2))
    slots = dev([3, 40, 41, 100, 7], np.int64)
    torch.cuda.synchronize()
    qr = mx.kv_append_rope(c, q, k, v, rp, pos[:5], slots, stream=side)
    mx.kv_copy_blocks(c, dev([0, 2]), dev([8, 7]), stream=side)
    t, refs, ring, state = dev([[0, 2], [-1, -1]]), mx.kv_refs(9), dev([1, 3, 4, 5, 6, 7, 8, -1, -1]), dev([0, 7, 0], np.int64)
    torch.cuda.synchronize()
    f = mx.kv_fork(t, dev([0]), dev([1]), dev([20]), refs, ring, state, 16, stream=side)
    st = mx.kv_free(t, dev([0, 1]), dev([0, 0]), dev([2, 2]), refs, ring, f.ring_state, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(qr, mx.rope(q, rp, pos[:5])) and torch.equal(c.k[8], c.k[0]) and c.k[0].any()
    assert host(f.lens).tolist() == [20] and host(st).tolist() == [1, 10, 0] and host(ring)[[7, 8, 0]].tolist() == [0, 1, 2]
    assert mx.device_status() == 0


@pytest.mark.parametrize("share", [True, False])
def test_many_requests_behind_many_prefixes(mx, share):
    """Hundreds of groups, of one and of several requests, and more requests than a CTA of the plan has threads."""
    import torch
    rng = np.random.default_rng(61)
    groups = []
    for g in range(300):
        m = int(rng.integers(1, 5))
        groups.append(([1] * m, int(rng.integers(0, 60)), [int(x) for x in rng.integers(1, 40, m)]))
    c, q, cu, kv, table, slots, starts, pre, max_q, most, q_lens, _ = shared_case(mx, rng, 0, 16, 1, 4, groups, [(1, 5)], [(1, 9)])
    o, lse = results(q)
    mx.kv_attention_shared(q, c, cu, kv, table, starts, pre, max_q, most, 128 ** -0.5, out=(o, lse), share=share)
    assert mx.device_status() == 0
    compare(c, q, cu, slots, o, lse, lambda r, n, k: more_ref.window_mask(n, k, 1 << 30, 0))
    # by the prompts' kernel: every group may have 20 tokens
    o2, lse2 = results(q)
    mx.kv_attention_shared(q, c, cu, kv, table, starts, pre, max_q, 20, 128 ** -0.5, out=(o2, lse2), share=share)
    assert mx.device_status() == 0
    compare(c, q, cu, slots, o2, lse2, lambda r, n, k: more_ref.window_mask(n, k, 1 << 30, 0))


def test_prompts_of_many_blocks_in_a_window(mx):
    """More blocks of rows than a warp has lanes, for one request beside others."""
    rng = np.random.default_rng(71)
    c, q, cu, kv, table, slots = build(mx, rng, 0, 64, 1, 8, [1200, 1, 40], [1300, 200, 90])
    o, lse = results(q)
    mx.kv_attention(q, c, cu, kv, table, 1200, 128 ** -0.5, out=(o, lse), window=130, sinks=3)
    assert mx.device_status() == 0
    compare(c, q, cu, slots, o, lse, lambda r, n, k: more_ref.window_mask(n, k, 130, 3))


def test_far_blocks(mx):
    """Blocks whose offsets pass 32 bits: 2.2 million rows of 8 heads behind one another."""
    import torch
    rng = np.random.default_rng(41)
    blocks, H, page = 70000, 8, 128                          # 4.6 GB of codes each of K and V
    c = mx.KvCache.empty(blocks, H, page)
    table = dev([[69999, 3, 69998, 69997]])
    k, v = bf16(rng, 400, H, 128).cuda(), bf16(rng, 400, H, 128).cuda()
    slots = np.concatenate([host(table)[0, j].astype(np.int64) * page + np.arange(page) for j in range(4)])[:400]
    rp, pos = mx.Rope.make(), dev(np.arange(400))
    q = mx.kv_append_rope(c, bf16(rng, 400, H, 128).cuda(), k, v, rp, pos, dev(slots, np.int64))
    o, lse = mx.kv_attention(q[-2:], c, dev([0, 2]), dev([400]), table, 2, 0.09, window=140, sinks=130)
    compare(c, q[-2:], dev([0, 2]), [slots], o, lse, lambda r, n, k: more_ref.window_mask(n, k, 140, 130), scale=0.09)
    o, lse = mx.kv_attention_shared(q[-2:], c, dev([0, 1, 2]), dev([399, 399]), torch.cat([table, table]), dev([0, 2]), dev([256]), 1, 2, 0.09, share=True)
    compare(c, q[-2:], dev([0, 1, 2]), [slots[:399]] * 2, o, lse, lambda r, n, k: more_ref.window_mask(n, k, 1 << 30, 0), scale=0.09)
    mx.kv_copy_blocks(c, dev([69999]), dev([60000]))
    assert torch.equal(c.k[60000], c.k[69999]) and torch.equal(c.v_sf[60000], c.v_sf[69999]) and c.k[60000].any()
    assert mx.device_status() == 0
