"""4-bit cache on the GPU against plain 64-bit forms: the step plan (whole numbers,
equal), store and load (codes, scales and values equal), and attention within
a bound derived from its roundings.

Attention's bound, per output element, with a = sum p |v| / sum p and s = the
largest scale sum_d |q_d k_d| of the row:
  2^-8 |o|              o rounded to bf16 (half a step)
  2^-11 a               P rounded to binary16 (half a step), weighted by |v|
  2 (2^-17 s + 2^-20) a the scores: 128 fp32 products and sums (128 * 2^-24 of their
                        absolute sum, s), the base-2 exponent and its approximation;
                        they enter the numerator and the denominator
  n 2^-33 max|v|        weights below the smallest binary16: P carries 2^8
lse: 2^-17 s + 2^-20 + 2^-22 |lse|."""
import numpy as np
import pytest

from tests import kv_ref
from tests.helpers import host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    import torch
    from mxfp8_block_scaled_fa_gb300 import build, mxfa
    build.build()
    assert torch.cuda.is_available()
    assert mxfa.device_status() == 0
    return mxfa


def bf16(rng, *shape, scale=1.0):
    import torch
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).bfloat16()


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def scales(fmt):
    return (1.0, 1.0) if fmt == 0 else (float(np.float32(6.0 / 2688)), float(np.float32(9.0 / 2688)))


def new_cache(mx, blocks, H, page, fmt, fill=None):
    ks, vs = scales(fmt)
    c = mx.KvCache.empty(blocks, H, page, fmt, ks, vs)
    if fill is not None:
        for t in (c.k, c.v, c.k_sf, c.v_sf):
            t.fill_(fill)
    return c


def cached(c, slots):
    """Values of cache rows, in float64, decoded by the reference."""
    slots = np.asarray(slots)
    b, r = slots // c.pages.page, slots % c.pages.page
    ks, vs = scales(c.fmt)
    return (kv_ref.dequantize(host(c.k)[b, :, r], host(c.k_sf)[b, :, r], c.fmt, ks),
            kv_ref.dequantize(host(c.v)[b, :, r], host(c.v_sf)[b, :, r], c.fmt, vs))


# ------------------------------------------------------------------------ store and load
def edge_rows(T, H, rng):
    x = rng.standard_normal((T, H, 128)).astype(np.float32) * 2
    flat = x.reshape(-1, 128)
    flat[0, :32] = 0.0
    flat[0, 32:64] = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0] * 4) * np.array([1, -1] * 16)
    flat[0, 64:96] = 2.0 ** -40
    flat[0, 96:] = 3.0e38
    if len(flat) > 1:
        flat[1, :32] = np.linspace(-7.9, 7.9, 32)
        flat[1, 37] = np.inf
        flat[1, 70] = np.nan
        flat[1, 127] = -np.inf
    if len(flat) > 2:
        flat[2, :] = 2.0 ** -130
        flat[2, :32] = 2.0 ** (np.arange(32) - 20.0)
    return x


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("T,H,page", [(1, 1, 16), (2, 3, 16), (17, 8, 32), (333, 2, 64), (129, 5, 128), (40, 16, 16)])
def test_append_and_load(mx, fmt, T, H, page):
    import torch
    rng = np.random.default_rng(T + 7 * H)
    blocks = -(-T // page) + 3
    c = new_cache(mx, blocks, H, page, fmt, fill=0x5A)
    before = [host(t).copy() for t in (c.k, c.v, c.k_sf, c.v_sf)]
    fused = np.concatenate([rng.standard_normal((T, 2, 128)).astype(np.float32), edge_rows(T, H, rng), edge_rows(T, H, rng)], 1)
    fused = torch.from_numpy(fused).bfloat16().cuda()
    k, v = fused[:, 2: 2 + H], fused[:, 2 + H:]         # strided tokens
    slots = rng.permutation(blocks * page)[:T].astype(np.int64)
    if T > 4:
        slots[[1, T - 1]] = -1
    mx.kv_append(c, k, v, torch.from_numpy(slots).cuda())
    gk, gv = mx.kv_load(c, torch.from_numpy(slots).cuda())
    torch.cuda.synchronize()
    live = slots >= 0
    b, r = slots[live] // page, slots[live] % page
    want = [x.copy() for x in before]
    for i, (t, st, got) in enumerate(((k, scales(fmt)[0], gk), (v, scales(fmt)[1], gv))):
        codes, sf, val = kv_ref.quantize(f64(t)[live], fmt, st)
        want[i][b, :, r], want[2 + i][b, :, r] = codes, sf
        full = np.zeros((T, H, 128))
        full[live] = val
        np.testing.assert_array_equal(host(got.float()), host(torch.from_numpy(kv_ref.f32(full)).bfloat16().float()))
    # the cache byte for byte, rows without a token as they were
    for t, w in zip((c.k, c.v, c.k_sf, c.v_sf), want):
        np.testing.assert_array_equal(host(t), w)
    assert mx.device_status() == 0


@pytest.mark.parametrize("fmt", [0, 1])
def test_load_repeats_and_ranges(mx, fmt):
    import torch
    rng = np.random.default_rng(3)
    c = new_cache(mx, 4, 2, 16, fmt)
    k, v = bf16(rng, 64, 2, 128).cuda(), bf16(rng, 64, 2, 128).cuda()
    mx.kv_append(c, k, v, torch.arange(64, device="cuda"))
    slots = torch.tensor([5, 5, 63, -1, 0, 64, 1 << 40], device="cuda")
    gk, gv = mx.kv_load(c, slots)
    assert mx.device_status() == 7                      # 64 and 2^40 are past the cache
    ak, av = mx.kv_load(c, torch.arange(64, device="cuda"))
    for g, a in ((gk, ak), (gv, av)):
        assert torch.equal(g[:5], torch.stack([a[5], a[5], a[63], torch.zeros_like(a[0]), a[0]]))
        assert not g[5:].any()
    codes = c.k.clone()
    mx.kv_append(c, k[:3], v[:3], torch.tensor([64, 1 << 40, -(1 << 40)], device="cuda"))
    assert mx.device_status() == 7 and torch.equal(codes, c.k)


# ----------------------------------------------------------------------------------- plan
def run_plan(mx, ctx, new, table, ring, head, tail, page, tokens, inplace=False):
    import torch
    i32 = lambda x: torch.tensor(np.asarray(x, np.int32), device="cuda")
    c, n, t, f = i32(ctx), i32(new), i32(table), i32(ring)
    state = torch.tensor([head, tail, -5], dtype=torch.int64, device="cuda")
    out = None
    if inplace:
        out = mx.KvStep(torch.empty(len(ctx) + 1, dtype=torch.int32, device="cuda"), c,
                        torch.empty(tokens, dtype=torch.int64, device="cuda"),
                        torch.empty(tokens, dtype=torch.int32, device="cuda"), state)
    s = mx.kv_plan(c, n, t, f, state, page, tokens, out=out)
    got = [host(x).tolist() for x in (s.cu_q, s.kv_lens, s.slots, s.positions, s.ring_state)]
    return got, host(t), host(f)


def random_step(rng, R, page, width, spare, prompts):
    new = np.ones(R, np.int64)
    new[rng.random(R) < 0.2] = 0
    new[rng.random(R) < 0.1] = -1
    for r in rng.permutation(R)[:prompts]:
        new[r] = rng.integers(1, max(2, width * page // 2))
    ctx = np.array([0 if rng.random() < 0.2 else rng.integers(0, width * page - max(0, a) + 1) for a in new])
    have = -(-ctx // page)
    blocks = int(have.sum()) + spare
    perm = rng.permutation(blocks)
    table, at = np.full((R, width), -1), 0
    for r in range(R):
        table[r, :have[r]] = perm[at: at + have[r]]
        at += have[r]
    head = int(rng.integers(0, 5 * blocks + 1))
    ring = np.full(max(blocks, 1), -9)
    ring[(head + np.arange(spare)) % max(blocks, 1)] = perm[at:]
    return ctx, new, table, ring, head, head + spare


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("R,page,width,spare,prompts", [
    (1, 16, 4, 3, 1), (7, 16, 9, 40, 2), (33, 32, 5, 7, 4), (64, 64, 12, 0, 3), (513, 16, 8, 90, 30), (1030, 128, 3, 2000, 9),
    (16384, 16, 3, 4000, 40)])
def test_plan(mx, R, page, width, spare, prompts, inplace):
    for seed in range(3 if R < 10000 else 1):
        rng = np.random.default_rng(1000 * R + seed)
        ctx, new, table, ring, head, tail = random_step(rng, R, page, width, spare, prompts)
        tokens = int(np.maximum(new, 0).sum()) + int(rng.integers(0, 40))
        got, gt, gf = run_plan(mx, ctx, new, table, ring, head, tail, page, tokens, inplace)
        t, f = table.tolist(), ring.tolist()
        want = kv_ref.plan(ctx.tolist(), new.tolist(), t, f, head, tail, page, tokens)
        for g, w in zip(got, want):
            assert g == w
        np.testing.assert_array_equal(gt, t)
        np.testing.assert_array_equal(gf, f)
        assert mx.device_status() == 0


def test_plan_no_requests_and_too_long(mx):
    got, _, _ = run_plan(mx, [], [], np.zeros((0, 4)), [1, 2], 0, 2, 16, 5)
    assert got == [[0], [], [-1] * 5, [-1] * 5, [0, 2, 0]]
    # a request past its row of the table gets nothing and is recorded; the others are served
    got, t, _ = run_plan(mx, [60, 3, 0], [5, 1, 20], [[1, 2, 3, 4], [5, -1, -1, -1], [-1] * 4], list(range(10, 20)), 0, 10, 16, 26)
    assert got[1] == [60, 4, 20] and got[2] == [-1] * 5 + [83] + list(range(160, 180)) and got[4] == [2, 10, 0]
    assert t[0].tolist() == [1, 2, 3, 4] and t[2].tolist() == [10, 11, -1, -1]
    assert mx.device_status() == 7


# ------------------------------------------------------------------------------ attention
def build(mx, rng, fmt, page, H, G, q_lens, kv_lens, extra=2, poison=True, kscale=1.0, pad_rows=3):
    """A cache with the requests' keys in random pages (unused rows hold NaN blocks if `poison`), and q."""
    import torch
    pages = [-(-k // page) for k in kv_lens]
    blocks = sum(pages) + extra
    width = max(pages + [1]) + 1
    perm = rng.permutation(blocks)
    table, at, slots = np.full((len(kv_lens), width), -1, np.int32), 0, []
    for r, (n, k) in enumerate(zip(pages, kv_lens)):
        table[r, :n] = perm[at: at + n]
        at += n
        p = np.arange(k)
        slots.append(table[r, p // page].astype(np.int64) * page + p % page if k else np.zeros(0, np.int64))
    c = new_cache(mx, blocks, H, page, fmt, fill=0xFF if poison else None)
    T = sum(kv_lens)
    k, v = bf16(rng, T, H, 128, scale=kscale), bf16(rng, T, H, 128)
    if T:
        mx.kv_append(c, k.cuda(), v.cuda(), torch.from_numpy(np.concatenate(slots)).cuda())
    Hq = H * G
    nq = sum(q_lens)
    fused = bf16(rng, nq + pad_rows, Hq + 2, 128).cuda()
    cu = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    return c, fused[:, 1: 1 + Hq], torch.from_numpy(cu).cuda(), torch.tensor(kv_lens, dtype=torch.int32, device="cuda"), \
        torch.from_numpy(table).cuda(), slots


def check(mx, c, q, cu, kv, table, slots, causal, scale=128 ** -0.5, max_q=None):
    import torch
    T, Hq, _ = q.shape
    o = torch.full((T, Hq, 128), 77.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((Hq, T), 77.0, dtype=torch.float32, device="cuda")
    n = np.diff(host(cu))
    mx.kv_attention(q, c, cu, kv, table, int(max(n.max(), 1)) if max_q is None else max_q, scale, causal=causal, out=(o, lse))
    torch.cuda.synchronize()
    compare(c, q, cu, slots, causal, scale, o, lse)
    return o, lse


def within(go, gl, ref, n, vmax):
    """Asserts the bounds of the header; go [n, Hq, 128], gl [n, Hq], ref = kv_ref.attention's."""
    ro, rl, ra, rs = ref
    ds = 2.0 ** -17 * rs + 2.0 ** -20
    bad = np.isnan(ro)
    np.testing.assert_array_equal(np.isnan(go), bad)
    with np.errstate(invalid="ignore"):
        tol = 2.0 ** -8 * np.abs(ro) + (2.0 ** -11 + 2 * ds[..., None]) * ra + n * 2.0 ** -33 * vmax
        err = np.where(bad, 0.0, np.abs(go - ro) - tol)
    assert err.max(initial=-1.0) <= 0, (float(err.max()), np.unravel_index(err.argmax(), err.shape))
    np.testing.assert_array_equal(np.isneginf(gl), np.isneginf(rl))
    np.testing.assert_array_equal(np.isnan(gl), np.isnan(rl))
    fine = np.isfinite(rl)
    assert (np.abs(gl[fine] - rl[fine]) <= ds[fine] + 2.0 ** -22 * np.abs(rl[fine])).all()


def compare(c, q, cu, slots, causal, scale, o, lse):
    cu_h, q64, go, gl = host(cu), f64(q), f64(o), host(lse).astype(np.float64).T
    for r, sl in enumerate(slots):
        a, b = cu_h[r], cu_h[r + 1]
        if a == b:
            continue
        k, v = cached(c, sl) if len(sl) else (np.zeros((0, c.pages.H, 128)),) * 2
        vmax = np.abs(v[np.isfinite(v)]).max() if np.isfinite(v).any() else 0.0
        within(go[a:b], gl[a:b], kv_ref.attention(q64[a:b], k, v, scale, causal), len(sl), vmax)
    end = cu_h[-1]
    assert (go[end:] == 77.0).all() and (gl[end:] == 77.0).all()     # rows behind the last query, left as they were


DECODE = [
    # G, H, page, kv lengths
    (1, 1, 16, [1]), (1, 2, 16, [2, 31, 32, 33]), (4, 2, 16, [127, 128, 129, 0, 500]), (8, 1, 32, [1000, 15, 16, 17]),
    (16, 1, 64, [257, 3, 1024]), (3, 5, 128, [700, 128, 1]), (7, 2, 16, [2500, 1, 64]), (12, 1, 64, [640]), (5, 3, 32, [95] * 20),
]


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("G,H,page,kv", DECODE)
def test_attention_one_token(mx, fmt, G, H, page, kv):
    rng = np.random.default_rng(sum(kv) + G)
    args = build(mx, rng, fmt, page, H, G, [1] * len(kv), kv)
    check(mx, *args, causal=True)
    assert mx.device_status() == 0


MORE = [
    # G, H, page, query lengths, kv lengths
    (4, 2, 16, [5, 0, 3, 1], [300, 40, 3, 0]), (8, 1, 32, [4, 4], [129, 4]), (1, 3, 64, [16, 7], [200, 7]),
    (2, 2, 16, [33, 9, 2], [400, 9, 1000]), (4, 1, 128, [70, 1], [513, 77]), (1, 1, 16, [200], [200]), (3, 2, 16, [6, 50, 11], [3, 20, 11]),
    (16, 1, 16, [9], [1500]), (40, 1, 16, [1, 2], [100, 90]), (8, 2, 16, [130, 31], [258, 640]),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("G,H,page,ql,kv", MORE)
def test_attention_more_tokens(mx, fmt, causal, G, H, page, ql, kv):
    rng = np.random.default_rng(sum(kv) + sum(ql))
    args = build(mx, rng, fmt, page, H, G, ql, kv)
    check(mx, *args, causal=causal)
    assert mx.device_status() == 0


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("ql,kv", [([1], [40000]), ([1, 1, 1], [20000, 5, 9000]), ([3, 2], [12000, 8200]), ([24], [6000])])
def test_attention_long(mx, fmt, ql, kv):
    """Keys split over many CTAs and joined; the same call twice gives the same bits."""
    import torch
    rng = np.random.default_rng(11)
    args = build(mx, rng, fmt, 64, 1, 8, ql, kv, kscale=2.0)
    o, lse = check(mx, *args, causal=True)
    o2, lse2 = check(mx, *args, causal=True)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert mx.device_status() == 0


MIXED = [
    # G, H, page, query lengths, kv lengths: prompts among decoding requests, many keys behind
    # few rows, blocks of rows that end inside a token's group, empty ones
    (8, 2, 16, [130, 1, 1, 3, 40, 0], [400, 900, 17, 64, 2000, 30]), (4, 1, 64, [100], [9000]), (16, 1, 32, [17, 1, 5], [5000, 3000, 5]),
    (12, 2, 16, [50, 2], [64, 700]), (1, 4, 128, [513, 1], [513, 1300]), (5, 1, 16, [300, 60, 1], [100, 60, 0]),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("G,H,page,ql,kv", MIXED)
def test_attention_mixed(mx, fmt, causal, G, H, page, ql, kv):
    import torch
    rng = np.random.default_rng(sum(kv) + 3 * sum(ql))
    args = build(mx, rng, fmt, page, H, G, ql, kv)
    o, lse = check(mx, *args, causal=causal)
    o2, lse2 = check(mx, *args, causal=causal, max_q=max(ql) + 5)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert mx.device_status() == 0


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("size", [1e-30, 1e-3, 300.0, 1e30])
def test_attention_query_range(mx, fmt, size):
    """Queries far from one (the scale brings the scores back), and rows of zeros."""
    rng = np.random.default_rng(5)
    c, q, cu, kv, table, slots = build(mx, rng, fmt, 16, 2, 2, [1, 2], [70, 50])
    q = (q.float() * size).bfloat16()
    q[0, 1] = 0
    check(mx, c, q, cu, kv, table, slots, causal=True, scale=128 ** -0.5 / size)
    assert mx.device_status() == 0


@pytest.mark.parametrize("ql", [[1, 1], [4, 3], [40, 50]])
@pytest.mark.parametrize("fmt", [0, 1])
def test_attention_sharp(mx, fmt, ql):
    """Scores spread over hundreds: one key takes all the weight, others vanish."""
    rng = np.random.default_rng(6)
    c, q, cu, kv, table, slots = build(mx, rng, fmt, 16, 2, 4, ql, [700, 333], kscale=1.2)
    check(mx, c, (q.float() * 30).bfloat16(), cu, kv, table, slots, causal=True)
    assert mx.device_status() == 0


@pytest.mark.parametrize("ql", [[6, 6], [60, 45]])
@pytest.mark.parametrize("where", ["k", "v"])
@pytest.mark.parametrize("fmt", [0, 1])
def test_attention_nan_only_where_seen(mx, fmt, where, ql):
    """A NaN block in a late key reaches the queries that see the key and no other."""
    import torch
    rng = np.random.default_rng(8)
    c, q, cu, kv, table, slots = build(mx, rng, fmt, 16, 2, 2, ql, [100, 64])
    sf = c.k_sf if where == "k" else c.v_sf
    codes = c.k if where == "k" else c.v
    for r, key in ((0, 97), (1, 61), (1, 63)):
        b, row = divmod(int(slots[r][key]), 16)
        sf[b, 1, row, 2] = 0xFF if fmt == 0 else 0x7F
        codes[b, 1, row, (32 if fmt == 0 else 16): (48 if fmt == 0 else 24)] = 0
    o, lse = check(mx, c, q, cu, kv, table, slots, causal=True)
    assert torch.isnan(o).any() and not torch.isnan(o).all()
    assert mx.device_status() == 0


@pytest.mark.parametrize("ql", [[1, 1, 1], [2, 40, 3]])
def test_attention_bad_index(mx, ql):
    """Blocks outside the cache count as keys that are not there; lengths outside
    their tables leave the request out.  Both are recorded, nothing else changes."""
    import torch
    rng = np.random.default_rng(9)
    c, q, cu, kv, table, slots = build(mx, rng, 0, 16, 1, 4, ql, [100, 200, 60])
    table[1, 3], table[1, 7] = c.k.shape[0], -1
    keep = np.concatenate([np.arange(0, 48), np.arange(64, 112), np.arange(128, 200)])
    o = torch.full(q.shape, 77.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((4, q.shape[0]), 77.0, device="cuda")
    mx.kv_attention(q, c, cu, kv, table, max(ql), 0.1, causal=False, out=(o, lse))
    assert mx.device_status() == 7
    compare(c, q, cu, [slots[0], slots[1][keep], slots[2]], False, 0.1, o, lse)
    bad = kv.clone()
    bad[0] = table.shape[1] * 16 + 1
    o.fill_(77.0), lse.fill_(77.0)
    mx.kv_attention(q, c, cu, bad, table, max(ql), 0.1, causal=False, out=(o, lse))
    assert mx.device_status() == 7
    assert (o[:ql[0]] == 77.0).all() and (o[ql[0]: sum(ql)] != 77.0).any(-1).all()
    short = cu.clone()
    short[3] = q.shape[0] + 1                      # the last request would pass the end of q
    o.fill_(77.0), lse.fill_(77.0)
    mx.kv_attention(q, c, short, kv, table, max(ql) + 10, 0.1, causal=False, out=(o, lse))
    assert mx.device_status() == 7 and (o[ql[0] + ql[1]:] == 77.0).all()


@pytest.mark.parametrize("ql", [[1, 1], [40, 24]])
def test_attention_far_offsets(mx, ql):
    """Pages past 4 GB of codes (the byte offset needs more than 32 bits)."""
    import torch
    rng = np.random.default_rng(10)
    H, page, blocks = 8, 64, 140000                     # 4.6 GB of codes each for K and V
    ks, vs = scales(1)
    u8 = lambda *s: torch.empty(s, dtype=torch.uint8, device="cuda")
    one = lambda x: torch.tensor([x], dtype=torch.float32, device="cuda")
    c = mx.KvCache(u8(blocks, H, page, 64), u8(blocks, H, page, 64), u8(blocks, H, page, 8), u8(blocks, H, page, 8), 1, one(ks), one(vs))
    table = torch.tensor([[blocks - 1, 5], [blocks - 3, blocks - 2]], dtype=torch.int32, device="cuda")
    lens = [90, 128]
    slots = [np.concatenate([np.arange(64) + (blocks - 1) * page, np.arange(26) + 5 * page]),
             np.concatenate([np.arange(64) + (blocks - 3) * page, np.arange(64) + (blocks - 2) * page])]
    k, v = bf16(rng, sum(lens), H, 128), bf16(rng, sum(lens), H, 128)
    sl = torch.from_numpy(np.concatenate(slots)).cuda()
    mx.kv_append(c, k.cuda(), v.cuda(), sl)
    gk, gv = mx.kv_load(c, sl)
    wk, wv = kv_ref.quantize(f64(k), 1, ks)[2], kv_ref.quantize(f64(v), 1, vs)[2]
    r16 = lambda x: torch.from_numpy(x).float().bfloat16()
    assert torch.equal(gk.cpu(), r16(wk)) and torch.equal(gv.cpu(), r16(wv))
    cu = np.array([0, ql[0], sum(ql)], np.int32)
    q = bf16(rng, sum(ql), 2 * H, 128).cuda()
    o, lse = mx.kv_attention(q, c, torch.from_numpy(cu).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), table, max(ql), 128 ** -0.5)
    at, go, gl = 0, f64(o), host(lse).astype(np.float64).T
    for r, n in enumerate(lens):
        ref = kv_ref.attention(f64(q)[cu[r]: cu[r + 1]], wk[at: at + n], wv[at: at + n], 128 ** -0.5, True)
        within(go[cu[r]: cu[r + 1]], gl[cu[r]: cu[r + 1]], ref, n, np.abs(wv).max())
        at += n
    assert mx.device_status() == 0


# --------------------------------------------------------------------------- as one run
def serve(mx, fmt, page, H, G, steps, stream=None, graph=False):
    """A small server: requests come with prompts, decode, and end; blocks are reused.
    Every step's output is checked against attention over all tokens stored so far."""
    import torch
    rng = np.random.default_rng(page + H)
    R, blocks, width, T = 5, 24, 6, 64
    c = new_cache(mx, blocks, H, page, fmt, fill=0xFF)
    ring, state = mx.kv_ring(blocks)
    table = torch.full((R, width), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(R, dtype=torch.int32, device="cuda")
    new = torch.zeros(R, dtype=torch.int32, device="cuda")
    ks, vs = scales(fmt)
    qkv = torch.zeros(T, H * G + 2 * H, 128, dtype=torch.bfloat16, device="cuda")
    out = (torch.empty(T, H * G, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(H * G, T, dtype=torch.float32, device="cuda"))
    i32 = dict(dtype=torch.int32, device="cuda")
    step_buf = mx.KvStep(torch.zeros(R + 1, **i32), lens, torch.empty(T, dtype=torch.int64, device="cuda"), torch.empty(T, **i32), state)

    def step(s=None):
        mx.kv_plan(lens, new, table, ring, state, page, T, out=step_buf, stream=s)
        mx.kv_append(c, qkv[:, H * G: H * G + H], qkv[:, H * G + H:], step_buf.slots, stream=s)
        mx.kv_attention(qkv[:, :H * G], c, step_buf.cu_q, lens, table, T, 128 ** -0.5, out=out, stream=s)

    g = None
    if graph:
        step()                                          # nothing new: no effect
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
    keys = [np.zeros((0, H, 128)) for _ in range(R)]
    vals = [np.zeros((0, H, 128)) for _ in range(R)]
    for n in range(steps):
        counts = [int(rng.integers(1, 12)) if len(keys[r]) == 0 else -1 if rng.random() < 0.12 else 1 for r in range(R)]
        x = bf16(rng, T, H * G + 2 * H, 128)
        qkv.copy_(x), new.copy_(torch.tensor(counts, dtype=torch.int32))
        out[0].fill_(77.0), out[1].fill_(77.0)
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        g.replay() if graph else step(stream)
        if stream is not None:
            torch.cuda.current_stream().wait_stream(stream)
        torch.cuda.synchronize()
        assert host(state)[2] == 0
        at = 0
        go, gl, x64 = f64(out[0]), host(out[1]).astype(np.float64).T, f64(x)
        for r, m in enumerate(counts):
            if m < 0:
                keys[r], vals[r] = keys[r][:0], vals[r][:0]
                continue
            rows = x64[at: at + m]
            keys[r] = np.concatenate([keys[r], kv_ref.quantize(rows[:, H * G: H * G + H], fmt, ks)[2]])
            vals[r] = np.concatenate([vals[r], kv_ref.quantize(rows[:, H * G + H:], fmt, vs)[2]])
            ref = kv_ref.attention(rows[:, :H * G], keys[r], vals[r], 128 ** -0.5, True)
            within(go[at: at + m], gl[at: at + m], ref, len(keys[r]), np.abs(vals[r]).max())
            at += m
        assert (go[at:] == 77.0).all()
        assert host(lens).tolist() == [len(k) for k in keys]
    used = sum(-(-len(k) // page) for k in keys)
    taken, put, _ = host(state).tolist()
    assert put - taken == blocks - used                 # every block is free or in use
    live = [b for r in range(R) for b in host(table)[r, : -(-len(keys[r]) // page)].tolist()]
    free = [int(host(ring)[i % blocks]) for i in range(taken, put)]
    assert sorted(live + free) == list(range(blocks))
    assert mx.device_status() == 0


@pytest.mark.parametrize("fmt", [0, 1])
def test_serving_steps(mx, fmt):
    serve(mx, fmt, 16, 2, 2, 14)


def test_serving_on_another_stream(mx):
    import torch
    serve(mx, 0, 16, 1, 4, 8, stream=torch.cuda.Stream())


@pytest.mark.parametrize("fmt", [0, 1])
def test_serving_as_a_replayed_graph(mx, fmt):
    serve(mx, fmt, 16, 2, 2, 14, graph=True)


def test_two_graphs_and_streams_at_once(mx):
    """Captured calls with workspaces of their own run at the same time."""
    import torch
    rng = np.random.default_rng(12)
    sets = [build(mx, rng, f, 64, 2, 4, [1, 1, 1], [5000, 3000, 700]) for f in (0, 1)]
    graphs, outs = [], []
    for c, q, cu, kv, table, _ in sets:
        o = (torch.full(q.shape, 77.0, dtype=torch.bfloat16, device="cuda"), torch.full((8, q.shape[0]), 77.0, device="cuda"))
        ws = torch.full((mx.mxfa_kv_attn_workspace_size(3, 1, table.shape[1] * 64, 8, 2),), 0xFF, dtype=torch.uint8, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            mx.kv_attention(q, c, cu, kv, table, 1, 128 ** -0.5, out=o, ws=ws)
        graphs.append((g, ws)), outs.append(o)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for (g, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for (c, q, cu, kv, table, slots), o in zip(sets, outs):
        compare(c, q, cu, slots, True, 128 ** -0.5, *o)
    assert mx.device_status() == 0


def test_workspace(mx):
    """Short contexts need none; where one is needed, too small a one is refused."""
    import torch
    rng = np.random.default_rng(13)
    for keys, need_any in ((50, False), (5000, True)):
        c, q, cu, kv, table, slots = build(mx, rng, 0, 16, 1, 4, [1], [keys])
        need = mx.mxfa_kv_attn_workspace_size(1, 1, table.shape[1] * 16, 4, 1)
        assert (need > 0) == need_any
        if need:
            with pytest.raises(mx.MxfaError) as e:
                mx.kv_attention(q, c, cu, kv, table, 1, 0.1, ws=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
            assert e.value.status == 4
            o = [torch.full(x, 77.0, dtype=d, device="cuda") for x, d in ((q.shape, torch.bfloat16), ((4, q.shape[0]), torch.float32))]
            mx.kv_attention(q, c, cu, kv, table, 1, 128 ** -0.5, out=o, ws=torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda"))
            compare(c, q, cu, slots, True, 128 ** -0.5, *o)


# ------------------------------------------------------- calls that allocate their results
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("page,G,ql,kv", [(16, 4, [1, 1, 1], [70, 0, 9]), (64, 8, [1, 3], [3000, 41]), (32, 2, [90, 1, 0, 12], [500, 77, 30, 12])])
def test_new_buffers_are_as_given_ones(mx, fmt, page, G, ql, kv):
    """The same bits from a call that allocates its results, one that is given them, and one on another stream."""
    import torch
    rng = np.random.default_rng(29)
    c, q, cu, lens, table, slots = build(mx, rng, fmt, page, 2, G, ql, kv)
    n, most, scale = int(cu[-1]), max(ql), 128 ** -0.5
    o, lse = mx.kv_attention(q, c, cu, lens, table, most, scale)
    assert o.shape == q.shape and o.dtype == torch.bfloat16 and lse.shape == (2 * G, q.shape[0]) and o.is_contiguous()
    given = torch.empty_like(o, memory_format=torch.contiguous_format), torch.empty_like(lse)
    mx.kv_attention(q, c, cu, lens, table, most, scale, causal=1, out=given)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = mx.kv_attention(q, c, cu, lens, table, most, scale, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for x, y in (given, other):
        assert torch.equal(o[:n].view(torch.int16), x[:n].view(torch.int16)) and torch.equal(lse[:, :n], y[:, :n])
    o[n:], lse[:, n:] = 77.0, 77.0                                   # not written by the call
    compare(c, q, cu, slots, True, scale, o, lse)
    sl = torch.from_numpy(np.concatenate(slots + [np.array([-1])])).cuda()
    k, v = mx.kv_load(c, sl)
    k2, v2 = mx.kv_load(c, sl, out=(torch.empty_like(k), torch.empty_like(v)))
    assert torch.equal(k.view(torch.int16), k2.view(torch.int16)) and torch.equal(v.view(torch.int16), v2.view(torch.int16))


def test_plan_with_new_buffers(mx):
    import torch
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    made = []
    for own in (False, True):
        ring, state = mx.kv_ring(9)
        table = torch.full((3, 4), -1, dtype=torch.int32, device="cuda")
        e = lambda n, t: torch.empty(n, dtype=t, device="cuda")
        out = mx.KvStep(e(4, torch.int32), e(3, torch.int32), e(40, torch.int64), e(40, torch.int32), e(3, torch.int64)) if own else None
        s = mx.kv_plan(i32(0, 0, 0), i32(17, 1, 16), table, ring, state, 16, 40, out=out)
        made.append([s.cu_q, s.kv_lens, s.slots, s.positions, s.ring_state, table, ring])
    for x, y in zip(*made):
        assert x.dtype == y.dtype and torch.equal(x, y)
    empty = mx.kv_plan(i32(), i32(), torch.empty((0, 4), dtype=torch.int32, device="cuda"), ring, state, 16, 0)
    assert empty.cu_q.tolist() == [0] and empty.slots.shape == (0,)


def test_refusals_name_what_is_wrong(mx):
    """Nothing of a refused call runs, whichever check it fails."""
    import torch
    c = new_cache(mx, 4, 2, 16, 0)
    before = c.k.clone()
    rows = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    slots = torch.zeros(5, dtype=torch.int64, device="cuda")
    bad_rows = [(ValueError, rows(5, 3, 128)), (TypeError, rows(5, 2, 128).float()), (ValueError, rows(5, 128, 2).transpose(1, 2)),
                (ValueError, rows(5, 2, 128).cpu()), (ValueError, rows(4, 2, 128)), (mx.MxfaError, rows(1, 2, 128).expand(5, 2, 128)),
                (mx.MxfaError, rows(2600)[1:1 + 5 * 256].view(5, 2, 128))]
    for err, x in bad_rows:
        with pytest.raises(err):
            mx.kv_append(c, x, rows(5, 2, 128), slots)
        with pytest.raises(err):
            mx.kv_append(c, rows(5, 2, 128), x, slots)
    for err, s in ((TypeError, slots.int()), (ValueError, slots[:4]), (ValueError, slots.cpu()), (ValueError, torch.zeros(10, dtype=torch.int64, device="cuda")[::2])):
        with pytest.raises(err):
            mx.kv_append(c, rows(5, 2, 128), rows(5, 2, 128), s)
    with pytest.raises(TypeError):
        mx.kv_load(c, slots.int())
    with pytest.raises(ValueError):
        mx.kv_load(c, slots.cpu())
    good = dict(q=rows(5, 4, 128), cache=c, cu_q=i32(2), kv_lens=i32(1), block_table=i32(1, 4), max_q=5, scale=0.1)
    for err, kw in ((ValueError, dict(q=rows(5, 3, 128))), (TypeError, dict(q=rows(5, 4, 128).half())), (ValueError, dict(cu_q=i32(3))),
                    (TypeError, dict(kv_lens=i32(1).long())), (ValueError, dict(block_table=i32(2, 4))), (ValueError, dict(block_table=i32(4))),
                    (ValueError, dict(block_table=i32(1, 8)[:, ::2])), (mx.MxfaError, dict(scale=0.0)), (mx.MxfaError, dict(scale=float("nan"))),
                    (mx.MxfaError, dict(max_q=-1)), (ValueError, dict(ws=torch.empty(1, dtype=torch.uint8, device="cuda").expand(1 << 20)))):
        with pytest.raises(err):
            mx.kv_attention(**{**good, **kw})
    plan = dict(ctx_lens=i32(3), new_lens=i32(3), block_table=i32(3, 4), free_ring=i32(8), ring_state=torch.zeros(3, dtype=torch.int64, device="cuda"),
                page=16, tokens=4)
    for err, kw in ((ValueError, dict(new_lens=i32(2))), (TypeError, dict(free_ring=i32(8).long())), (mx.MxfaError, dict(page=48)),
                    (ValueError, dict(ring_state=torch.zeros(2, dtype=torch.int64, device="cuda"))), (mx.MxfaError, dict(block_table=i32(3, 0)))):
        with pytest.raises(err):
            mx.kv_plan(**{**plan, **kw})
    with pytest.raises(mx.MxfaError):
        mx.kv_plan(**{**plan, "new_lens": plan["ctx_lens"], "free_ring": plan["ctx_lens"]})     # written and read
    torch.cuda.synchronize()
    assert torch.equal(c.k, before) and mx.device_status() == 0


@pytest.mark.parametrize("fmt", [0, 1])
def test_copies_of_a_cache(mx, fmt):
    """A deep copy has its own rows, a shallow one shares them."""
    import copy
    import torch
    rng = np.random.default_rng(31)
    c = new_cache(mx, 3, 2, 16, fmt)
    x, slots = bf16(rng, 7, 2, 128).cuda(), torch.arange(7, device="cuda")
    mx.kv_append(c, x, x, slots)
    k0, v0 = mx.kv_load(c, slots)
    deep, flat = copy.deepcopy(c), copy.copy(c)
    y = bf16(rng, 7, 2, 128).cuda()
    mx.kv_append(deep, y, y, slots)
    assert torch.equal(mx.kv_load(c, slots)[0], k0) and not torch.equal(mx.kv_load(deep, slots)[0], k0)
    mx.kv_append(flat, y, y, slots)
    for a, b in zip(mx.kv_load(c, slots), mx.kv_load(deep, slots)):
        assert torch.equal(a, b)


def test_mixed_calls_at_once_on_filled_workspaces(mx):
    """Prompts among decoding requests, items cut between CTAs: two captured calls on two streams and two eager ones,
    each on a workspace that is filled anew before every run, leave no row unjoined."""
    import torch
    rng = np.random.default_rng(41)
    runs = []
    for fmt, ql, kv in ((0, [100, 1, 1, 3], [9000, 700, 4000, 64]), (1, [1, 300, 1], [3000, 5000, 17])):
        args = build(mx, rng, fmt, 64, 2, 4, ql, kv)
        c, q, cu, lens, table, _ = args
        need = mx.mxfa_kv_attn_workspace_size(len(ql), max(ql), table.shape[1] * 64, 8, 2)
        assert need > 0
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        o = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda"), torch.empty(8, q.shape[0], device="cuda")

        def call(c=c, q=q, cu=cu, lens=lens, table=table, most=max(ql), o=o, ws=ws):
            ws.fill_(0xFF), o[0].fill_(77.0), o[1].fill_(77.0)
            mx.kv_attention(q, c, cu, lens, table, most, 128 ** -0.5, out=o, ws=ws)
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        runs.append((args, call, g, o, torch.cuda.Stream()))
    for captured in (False, True):
        torch.cuda.synchronize()
        for _ in range(20):
            for _, call, g, _, s in runs:
                with torch.cuda.stream(s):
                    g.replay() if captured else call()
        torch.cuda.synchronize()
        for (c, q, cu, _, _, slots), _, _, o, _ in runs:
            compare(c, q, cu, slots, True, 128 ** -0.5, *o)
    assert mx.device_status() == 0


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("n,h,page", [(3, 0, 16), (0, 2, 16), (3, 2, 0)])
def test_empty_cache_refused_on_a_gpu(mx, fmt, n, h, page):
    with pytest.raises(ValueError):
        mx.KvCache.empty(n, h, page, fmt)


@pytest.mark.parametrize("fmt", [0, 1])
def test_results_over_the_cache_refused_on_a_gpu(mx, fmt):
    """Results that lie over the cache they are read from: refused, and nothing of the cache changes."""
    import torch
    rng = np.random.default_rng(43)
    c, q, cu, lens, table, slots = build(mx, rng, fmt, 16, 2, 2, [1, 2], [70, 50], poison=False)
    before = [t.clone() for t in (c.k, c.v, c.k_sf, c.v_sf)]
    n = q.shape[0]
    o, lse = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda"), torch.empty((4, n), device="cuda")
    over = lambda t, like: t.view(-1)[: like.numel() * like.element_size()].view(like.dtype).view(like.shape)
    sl = torch.arange(3, device="cuda")
    k = torch.empty((3, 2, 128), dtype=torch.bfloat16, device="cuda")
    for t in (c.k, c.v):
        for out in ((over(t, o), lse), (o, over(t, lse))):
            with pytest.raises(mx.MxfaError) as e:
                mx.kv_attention(q, c, cu, lens, table, 2, 0.1, out=out)
            assert e.value.status == 1
        for out in ((over(t, k), k), (k, over(t, k))):
            with pytest.raises(mx.MxfaError) as e:
                mx.kv_load(c, sl, out=out)
            assert e.value.status == 1
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(before, (c.k, c.v, c.k_sf, c.v_sf))) and mx.device_status() == 0


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("ql,kv", [([1, 2], [1, 40]), ([6, 3], [300, 3]), ([1, 1], [5000, 2]), ([70, 20], [90, 10])])
def test_attention_infinite_query(mx, fmt, ql, kv):
    """An infinite channel makes every score of its row infinite or NaN, and so the row NaN, also
    where all of them are -inf; a row that sees no key has O = 0, lse = -inf whatever it holds."""
    import torch
    rng = np.random.default_rng(47)
    c, q, cu, lens, table, slots = build(mx, rng, fmt, 16, 2, 2, ql, kv)
    ones = torch.ones(sum(kv), 2, 128, dtype=torch.bfloat16, device="cuda")
    mx.kv_append(c, ones, bf16(rng, sum(kv), 2, 128).cuda(), torch.from_numpy(np.concatenate(slots)).cuda())
    q = q.contiguous()
    q[0, 0, 5] = -np.inf                                      # every score -inf
    q[0, 3, 7] = np.inf
    q[ql[0] + ql[1] - 1, 1, 9] = -np.inf                      # the last query of the second request
    q[ql[0] + ql[1] - 1, 2, 100] = np.nan
    if ql[1] > kv[1]:
        q[ql[0], :, 3] = -np.inf                              # sees no key
    o, lse = check(mx, c, q, cu, lens, table, slots, causal=True)
    assert torch.isnan(o[0, 0]).all() and torch.isnan(lse[0, 0]) and not torch.isnan(o[0, 1]).any()
    assert mx.device_status() == 0


def many_requests(rng, R, prompts, most, long):
    """Query and key lengths of R requests: decoding ones, idle ones, requests without keys, some prompts, one long context."""
    ql, kv = [1] * R, [int(k) for k in rng.integers(1, most, R)]
    for i in rng.permutation(R)[: R // 10]:
        ql[i] = 0
    for i in rng.permutation(R)[: R // 20]:
        kv[i] = 0
    for i in (0, R // 2, R - 1)[:prompts]:
        ql[i] = int(rng.integers(50, 90))
        kv[i] = ql[i] + int(rng.integers(0, 200))
    if long:
        ql[R - 2], kv[R - 2] = 1, long
    return ql, kv


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("R,prompts,most,long", [
    (127, 0, 60, 3000), (128, 0, 60, 3000), (129, 0, 60, 3000), (600, 0, 40, 1500), (1300, 0, 24, 2000),   # several turns of the scans
    (130, 2, 60, 3000), (513, 3, 30, 1500), (1300, 3, 20, 1100)])                                        # the same with prompts
def test_attention_many_requests(mx, fmt, R, prompts, most, long):
    import torch
    rng = np.random.default_rng(R + prompts)
    ql, kv = many_requests(rng, R, prompts, most, long)
    args = build(mx, rng, fmt, 16, 2, 2, ql, kv)
    assert mx.mxfa_kv_attn_workspace_size(R, max(ql), args[4].shape[1] * 16, 4, 2) > 0
    o, lse = check(mx, *args, causal=True)
    o2, lse2 = check(mx, *args, causal=True)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert mx.device_status() == 0


@pytest.mark.parametrize("R,H,G,q", [(1300, 8, 1, 1), (1000, 8, 3, 4)])
def test_attention_more_whole_items_than_ctas(mx, R, H, G, q):
    """Short contexts whose items are dealt out in more than one turn of the grid."""
    import torch
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert R * H > 16 * sms * (4 if G * q <= 8 else 3)
    rng = np.random.default_rng(R)
    ql, kv = many_requests(rng, R, 0, 40, 0)
    ql = [n * q for n in ql]
    args = build(mx, rng, 0, 16, H, G, ql, kv)
    assert mx.mxfa_kv_attn_workspace_size(R, q, args[4].shape[1] * 16, H * G, H) == 0
    check(mx, *args, causal=True)
    assert mx.device_status() == 0


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("R,page,width,spare,prompts", [(7, 16, 9, 40, 2), (33, 32, 5, 7, 4), (513, 16, 8, 90, 30)])
def test_plan_of_more_tokens_than_rows(mx, R, page, width, spare, prompts, inplace):
    """Tokens behind the last row of slots are planned all the same: blocks, lengths and counters are as with rows for all."""
    for seed, share in enumerate((0.0, 0.3, 0.9)):
        rng = np.random.default_rng(2000 * R + seed)
        ctx, new, table, ring, head, tail = random_step(rng, R, page, width, spare, prompts)
        tokens = int(np.maximum(new, 0).sum() * share)
        got, gt, gf = run_plan(mx, ctx, new, table, ring, head, tail, page, tokens, inplace)
        t, f = table.tolist(), ring.tolist()
        cu, kv, slots, pos, state = kv_ref.plan(ctx.tolist(), new.tolist(), t, f, head, tail, page, tokens)
        assert got == [cu, kv, slots[:tokens], pos[:tokens], state]
        np.testing.assert_array_equal(gt, t)
        np.testing.assert_array_equal(gf, f)
        assert mx.device_status() == 0


def test_attention_of_unserved_requests(mx):
    """A request without blocks keeps its length and gets no slots; its rows read the stored keys alone, and no other request's change."""
    import torch
    rng = np.random.default_rng(53)
    c, q, cu, lens, table, slots = build(mx, rng, 0, 16, 2, 2, [0, 0, 0], [16, 40, 32], extra=0, pad_rows=9)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    ring, state = torch.full((c.k.shape[0],), -7, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int64, device="cuda")
    s = mx.kv_plan(lens, i32(3, 4, 2), table, ring, state, 16, 9)
    assert s.ring_state.tolist() == [0, 0, 2] and s.kv_lens.tolist() == [16, 44, 32] and s.cu_q.tolist() == [0, 3, 7, 9]
    at = int(table[1, 2]) * 16 + 8
    assert s.slots.tolist() == [-1] * 3 + list(range(at, at + 4)) + [-1] * 2 and s.positions.tolist() == [16, 17, 18, 40, 41, 42, 43, 32, 33]
    k = bf16(rng, 9, 2, 128).cuda()
    mx.kv_append(c, k, k, s.slots)
    check(mx, c, q, s.cu_q, s.kv_lens, table, [slots[0], np.concatenate([slots[1], np.arange(at, at + 4)]), slots[2]], causal=True)
    assert mx.device_status() == 0
