"""Rotary positions, windowed and shared-prefix attention and shared pages without a GPU: the
reference forms on hand-worked values, and the refusals of the C ABI and of the Python layer (all
before any launch)."""
import ctypes
import math

import numpy as np
import pytest
import torch

from tests import kv_ref, more_ref


@pytest.fixture(scope="module")
def mx():
    from mxfp8_block_scaled_fa_gb300 import build, mxfa
    build.build()
    mxfa.lib()
    return mxfa


# ------------------------------------------------------------------------- reference forms
def test_reference_rotation_by_hand():
    x = np.arange(128.0).reshape(1, 1, 128)
    quarter = np.full((1, 8), math.pi / 2)
    y, size = more_ref.rotate(x, quarter, 16, False)
    np.testing.assert_allclose(y[0, 0, :18], [-8, -9, -10, -11, -12, -13, -14, -15, 0, 1, 2, 3, 4, 5, 6, 7, 16, 17], atol=1e-12)
    assert size[0, 0, 3] == 3 + 11 and size[0, 0, 16] == 0
    y, _ = more_ref.rotate(x, quarter, 16, True, 2.0)
    np.testing.assert_allclose(y[0, 0, :4], [-2, 0, -6, 4], atol=1e-12)
    # angles: a quarter turn a position, and a far one that only whole numbers keep
    np.testing.assert_allclose(more_ref.angles([1 << 62], [0, 1, 2, 5]), [[0], [math.pi / 2], [math.pi], [math.pi / 2]])
    assert more_ref.angles([(1 << 64) - 1], [1 << 30])[0, 0] == pytest.approx(2 * math.pi * (1 - 2.0 ** -34), abs=1e-15)


@pytest.mark.parametrize("inter", [False, True])
def test_reference_gradient_by_differences(inter):
    rng = np.random.default_rng(5)
    x, dy = rng.standard_normal((2, 3, 2, 128))
    angle = rng.uniform(-9, 9, (3, 24))
    grad, _ = more_ref.rotate(dy, angle, 48, inter, 1.3, inverse=True)
    for at in [(0, 0, 0), (1, 1, 23), (2, 0, 47), (2, 1, 48), (1, 0, 24), (0, 1, 127)]:
        h = np.zeros_like(x)
        h[at] = 0.5
        up, down = (more_ref.rotate(z, angle, 48, inter, 1.3)[0] for z in (x + h, x - h))
        assert ((up - down) * dy).sum() == pytest.approx(grad[at], abs=1e-12)


def test_reference_masked_attention_is_attention():
    rng = np.random.default_rng(6)
    q, k, v = rng.standard_normal((3, 4, 128)), rng.standard_normal((7, 2, 128)), rng.standard_normal((7, 2, 128))
    for got, want in zip(more_ref.attention(q, k, v, 0.1, more_ref.window_mask(3, 7, 100, 0)), kv_ref.attention(q, k, v, 0.1, True)):
        np.testing.assert_allclose(got, want, atol=1e-12)
    np.testing.assert_array_equal(more_ref.window_mask(2, 6, 2, 1), [[1, 0, 0, 1, 1, 0], [1, 0, 0, 0, 1, 1]])
    assert not more_ref.window_mask(3, 2, 5, 1)[0].any()


def test_reference_pages_by_hand():
    table = [[4, 7, 2], [-1, 5, 5], [-1, -1, -1]]
    refs, ring = [0] * 9, [0, 1, 3, 6, 8, -7, -7, -7, -7]
    got = more_ref.fork(table, [0, 0], [1, 2], [32, 41], refs, ring, 2, 5, 16)
    assert got == ([-1, 2], [-1, 3], [32, 41], [3, 5, 0])
    assert table == [[4, 7, 2], [4, 7, 5], [4, 7, 3]] and refs == [0, 0, 0, 0, 2, 0, 0, 2, 0]
    assert more_ref.free(table, [0, 2], [0, 1], [3, 3], refs, ring, 3, 5, 8) == [3, 7, 8]
    assert refs == [0, 0, 0, 0, 1, 0, 0, 0, 0] and ring[5:7] == [2, 3]
    assert more_ref.fork(table, [1], [2], [17], refs, ring, 5, 5, 16) == ([-1], [-1], [16], [5, 5, 1])
    assert table[2][1] == -1


# --------------------------------------------------------------------------- frequencies
def test_frequencies(mx):
    f = lambda rp: [(int(t) % 2 ** 64) / 2 ** 64 * 2 * math.pi for t in rp.turns]
    plain = [10000.0 ** (-2 * i / 64) for i in range(32)]
    np.testing.assert_allclose(f(mx.Rope.make(64, device="cpu")), plain, rtol=1e-12)
    np.testing.assert_allclose(f(mx.Rope.make(64, scaling="linear", factor=4.0, device="cpu")), np.array(plain) / 4, rtol=1e-12)
    ntk = f(mx.Rope.make(64, scaling="ntk", factor=4.0, device="cpu"))
    assert ntk[0] == pytest.approx(1.0) and ntk[-1] == pytest.approx(plain[-1] / 4)
    rp = mx.Rope.make(64, scaling="yarn", factor=4.0, original=2048, interleaved=True, device="cpu")
    yarn = np.array(f(rp)) / plain
    turns = 2048 * np.array(plain) / (2 * math.pi)
    np.testing.assert_allclose(yarn[turns >= 32], 1.0)
    np.testing.assert_allclose(yarn[turns <= 1], 0.25)
    assert (np.diff(yarn) <= 1e-12).all() and rp.gain == pytest.approx(0.1 * math.log(4) + 1) and rp.interleaved
    # a frequency above a turn a position, and one that does not turn
    got = mx.Rope.from_freqs([2 * math.pi * 0.75, 0.0, -1.0] + [0.0] * 5, device="cpu").turns
    assert int(got[0]) == pytest.approx(-2.0 ** 62, rel=1e-15) and int(got[1]) == 0
    assert int(got[2]) == -int(mx.Rope.make(16, device="cpu").turns[0])
    for bad in (dict(rot=24), dict(rot=144), dict(rot=0), dict(base=1.0), dict(factor=0.5), dict(scaling="other"), dict(original=0)):
        with pytest.raises(ValueError):
            mx.Rope.make(**dict(dict(device="cpu"), **bad))


def test_positions_of_sequences(mx):
    assert mx.rope_positions(mx.Seqs.dense(2, 3), "cpu").tolist() == [0, 1, 2, 0, 1, 2]
    s = mx.Seqs.varlen([2, 0, 3], "cpu")
    p = mx.rope_positions(s, "cpu")
    assert p.tolist() == [0, 1, 0, 1, 2] and p.dtype is torch.int32


# ------------------------------------------------------------------------------- refusals
def _cache(mx, **kw):
    d = dict(k=0x100000, v=0x110000, k_sf=0x120000, v_sf=0x130000, k_scale=0x140000, v_scale=0x150000, num_blocks=4, page=16,
             H=2, D=128, fmt=0)
    d.update(kw)
    return mx.KvPages(*[d[n] for n, _ in mx.KvPages._fields_])


def _rot(mx, **kw):
    d = dict(turns=0x1000, rot=128, layout=0, gain=1.0)
    d.update(kw)
    return mx.Rotation(*[d[n] for n, _ in mx.Rotation._fields_])


BAD_ROTATIONS = [(dict(turns=None), 1), (dict(rot=0), 1), (dict(rot=256), 1), (dict(layout=2), 1), (dict(gain=float("nan")), 1),
                 (dict(gain=float("inf")), 1), (dict(gain=1e39), 1), (dict(rot=24), 2), (dict(turns=0x1004), 3)]


def test_rope_checks(mx):
    L = mx.lib()
    base = dict(x=0x10000, xs=256, y=0x20000, ys=256, pos=0x2000, T=3, H=2, D=128)

    def call(rot=None, **kw):
        return L.mxfa_rope(*dict(base, **kw).values(), ctypes.byref(rot if rot is not None else _rot(mx)), 0, None)
    for kw, status in BAD_ROTATIONS:
        assert call(_rot(mx, **kw)) == status, kw
    assert L.mxfa_rope(*base.values(), None, 0, None) == 1
    for n in ("x", "y", "pos"):
        assert call(**{n: None}) == 1
    assert call(T=-1) == 1 and call(H=0) == 1 and call(xs=248) == 1 and call(ys=128) == 1
    assert call(D=64) == 2 and call(H=65537, xs=1 << 30, ys=1 << 30) == 2 and call(T=1 << 31) == 2 and call(T=1 << 30) == 2
    assert call(x=0x10008) == 3 and call(y=0x20004) == 3 and call(pos=0x2002) == 3 and call(xs=260) == 3 and call(ys=260) == 3
    # x: 3 rows of 512 bytes; partly in place, in place with another stride, over positions and turns
    for kw in (dict(y=0x10000 + 512), dict(y=0x10000 - 16), dict(y=0x10000, ys=512), dict(y=0x2000), dict(y=0x1000 + 496),
               dict(pos=0x20000 + 3 * 512 - 4)):
        assert call(**kw) == 1, kw
    assert call(T=0) == 0


def test_append_rope_checks(mx):
    L, ref = mx.lib(), ctypes.byref(_cache(mx))
    base = dict(q=0x10000, qs=512, Hq=4, k=0x20000, ks=256, v=0x30000, vs=256, T=3, pos=0x2000, slots=0x3000)
    last = dict(out=0x40000, outs=512)

    def call(rot=None, cache=ref, **kw):
        d = dict(base, **{k: v for k, v in kw.items() if k in base})
        e = dict(last, **{k: v for k, v in kw.items() if k in last})
        return L.mxfa_kv_append_rope(cache, *d.values(), ctypes.byref(rot if rot is not None else _rot(mx)), *e.values(), None)
    for kw, status in BAD_ROTATIONS:
        assert call(_rot(mx, **kw)) == status, kw
    for kw, status in ((dict(k=None), 1), (dict(page=48), 2), (dict(v=0x110008), 3)):
        assert call(cache=ctypes.byref(_cache(mx, **kw))) == status, kw
    for n in ("q", "k", "v", "pos", "slots", "out"):
        assert call(**{n: None}) == 1, n
    assert call(T=-1) == 1 and call(Hq=0) == 1 and call(qs=504) == 1 and call(outs=256) == 1 and call(ks=248) == 1 and call(vs=8) == 1
    assert call(T=1 << 29) == 2 and call(Hq=65537, qs=1 << 30, outs=1 << 30) == 2
    for n in ("q", "k", "v", "out", "slots"):
        assert call(**{n: {**base, **last}[n] + 4}) == 3, n
    assert call(pos=0x2002) == 3 and call(qs=516) == 3 and call(ks=260) == 3 and call(vs=260) == 3 and call(outs=516) == 3
    for kw in (dict(out=0x10000 + 16), dict(out=0x10000, outs=1024), dict(out=0x20000), dict(out=0x30000 + 1024), dict(out=0x2000),
               dict(out=0x3000), dict(out=0x1000), dict(out=0x100000), dict(out=0x130000), dict(k=0x100000), dict(v=0x120000),
               dict(q=0x110000 + 8176), dict(slots=0x120000), dict(pos=0x130000)):
        assert call(**kw) == 1, kw
    # q in place within a projection whose rows hold q, k, v: k inside q's heads is refused
    inside = dict(q=0x10000, out=0x10000, qs=1024, outs=1024, ks=1024, vs=1024)
    assert call(**inside, k=0x10000 + 512, v=0x10000 + 2048 - 512) == 1
    assert call(**inside, k=0x10000 + 1024, v=0x10000 + 2048 - 256) == 1
    assert call(T=0) == 0


def test_window_checks(mx):
    L, ref = mx.lib(), ctypes.byref(_cache(mx))
    base = dict(q=0x10000, qs=512, T=3, cu=0x20000, kv=0x30000, R=1, bt=0x40000, nb=64, mq=3, Hq=4, s=0.1, w=100, sk=4, o=0x50000,
                lse=0x60000, ws=0x10000000, wb=1 << 30)

    def call(**kw):
        return L.mxfa_kv_attn_window(ref, *dict(base, **kw).values(), None)
    for n in ("q", "cu", "kv", "bt", "o", "lse"):
        assert call(**{n: None}) == 1, n
    assert call(w=0) == 1 and call(w=-5) == 1 and call(sk=-1) == 1 and call(Hq=3) == 1 and call(s=0.0) == 1 and call(nb=0) == 1
    assert call(T=1 << 31) == 2 and call(nb=1 << 27) == 2 and call(o=0x50008) == 3 and call(qs=516) == 3
    for kw in (dict(o=0x10000), dict(lse=0x50000), dict(o=0x100000), dict(lse=0x130000)):
        assert call(**kw) == 1, kw
    assert call(T=0) == 0 and call(R=0) == 0 and call(mq=0) == 0
    size = L.mxfa_kv_attn_window_workspace_size
    assert size(1, 1, 100, 5, 2, 10, 0) == 0 and size(1, 1, 100, 4, 2, 0, 0) == 0
    # a window short enough needs no workspace however long the context; one as long as the context needs what it needs
    assert size(1, 1, 1 << 20, 4, 2, 500, 4) == 0
    assert size(3, 200, 4096, 4, 2, 1 << 30, 0) == L.mxfa_kv_attn_workspace_size(3, 200, 4096, 4, 2)


def test_shared_checks(mx):
    L, ref = mx.lib(), ctypes.byref(_cache(mx))
    base = dict(q=0x10000, qs=512, T=3, cu=0x20000, kv=0x30000, R=2, bt=0x40000, nb=64, mq=3, Hq=4, s=0.1, st=0x70000, pl=0x78000,
                g=1, mg=3, sh=0, o=0x50000, lse=0x60000, ws=0x10000000, wb=1 << 34)

    def call(**kw):
        return L.mxfa_kv_attn_shared(ref, *dict(base, **kw).values(), None)
    for n in ("q", "cu", "kv", "bt", "o", "lse", "st", "pl"):
        assert call(**{n: None}) == 1, n
    assert call(sh=3) == 1 and call(sh=-1) == 1
    assert call(g=-1) == 1 and call(mg=-1) == 1 and call(Hq=3) == 1 and call(ws=None) == 1 and call(wb=16) == 4
    assert call(g=1 << 21) == 2 and call(T=1 << 31) == 2 and call(st=0x70002) == 3 and call(pl=0x78002) == 3
    for kw in (dict(o=0x70000), dict(lse=0x78000), dict(ws=0x70000), dict(o=0x10000), dict(ws=0x50000), dict(lse=0x110000)):
        assert call(**kw) == 1, kw
    assert call(T=0) == 0 and call(R=0) == 0 and call(mq=0) == 0
    size = L.mxfa_kv_attn_shared_workspace_size
    assert size(2, 1, 3, 3, 3, 1024, 5, 2) == 0 and size(2, -1, 3, 3, 3, 1024, 4, 2) == 0
    assert size(2, 0, 3, 3, 3, 1024, 4, 2) == L.mxfa_kv_attn_workspace_size(2, 3, 1024, 4, 2)
    assert size(2, 1, 3, 3, 3, 1024, 4, 2) >= 3 * 4 * 520


def _page_calls(mx):
    L = mx.lib()
    fork = dict(bt=0x10000, R=4, w=8, src=0x2000, dst=0x2100, lens=0x2200, F=3, refs=0x3000, nb=16, ring=0x4000, rs=16, ri=0x5000,
                ro=0x5100, page=16, a=0x6000, b=0x6100, ln=0x6200)
    free = dict(bt=0x10000, R=4, w=8, rows=0x2000, first=0x2100, end=0x2200, F=3, refs=0x3000, nb=16, ring=0x4000, rs=16, ri=0x5000,
                ro=0x5100)
    return [(L.mxfa_kv_fork, fork), (L.mxfa_kv_free, free)]


@pytest.mark.parametrize("which", [0, 1])
def test_page_call_checks(mx, which):
    f, base = _page_calls(mx)[which]
    call = lambda **kw: f(*dict(base, **kw).values(), None)
    pointers = [n for n, v in base.items() if v >= 0x2000]
    for n in pointers:
        assert call(**{n: None}) == 1, n
        assert call(**{n: base[n] + (4 if n in ("ri", "ro") else 2)}) == 3, n
    for n in ("R", "w", "nb", "rs"):
        assert call(**{n: 0}) == 1 and call(**{n: -1}) == 1, n
    assert call(F=-1) == 1
    assert call(F=16385) == 2 and call(R=1 << 21) == 2 and call(nb=1 << 31) == 2 and call(rs=1 << 31) == 2 and call(R=1 << 10, w=1 << 21) == 2
    size = dict(bt=128, refs=64, ring=64, ri=24, ro=24, **{n: 12 for n in pointers if n not in ("bt", "refs", "ring", "ri", "ro")})
    written = ("bt", "refs", "ro", "a", "b", "ln") if which == 0 else ("refs", "ring", "ro")
    for w in written:
        for o in size:
            if o == w or (w, o) == ("ro", "ri"):
                continue
            for at in (base[o], base[o] + (size[o] - 1) // 8 * 8):
                assert call(**{w: at}) == 1, (w, o)
    assert call(ro=0x5008) == 1                                      # partly over its input
    if which == 0:
        assert call(page=24) == 2 and call(w=1 << 27, R=1) == 2
    else:
        assert call(w=(1 << 26) + 1, R=1) == 2
        assert call(rs=15) == 1                                      # fewer places than blocks


def test_copy_checks(mx):
    L, f = mx.lib(), mx.lib().mxfa_kv_copy_blocks
    ref = ctypes.byref(_cache(mx))
    assert f(ref, None, 0x2000, 3, None) == 1 and f(ref, 0x1000, None, 3, None) == 1 and f(ref, 0x1000, 0x2000, -1, None) == 1
    assert f(ref, 0x1002, 0x2000, 3, None) == 3 and f(ref, 0x1000, 0x2002, 3, None) == 3
    assert f(ref, 0x100000, 0x2000, 3, None) == 1 and f(ref, 0x1000, 0x130000, 3, None) == 1
    assert f(ref, 0x1000, 0x2000, 8193, None) == 2
    assert f(ctypes.byref(_cache(mx, D=64)), 0x1000, 0x2000, 3, None) == 2
    assert f(ctypes.byref(_cache(mx, v=0x100000)), 0x1000, 0x2000, 3, None) == 1
    assert f(ref, 0x1000, 0x2000, 0, None) == 0


def test_python_refusals(mx):
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)
    rows = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    i64 = lambda *s: torch.zeros(s, dtype=torch.int64)
    c = mx.KvCache(u8(3, 2, 16, 64), u8(3, 2, 16, 64), u8(3, 2, 16, 4), u8(3, 2, 16, 4), 0)
    rp = mx.Rope.make(device="cpu")
    for call in (mx.rope, mx.rope_bwd):
        with pytest.raises(ValueError):
            call(rows(5, 256), rp, i32(5))
        with pytest.raises((ValueError, TypeError)):
            call(rows(5, 2, 128).float(), rp, i32(5))
        with pytest.raises(ValueError):
            call(rows(5, 2, 128), rp, i32(5))                        # not on a GPU
    with pytest.raises(ValueError):
        mx.kv_append_rope(c, rows(5, 4, 128), rows(4, 2, 128), rows(5, 2, 128), rp, i32(5), i64(5))
    with pytest.raises(ValueError):
        mx.kv_append_rope(c, rows(5, 512), rows(5, 2, 128), rows(5, 2, 128), rp, i32(5), i64(5))
    with pytest.raises(TypeError):
        mx.kv_append_rope(c, rows(5, 4, 128), rows(5, 2, 128), rows(5, 2, 128), rp, i64(5), i64(5))
    with pytest.raises(TypeError):
        mx.kv_append_rope(c, rows(5, 4, 128), rows(5, 2, 128), rows(5, 2, 128), rp, i32(5), i32(5))
    with pytest.raises(ValueError):
        mx.kv_append_rope(c, rows(5, 4, 128), rows(5, 2, 128), rows(5, 2, 128), rp, i32(4), i64(5))
    attn = (rows(5, 4, 128), c, i32(2), i32(1), i32(1, 4))
    with pytest.raises(ValueError):
        mx.kv_attention(*attn, 5, 0.1, sinks=4)                      # without a window
    with pytest.raises(ValueError):
        mx.kv_attention(*attn, 5, 0.1, causal=False, window=4)
    for kw in (dict(window=0), dict(window=-3), dict(window=1 << 31), dict(window=(1 << 32) + 5), dict(window=4, sinks=-1),
               dict(window=4, sinks=(1 << 32) + 1)):
        with pytest.raises(ValueError):
            mx.kv_attention(*attn, 5, 0.1, **kw)
    with pytest.raises(ValueError):
        mx.kv_attention_shared(*attn, i32(2), i32(1), 5, (1 << 32) + 5, 0.1)
    with pytest.raises(ValueError):
        mx.kv_attention(*attn, 5, 0.1, window=4)                     # not on a GPU
    with pytest.raises(ValueError):
        mx.kv_attention_shared(*attn, i32(2), i32(2), 5, 5, 0.1)
    with pytest.raises(TypeError):
        mx.kv_attention_shared(*attn, i64(2), i32(1), 5, 5, 0.1)
    with pytest.raises(ValueError):
        mx.kv_attention_shared(*attn, i32(2), i32(1), 5, 5, 0.1)     # not on a GPU
    with pytest.raises(ValueError):
        mx.kv_fork(i32(3, 4), i32(2), i32(1), i32(2), i32(9), i32(9), i64(3), 16)
    with pytest.raises(TypeError):
        mx.kv_fork(i32(3, 4), i32(2), i64(2), i32(2), i32(9), i32(9), i64(3), 16)
    with pytest.raises(ValueError):
        mx.kv_fork(i32(3, 4), i32(2), i32(2), i32(2), i32(9), i32(9), i64(2), 16)
    with pytest.raises(ValueError):
        mx.kv_free(i32(12), i32(2), i32(2), i32(2), i32(9), i32(9), i64(3))
    with pytest.raises(ValueError):
        mx.kv_free(i32(3, 4), i32(2), i32(2), i32(2), i32(9), i32(9), i64(3))   # not on a GPU
    with pytest.raises(ValueError):
        mx.kv_copy_blocks(c, i32(2), i32(3))
    with pytest.raises(ValueError):
        mx.kv_copy_blocks(c, i32(2), i32(2))                         # not on a GPU
