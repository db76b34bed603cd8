"""4-bit cache without a GPU: the reference forms on hand-worked values, and the
refusals of the C ABI and of the Python layer (all before any launch)."""
import ctypes

import numpy as np
import pytest
import torch

from tests import kv_ref


@pytest.fixture(scope="module")
def mx():
    from mxfp8_block_scaled_fa_gb300 import build, mxfa
    build.build()
    mxfa.lib()
    return mxfa


def test_reference_quantization_by_hand():
    x = np.zeros((1, 128))
    x[0, :8] = [6.0, -5.0, 2.5, 0.25, 0.75, -7.9, 3.5, 1.75]   # amax 7.9: X = 0
    codes, sf, val = kv_ref.quantize(x, 0)
    assert sf[0].tolist() == [127, 104, 104, 104]              # a zero block takes the least scale
    assert val[0, :8].tolist() == [6.0, -4.0, 2.0, 0.0, 1.0, -6.0, 4.0, 2.0]
    assert codes[0, :4].tolist() == [0xE7, 0x04, 0xF2, 0x46]
    x[0, 32] = 2.0 ** 20                                       # above 6 * 2^13: saturates
    x[0, 64] = 2.0 ** -30                                      # below 2^-25: vanishes
    x[0, 96] = np.nan
    codes, sf, val = kv_ref.quantize(x, 0)
    assert sf[0].tolist() == [127, 140, 104, 255]
    assert val[0, 32] == 49152.0 and val[0, 64] == 0.0 and np.isnan(val[0, 96:]).all()
    y = np.zeros((1, 128))
    y[0, :3] = [12.0, 1.0, -0.5]                               # NVFP4, st = 1: scale 2
    codes, sf, val = kv_ref.quantize(y, 1, 1.0)
    assert sf[0, 0] == 0x40 and val[0, :3].tolist() == [12.0, 1.0, 0.0]   # -0.5 / 2 ties to 0
    np.testing.assert_array_equal(kv_ref.dequantize(codes, sf, 1, 1.0), val)


def test_reference_plan_by_hand():
    table = [[5, -1], [-1, -1], [7, 8]]
    ring = [0, 1, 2, 3, 4, 6, 9, 9, 9, 9]
    got = kv_ref.plan([16, 0, 17], [1, 17, -1], table, ring, 3, 6, 16, 20)
    assert got == ([0, 1, 18, 18], [17, 17, 0], [48] + list(range(64, 80)) + [96, -1, -1],
                   [16] + list(range(17)) + [-1, -1], [6, 8, 0])
    assert table[0] == [5, 3] and table[1] == [4, 6] and ring[6:8] == [7, 8]


def _cache(mx, **kw):
    d = dict(k=0x1000, v=0x2000, k_sf=0x3000, v_sf=0x4000, k_scale=0x5000, v_scale=0x6000, num_blocks=4,
             page=16, H=2, D=128, fmt=0)
    d.update(kw)
    return mx.KvPages(*[d[n] for n, _ in mx.KvPages._fields_])


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), 1), (dict(v_sf=None), 1), (dict(fmt=2), 1), (dict(num_blocks=0), 1), (dict(H=0), 1), (dict(page=0), 1),
    (dict(fmt=1, k_scale=None), 1), (dict(D=64), 2), (dict(page=48), 2), (dict(page=8), 2), (dict(page=256), 2),
    (dict(num_blocks=1 << 31), 2), (dict(k=0x1008), 3), (dict(k_sf=0x3004), 3), (dict(fmt=1, v_scale=0x6002), 3)])
def test_cache_checks(mx, kw, status):
    L, c = mx.lib(), _cache(mx, **kw)
    ref = ctypes.byref(c)
    assert L.mxfa_kv_append(ref, 0x10, 0x10, 256, 256, 3, 0x10, None) == status
    assert L.mxfa_kv_load(ref, 0x10, 3, 0x10, 0x10, None) == status
    assert L.mxfa_kv_attn(ref, 0x10, 512, 3, 0x10, 0x10, 1, 0x10, 4, 3, 4, 0.1, 1, 0x10, 0x10, 0x10, 1 << 30, None) == status


def test_row_call_checks(mx):
    L, ref = mx.lib(), ctypes.byref(_cache(mx))
    f = L.mxfa_kv_append
    assert f(ref, None, 0x10, 256, 256, 3, 0x10, None) == 1
    assert f(ref, 0x10, 0x10, 256, 256, 3, None, None) == 1
    assert f(ref, 0x10, 0x10, 256, 256, -1, 0x10, None) == 1
    assert f(ref, 0x10, 0x10, 248, 256, 3, 0x10, None) == 1           # tokens overlap
    assert f(ref, 0x10, 0x10, 260, 256, 3, 0x10, None) == 3           # stride not a multiple of 8
    assert f(ref, 0x18, 0x10, 256, 256, 3, 0x10, None) == 3
    assert f(ref, 0x10, 0x10, 256, 256, 3, 0x14, None) == 3
    assert f(ref, 0x10, 0x10, 256, 256, 1 << 30, 0x10, None) == 2
    assert f(ref, 0x10, 0x10, 256, 256, 0, 0x10, None) == 0           # nothing to do
    g = L.mxfa_kv_load
    assert g(ref, None, 3, 0x10, 0x10, None) == 1
    assert g(ref, 0x10, 3, None, 0x10, None) == 1
    assert g(ref, 0x10, 3, 0x10, 0x18, None) == 3
    assert g(ref, 0x10, 1 << 30, 0x10, 0x10, None) == 2
    assert g(ref, 0x10, 0, 0x10, 0x10, None) == 0


def test_attention_checks(mx):
    L, ref = mx.lib(), ctypes.byref(_cache(mx))
    base = dict(q=0x10, qs=512, T=3, cu=0x10, kv=0x10, R=1, bt=0x10, nb=64, mq=3, Hq=4, s=0.1, c=1, o=0x10, lse=0x10, ws=0x10,
                wb=1 << 30)

    def call(**kw):
        d = dict(base, **kw)
        return L.mxfa_kv_attn(ref, *d.values(), None)
    for n in ("q", "cu", "kv", "bt", "o", "lse"):
        assert call(**{n: None}) == 1, n
    assert call(Hq=3) == 1 and call(Hq=0) == 1 and call(nb=0) == 1 and call(R=-1) == 1 and call(mq=-1) == 1
    assert call(s=0.0) == 1 and call(s=float("nan")) == 1 and call(s=float("inf")) == 1
    assert call(qs=504) == 1 and call(qs=516) == 3
    assert call(q=0x18) == 3 and call(o=0x18) == 3 and call(ws=0x18) == 3 and call(cu=0x12) == 3
    assert call(T=1 << 31) == 2 and call(nb=1 << 27) == 2 and call(R=1 << 21) == 2
    assert call(T=0) == 0 and call(R=0) == 0 and call(mq=0) == 0


def test_plan_checks(mx):
    L = mx.lib()
    base = dict(ctx=0x1000, new=0x2000, R=8, bt=0x3000, nb=4, ring=0x4000, rs=64, ri=0x5000, ro=0x6000, page=16, T=32,
                cu=0x7000, kv=0x8000, slots=0x9000, pos=0xA000)

    def call(**kw):
        return L.mxfa_kv_plan(*dict(base, **kw).values(), None)
    for n in ("ctx", "new", "bt", "ring", "ri", "ro", "cu", "kv", "slots", "pos"):
        assert call(**{n: None}) == 1, n
    assert call(R=-1) == 1 and call(nb=0) == 1 and call(rs=0) == 1 and call(T=-1) == 1
    assert call(page=24) == 2 and call(R=16385) == 2 and call(T=1 << 31) == 2 and call(nb=1 << 27) == 2 and call(rs=1 << 31) == 2
    assert call(ctx=0x1002) == 3 and call(slots=0x9004) == 3 and call(ri=0x5004) == 3
    assert call(kv=0x1004) == 1 and call(ro=0x5008) == 1      # partly over their inputs
    assert call(kv=0x2000) == 1                               # over the new lengths


def test_python_refusals(mx):
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)
    good = lambda **kw: mx.KvCache(**{**dict(k=u8(3, 2, 16, 64), v=u8(3, 2, 16, 64), k_sf=u8(3, 2, 16, 4), v_sf=u8(3, 2, 16, 4), fmt=0), **kw})
    with pytest.raises(ValueError):
        good(fmt=3)
    with pytest.raises(ValueError):
        good(v=u8(3, 2, 16, 32))
    with pytest.raises(ValueError):
        good(k=u8(3, 2, 64))
    with pytest.raises(ValueError):
        good(k_sf=u8(3, 2, 16, 8))
    with pytest.raises(ValueError):
        good(fmt=1, k_sf=u8(3, 2, 16, 8), v_sf=u8(3, 2, 16, 8))           # no tensor scales
    with pytest.raises(TypeError):
        good(k=u8(3, 2, 16, 64).int())
    with pytest.raises(ValueError):
        good(k=u8(3, 2, 64, 16).transpose(2, 3))                          # not contiguous
    c = good()
    rows = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    slots = torch.zeros(5, dtype=torch.int64)
    with pytest.raises(ValueError):
        mx.kv_append(c, rows(5, 3, 128), rows(5, 3, 128), slots)          # heads
    with pytest.raises(TypeError):
        mx.kv_append(c, rows(5, 2, 128).float(), rows(5, 2, 128), slots)
    with pytest.raises(ValueError):
        mx.kv_append(c, rows(5, 2, 128), rows(4, 2, 128), slots)
    with pytest.raises(TypeError):
        mx.kv_append(c, rows(5, 2, 128), rows(5, 2, 128), slots.int())
    with pytest.raises(ValueError):
        mx.kv_append(c, rows(5, 128, 2).transpose(1, 2), rows(5, 2, 128), slots)
    with pytest.raises(ValueError):
        mx.kv_append(c, rows(5, 2, 128), rows(5, 2, 128), slots)          # not on a GPU
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    with pytest.raises(ValueError):
        mx.kv_attention(rows(5, 3, 128), c, i32(2), i32(1), i32(1, 4), 5, 0.1)
    with pytest.raises(ValueError):
        mx.kv_attention(rows(5, 4, 128), c, i32(3), i32(1), i32(1, 4), 5, 0.1)
    with pytest.raises(TypeError):
        mx.kv_attention(rows(5, 4, 128), c, i32(2).long(), i32(1), i32(1, 4), 5, 0.1)
    with pytest.raises(ValueError):
        mx.kv_plan(i32(3), i32(2), i32(3, 4), i32(8), torch.zeros(3, dtype=torch.int64), 16, 4)
    with pytest.raises(ValueError):
        mx.kv_plan(i32(3), i32(3), i32(3, 4), i32(8), torch.zeros(3, dtype=torch.int64), 16, 4)   # not on a GPU


def test_copy_has_its_own_addresses(mx):
    import copy
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)
    c = mx.KvCache(u8(3, 2, 16, 64), u8(3, 2, 16, 64), u8(3, 2, 16, 4), u8(3, 2, 16, 4), 0)
    d = copy.deepcopy(c)
    assert d.pages.k == d.k.data_ptr() != c.k.data_ptr() == c.pages.k and d.pages.v_sf == d.v_sf.data_ptr()
    assert copy.copy(c).pages.k == c.k.data_ptr()


def test_sizes(mx):
    L = mx.lib()
    assert L.mxfa_kv_codes_bytes(10, 16, 3) == 10 * 16 * 3 * 64
    assert L.mxfa_kv_sf_bytes(10, 16, 3, 0) == 10 * 16 * 3 * 4 and L.mxfa_kv_sf_bytes(10, 16, 3, 1) == 10 * 16 * 3 * 8
    assert L.mxfa_kv_codes_bytes(-1, 16, 3) == 0 and L.mxfa_kv_attn_workspace_size(1, 1, 100, 5, 2) == 0


def test_overlapping_buffers(mx):
    L, ref = mx.lib(), ctypes.byref(_cache(mx))
    # a plan: R = 8 requests of 4 pages, 64 ring entries, 32 tokens
    base = dict(ctx=0x1000, new=0x2000, R=8, bt=0x3000, nb=4, ring=0x4000, rs=64, ri=0x5000, ro=0x6000, page=16, T=32,
                cu=0x7000, kv=0x8000, slots=0x9000, pos=0xA000)
    size = dict(ctx=32, new=32, bt=128, ring=256, ri=24, ro=24, cu=36, kv=32, slots=256, pos=128)
    for w in ("bt", "ring", "ro", "cu", "kv", "slots", "pos"):
        for o in size:
            if o == w or (w, o) in (("kv", "ctx"), ("ro", "ri")):
                continue
            for at in (base[o], base[o] + (size[o] - 1) // 8 * 8):             # at its beginning and over its end
                assert L.mxfa_kv_plan(*dict(base, **{w: at}).values(), None) == 1, (w, o)
    # a load of 3 tokens: 3 * 512 bytes of k and of v, 24 of slots
    for slots, k, v in ((0x100, 0x1000, 0x1000), (0x100, 0x1000, 0x1500), (0x1000, 0x1000, 0x2000), (0x2100, 0x1000, 0x2000)):
        assert L.mxfa_kv_load(ref, slots, 3, k, v, None) == 1
    # attention of 3 tokens: q rows of 1024 bytes 2048 apart, o of 1024, lse 48 bytes
    base = dict(q=0x10000, qs=1024, T=3, cu=0x20000, kv=0x30000, R=1, bt=0x40000, nb=64, mq=3, Hq=4, s=0.1, c=1, o=0x50000,
                lse=0x60000, ws=0x10000000, wb=1 << 30)
    bad = [dict(o=0x10000), dict(o=0x10000 + 2 * 2048), dict(o=0x10400), dict(o=0x20000 - 16), dict(o=0x40000), dict(lse=0x50000),
           dict(lse=0x30000), dict(lse=0x10000 + 2 * 2048 + 1020)]
    if L.mxfa_kv_attn_workspace_size(1, 3, 1024, 4, 2):
        bad += [dict(ws=0x50000), dict(ws=0x10000)]
    for kw in bad:
        assert L.mxfa_kv_attn(ref, *dict(base, **kw).values(), None) == 1, kw


def test_attention_context_limits(mx):
    L, ref = mx.lib(), ctypes.byref(_cache(mx, page=128))
    call = lambda nb, mq: L.mxfa_kv_attn(ref, 0x10000, 512, 200, 0x20000, 0x30000, 1, 0x40000, nb, mq, 4, 0.1, 1, 0x50000, 0x90000, None, 0, None)
    # no workspace is given: 1 or 6 (too small) where the sizes are accepted
    assert call(1 << 24, 200) == 2 and call((1 << 18) + 1, 25) == 2             # more than 2^25 keys for more than 48 rows
    assert call(1 << 18, 25) != 2 and call(1 << 23, 24) != 2 and call((1 << 23) + 1, 24) == 2


def test_join_headers_have_one_writer():
    """Nothing orders two warps' stores of a join header after the launch's only barrier: each store of one
    kernel stands under the same test of the thread."""
    import os
    import re
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mxfp8_block_scaled_fa_gb300", "csrc")
    for name in ("kv_attn.cu", "kv_prefill.cu"):
        lines = open(os.path.join(csrc, name)).read().splitlines()
        writers = []
        for i, line in enumerate(lines):
            if re.search(r"headers\[blockIdx\.x\](\.parts)?\s*=[^=]", line):
                test = next(x for x in reversed(lines[: i + 1]) if re.search(r"\bif \(.*\b(tid|lane) == \d", x))
                writers.append(" ".join(sorted(re.findall(r"\b(?:tid|warp|lane) == \d+", test))))
        assert len(writers) == 2 and len(set(writers)) == 1, (name, writers)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("n,h,page", [(3, 0, 16), (0, 2, 16), (3, 2, 0), (0, 0, 0)])
def test_empty_cache_refused(mx, fmt, n, h, page):
    u8, one = (lambda *s: torch.zeros(s, dtype=torch.uint8)), torch.ones(1)
    sf = 4 if fmt == 0 else 8
    with pytest.raises(ValueError):
        mx.KvCache(u8(n, h, page, 64), u8(n, h, page, 64), u8(n, h, page, sf), u8(n, h, page, sf), fmt, one, one)
    with pytest.raises(ValueError):
        mx.KvCache.empty(n, h, page, fmt, device="cpu")


# a cache of 4 blocks, 2 heads, pages of 16: 8192 bytes each of codes, 1024 of NVFP4's scales
_FAR = dict(k=0x100000, v=0x110000, k_sf=0x120000, v_sf=0x130000, k_scale=0x140000, v_scale=0x150000, fmt=1)
_FAR_BYTES = dict(k=8192, v=8192, k_sf=1024, v_sf=1024, k_scale=4, v_scale=4)


@pytest.mark.parametrize("part", list(_FAR_BYTES))
def test_results_over_the_cache_refused(mx, part):
    L, ref = mx.lib(), ctypes.byref(_cache(mx, **_FAR))
    at, size = _FAR[part], _FAR_BYTES[part]
    last = at + (size - 1) // 16 * 16
    # a load of 3 tokens writes 1536 bytes each of k and v: over the beginning and over the end
    for x in (at, at - 1536 + 16, last):
        assert L.mxfa_kv_load(ref, 0x1000, 3, x, 0x20000, None) == 1
        assert L.mxfa_kv_load(ref, 0x1000, 3, 0x20000, x, None) == 1
    # attention of 5 tokens and 4 heads: o of 5120 bytes, lse of 80
    base = dict(q=0x10000, qs=1024, T=5, cu=0x20000, kv=0x30000, R=1, bt=0x40000, nb=128, mq=3, Hq=4, s=0.1, c=1, o=0x50000,
                lse=0x60000, ws=0x10000000, wb=1 << 30)
    bad = [dict(o=at), dict(o=at - 5120 + 16), dict(o=last), dict(lse=at), dict(lse=at - 76), dict(lse=last)]
    if L.mxfa_kv_attn_workspace_size(1, 3, 128 * 16, 4, 2):
        bad += [dict(ws=at), dict(ws=last), dict(ws=at - 16)]
    for kw in bad:
        assert L.mxfa_kv_attn(ref, *dict(base, **kw).values(), None) == 1, kw


@pytest.mark.parametrize("part", list(_FAR_BYTES))
def test_store_over_its_inputs_refused(mx, part):
    L, ref = mx.lib(), ctypes.byref(_cache(mx, **_FAR))
    at, size = _FAR[part], _FAR_BYTES[part]
    last = at + (size - 1) // 16 * 16
    good = dict(k=0x10000, v=0x20000, ks=256, vs=512, T=3, slots=0x30000)
    # 3 rows of 512 bytes: k's one after another, v's 1024 bytes apart; 24 bytes of slots
    bad = [dict(k=at), dict(k=last), dict(k=at - 1536 + 16), dict(v=at), dict(v=last), dict(v=at - 2560 + 16), dict(slots=at),
           dict(slots=last), dict(slots=at - 16)]
    for kw in bad if size > 4 else []:
        assert L.mxfa_kv_append(ref, *dict(good, **kw).values(), None) == 1, kw
    # its own buffers over one another: the rows are written, and NVFP4's scales read, by every CTA
    for other in ("k", "v", "k_sf", "v_sf"):
        if other == part:
            continue
        c = _cache(mx, **{**_FAR, part: _FAR[other] + _FAR_BYTES[other] // 2})
        assert L.mxfa_kv_append(ctypes.byref(c), *good.values(), None) == 1, other


def test_a_caches_tensors_stay(mx):
    """Calls go by the addresses of the tensors a cache was made with, so those cannot be exchanged."""
    import copy
    import dataclasses
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)
    c = mx.KvCache(u8(3, 2, 16, 64), u8(3, 2, 16, 64), u8(3, 2, 16, 8), u8(3, 2, 16, 8), 1, torch.ones(1), torch.ones(1))
    for name in ("k", "v", "k_sf", "v_sf", "fmt", "k_scale", "v_scale", "H", "page", "index", "raw", "pages"):
        value = getattr(c, name)
        with pytest.raises(AttributeError):
            setattr(c, name, value)
        with pytest.raises(AttributeError):
            delattr(c, name)
        assert getattr(c, name) is value
    c.note = 1                                                       # anything else is the owner's
    assert c.note == 1
    d = dataclasses.replace(c, k=u8(3, 2, 16, 64))
    assert d.pages.k == d.k.data_ptr() != c.pages.k and d.v is c.v
    for e in (d, copy.copy(c)):
        with pytest.raises(AttributeError):
            e.k = u8(3, 2, 16, 64)
    assert mx.KvCache(u8(3, 2, 16, 64), u8(3, 2, 16, 64), u8(3, 2, 16, 4), u8(3, 2, 16, 4), 0, torch.ones(1)).k_scale is None
