"""Refusals of the 4-bit cache's calls for pages and shared prefixes, without a GPU (all before any launch)."""
import ctypes

import pytest
import torch

from tests.test_more_kv_checks import _cache, mx  # noqa: F401


def test_fork_gap_checks(mx):
    f = mx.lib().mxfa_kv_fork_gap
    base = dict(bt=0x10000, R=4, w=8, src=0x2000, dst=0x2100, lens=0x2200, g0=0x2300, g1=0x2400, F=3, refs=0x3000, nb=16, ring=0x4000,
                rs=16, ri=0x5000, ro=0x5100, page=16, a=0x6000, b=0x6100, ln=0x6200)
    call = lambda **kw: f(*dict(base, **kw).values(), None)
    for n in ("bt", "src", "dst", "lens", "g0", "g1", "refs", "ring", "ri", "ro", "a", "b", "ln"):
        assert call(**{n: None}) == 1, n
        assert call(**{n: base[n] + (4 if n in ("ri", "ro") else 2)}) == 3, n
    assert call(F=-1) == 1 and call(F=16385) == 2 and call(page=24) == 2 and call(w=1 << 27, R=1) == 2
    for w in ("bt", "refs", "ro", "a", "b", "ln"):           # written over a list that is read
        for o in ("g0", "g1", "lens"):
            for at in (base[o], base[o] + 8):
                assert call(**{w: at}) == 1, (w, o)
    assert call(ro=0x5008) == 1 and call(a=0x6200) == 1


def test_fork_gap_refusals(mx):
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    args = (i32(3, 4), i32(2), i32(2), i32(2), i32(9), i32(9), torch.zeros(3, dtype=torch.int64), 16)
    for gap in ((i32(1), i32(2)), (i32(2), i32(3))):
        with pytest.raises(ValueError):
            mx.kv_fork(*args, gap=gap)
    with pytest.raises(TypeError):
        mx.kv_fork(*args, gap=(i32(2).long(), i32(2)))
    with pytest.raises(ValueError):
        mx.kv_fork(*args, gap=(i32(2), i32(2)))              # not on a GPU


def test_shared_workspace_by_mode(mx):
    """What is never shared needs no rows and no records of prefixes; the size without a mode suffices for every one."""
    L = mx.lib()
    size, any_mode = L.mxfa_kv_attn_shared_workspace_size_mode, L.mxfa_kv_attn_shared_workspace_size
    for R, groups, T, mq, mg, k, Hq, H in ((64, 1, 64, 1, 64, 16384, 32, 8), (8, 2, 16384, 4096, 16384, 32768, 32, 8), (3, 1, 3, 1, 3, 64, 4, 2)):
        auto, always, never = (size(R, groups, T, mq, mg, k, Hq, H, m) for m in (mx.KV_SHARE_AUTO, mx.KV_SHARE_ALWAYS, mx.KV_SHARE_NEVER))
        alone = L.mxfa_kv_attn_workspace_size(R, mq, k, Hq, H)
        assert auto == always == any_mode(R, groups, T, mq, mg, k, Hq, H) >= 1056 * T * Hq + alone
        lists = 4 * (groups + 1) + 8 * R + 4
        assert 8 * T * Hq + alone <= never <= 8 * T * Hq + alone + lists + 10 * 256
    assert size(2, 0, 3, 3, 3, 1024, 4, 2, 2) == L.mxfa_kv_attn_workspace_size(2, 3, 1024, 4, 2)
    assert size(2, 1, 3, 3, 3, 1024, 4, 2, 3) == 0 and size(2, 1, 3, 3, 3, 1024, 4, 2, -1) == 0 and size(2, 1, 3, 3, 3, 1024, 5, 2, 2) == 0
    # a call is refused for fewer bytes than its own mode needs
    c = _cache(mx)
    base = dict(q=0x10000, qs=512, T=3, cu=0x20000, kv=0x30000, R=2, bt=0x40000, nb=64, mq=3, Hq=4, s=0.1, st=0x70000, pl=0x78000,
                g=1, mg=3, sh=0, o=0x50000, lse=0x60000, ws=0x10000000, wb=0)
    call = lambda **kw: L.mxfa_kv_attn_shared(ctypes.byref(c), *dict(base, **kw).values(), None)
    for mode in (0, 1, 2):
        assert call(sh=mode, wb=size(2, 1, 3, 3, 3, 1024, 4, 2, mode) - 1) == 4
    assert call(sh=1, wb=size(2, 1, 3, 3, 3, 1024, 4, 2, 2)) == 4


def test_share_is_yes_no_or_none(mx):
    """The C values are other numbers than Python's truth values: KV_SHARE_NEVER would read as yes, KV_SHARE_AUTO as no."""
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    rows = torch.zeros((5, 4, 128), dtype=torch.bfloat16)
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)
    c = mx.KvCache(u8(3, 2, 16, 64), u8(3, 2, 16, 64), u8(3, 2, 16, 4), u8(3, 2, 16, 4), 0)
    for share in (mx.KV_SHARE_AUTO, mx.KV_SHARE_ALWAYS, mx.KV_SHARE_NEVER, "auto", 1.0):
        with pytest.raises(TypeError):
            mx.kv_attention_shared(rows, c, i32(2), i32(1), i32(1, 4), i32(2), i32(1), 5, 5, 0.1, share=share)
    for share in (None, True, False):
        with pytest.raises(ValueError):                      # not on a GPU
            mx.kv_attention_shared(rows, c, i32(2), i32(1), i32(1, 4), i32(2), i32(1), 5, 5, 0.1, share=share)
