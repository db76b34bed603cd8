"""Refusals of the 4-bit cache's calls for pages and shared prefixes, without a GPU (all before any launch)."""
import pytest
import torch

from tests.test_more_kv_checks import mx  # noqa: F401


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
