"""The one-to-one bindings of the 4-bit cache's, the rotation's and the pages' C entry points: each gives, from the same
buffers, the bytes that the function built on it gives."""
import ctypes

import numpy as np
import pytest

from tests.helpers import host
from tests.test_gpu_kv import bf16, new_cache
from tests.test_gpu_more_kv import build, dev, mx, shared_case  # noqa: F401

pytestmark = pytest.mark.gpu


def bits(t):
    import torch
    return t.contiguous().view(torch.uint8)


def same(a, b):
    import torch
    return all(torch.equal(bits(x), bits(y)) for x, y in zip(a, b))


def like(*ts):
    import torch
    return [torch.full_like(t, 7) for t in ts]


@pytest.mark.parametrize("side", [False, True])
def test_attention(mx, side):
    import torch
    rng = np.random.default_rng(1)
    st = torch.cuda.Stream() if side else None
    case = shared_case(mx, rng, 1, 16, 2, 4, [([1, 2, 1], 300, [1, 20, 300])], [], [])
    c, q, cu, kv, table, _, starts, pre, max_q, most, q_lens, _ = case
    q = q[: sum(q_lens)]
    T, R, nb, k = q.shape[0], kv.numel(), table.shape[1], table.shape[1] * 16
    own = table.clone()
    for r in range(1, 3):                                    # a table for the calls that know of no group
        own[r, :300 // 16] = table[0, :300 // 16]
    head = (c.pages, q, q.stride(0), T, cu, kv, R)
    ws = lambda n: torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")

    def check(want, f, size, t, *rest):
        o, lse = like(*want)
        w = ws(size)
        torch.cuda.synchronize()
        f(*head, t, nb, max_q, 8, 0.1, *rest, o, lse, w, size, st)
        torch.cuda.synchronize()
        assert same((o, lse), want)
    check(mx.kv_attention(q, c, cu, kv, own, max_q, 0.1), mx.mxfa_kv_attn, mx.mxfa_kv_attn_workspace_size(R, max_q, k, 8, 2), own, 1)
    check(mx.kv_attention(q, c, cu, kv, own, max_q, 0.1, window=100, sinks=3), mx.mxfa_kv_attn_window,
          mx.mxfa_kv_attn_window_workspace_size(R, max_q, k, 8, 2, 100, 3), own, 100, 3)
    for mode, share in ((mx.KV_SHARE_AUTO, None), (mx.KV_SHARE_ALWAYS, True), (mx.KV_SHARE_NEVER, False)):
        want = mx.kv_attention_shared(q, c, cu, kv, table, starts, pre, max_q, most, 0.1, share=share)
        args = (R, 1, T, max_q, most, k, 8, 2)
        for size in (mx.mxfa_kv_attn_shared_workspace_size(*args), mx.mxfa_kv_attn_shared_workspace_size_mode(*args, mode)):
            check(want, mx.mxfa_kv_attn_shared, size, table, starts, pre, 1, most, mode)
    assert mx.device_status() == 0


def test_rows(mx):
    import torch
    rng = np.random.default_rng(2)
    T, Hq, H = 37, 6, 3
    fused = bf16(rng, T, Hq + 2 * H, 128).cuda()
    q, k, v = fused[:, :Hq], fused[:, Hq: Hq + H], fused[:, Hq + H:]
    rp, pos, slots = mx.Rope.make(64, interleaved=True, gain=1.5), dev(rng.integers(0, 5000, T)), dev(rng.permutation(64)[:T], np.int64)
    rot = mx.Rotation(rp.turns.data_ptr(), 64, mx.ROPE_INTERLEAVED, 1.5)
    want, back = mx.rope(q, rp, pos), mx.rope_bwd(q, rp, pos)
    y, z = like(want, back)
    mx.mxfa_rope(q, q.stride(0), y, Hq * 128, pos, T, Hq, 128, rot, 0)
    mx.mxfa_rope(q, q.stride(0), z, Hq * 128, pos, T, Hq, 128, rot, 1)
    assert same((y, z), (want, back))
    one, two = (new_cache(mx, 4, H, 16, 0) for _ in range(2))
    want = mx.kv_append_rope(one, q, k, v, rp, pos, slots)
    y, = like(want)
    s = fused.stride(0)
    mx.mxfa_kv_append_rope(two.pages, q, s, Hq, k, s, v, s, T, pos, slots, rot, y, Hq * 128)
    stored = lambda c: (c.k, c.v, c.k_sf, c.v_sf)
    assert same((y, *stored(two)), (want, *stored(one)))
    mx.kv_append(one, v, k, slots)
    mx.mxfa_kv_append(two.pages, v, k, s, s, T, slots)
    assert same(stored(two), stored(one))
    want = mx.kv_load(one, slots)
    got = like(*want)
    mx.mxfa_kv_load(two.pages, slots, T, *got)
    assert same(got, want)
    mx.kv_copy_blocks(one, dev([0, 1]), dev([3, 2]))
    mx.mxfa_kv_copy_blocks(two.pages, dev([0, 1]), dev([3, 2]), 2)
    assert same(stored(two), stored(one)) and mx.device_status() == 0


def test_pages(mx):
    import torch
    ctx, add = dev([20, 0, 5]), dev([3, 40, -1])
    table = dev([[4, 5, -1, -1], [-1] * 4, [6, -1, -1, -1]])

    def fresh():
        ring, state = mx.kv_ring(10)
        ring[:4], state[1] = torch.arange(4, device="cuda"), 4
        return table.clone(), mx.kv_refs(10), ring, state
    t, refs, ring, state = fresh()
    want = mx.kv_plan(ctx, add, t, ring, state, 16, 44)
    u, refs2, ring2, state2 = fresh()
    names = ("cu_q", "kv_lens", "slots", "positions")
    got = like(*(getattr(want, n) for n in names))
    out = torch.zeros_like(state2)
    mx.mxfa_kv_plan(ctx, add, 3, u, 4, ring2, 10, state2, out, 16, 44, *got)
    assert same(got + [u, ring2, out], [getattr(want, n) for n in names] + [t, ring, want.ring_state])
    src, dst, lens = dev([1]), dev([2]), dev([37])
    for gap in (None, (dev([1]), dev([2]))):
        state, (u, refs2, ring2) = want.ring_state, (x.clone() for x in (t, refs, ring))
        f = mx.kv_fork(t, src, dst, lens, refs, ring, state, 16, gap=gap)
        from_, to, kept, out = like(f.from_blocks, f.to_blocks, f.lens, f.ring_state)
        if gap is None:
            mx.mxfa_kv_fork(u, 3, 4, src, dst, lens, 1, refs2, 10, ring2, 10, state, out, 16, from_, to, kept)
        else:
            mx.mxfa_kv_fork_gap(u, 3, 4, src, dst, lens, *gap, 1, refs2, 10, ring2, 10, state, out, 16, from_, to, kept)
        assert same((from_, to, kept, out, u, refs2), (f.from_blocks, f.to_blocks, f.lens, f.ring_state, t, refs))
        rows, first, end = dev([2]), dev([0]), dev([3])
        s = mx.kv_free(t, rows, first, end, refs, ring, f.ring_state)
        mx.mxfa_kv_free(u, 3, 4, rows, first, end, 1, refs2, 10, ring2, 10, f.ring_state, out)
        assert same((out, refs2, ring2), (s, refs, ring))
        want = mx.KvStep(*(getattr(want, n) for n in names), s)
    assert mx.device_status() == 0


def test_a_status_is_raised(mx):
    c = new_cache(mx, 2, 1, 16, 0)
    with pytest.raises(mx.MxfaError):
        mx.mxfa_kv_copy_blocks(c.pages, dev([0]), dev([1]), 8193)
    with pytest.raises(mx.MxfaError):
        mx.mxfa_rope(None, 128, None, 128, None, 1, 1, 128, mx.Rotation(None, 64, 0, 1.0), 0)
    assert ctypes.sizeof(mx.Rotation) == 24 and host(c.k).shape == (2, 1, 16, 64)
