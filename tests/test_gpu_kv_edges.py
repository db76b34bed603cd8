"""Pages and shared prefixes of the 4-bit cache at their edges: entries that are no blocks, pages given up behind a window, as
many forks as a call takes, groups of one request, a max_q far above the tokens there are.  Bounds as in test_gpu_more_kv.py."""
import numpy as np
import pytest

from tests import more_ref
from tests.helpers import host
from tests.test_gpu_more_kv import Server, build, compare, dev, mx, results, shared_case  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("none", [-1, -2, -2 ** 31])
@pytest.mark.parametrize("inplace", [False, True])
def test_fork_of_a_partial_page_that_is_not_there(mx, inplace, none):
    """Such a fork takes no place of the ring: the next ones get the blocks, and none is lost."""
    import torch
    table = [[1, none, -1, -1], [2, 3, -1, -1], [4, 99, -1, -1]] + [[-9] * 4 for _ in range(5)]
    t, refs, ring, state = dev(table), mx.kv_refs(8), dev([0, 5, 6, 7, -1, -1, -1, -1]), dev([0, 4, 0], np.int64)
    out = mx.KvFork(*(torch.full((5,), -7, dtype=torch.int32, device="cuda") for _ in range(3)), state) if inplace else None
    # rows 0 and 2 hold one good page each: their second one is not there, or past the cache
    f = mx.kv_fork(t, dev([0, 1, 2, 1, 0]), dev([3, 4, 5, 6, 7]), dev([20, 20, 31, 17, 5]), refs, ring, state, 16, out=out)
    assert mx.device_status() == 7
    assert host(f.from_blocks).tolist() == [-1, 3, -1, 3, 1] and host(f.to_blocks).tolist() == [-1, 0, -1, 5, 6]
    assert host(f.lens).tolist() == [16, 20, 16, 17, 5] and host(f.ring_state).tolist() == [3, 4, 0]
    assert host(t)[3:].tolist() == [[1, -1, -9, -9], [2, 0, -9, -9], [4, -1, -9, -9], [2, 5, -9, -9], [6, -9, -9, -9]]
    # everything given up: the ring holds every block once
    state = mx.kv_free(t, dev(range(8)), dev([0] * 8), dev([1, 2, 1, 2, 2, 2, 2, 1]), refs, ring, f.ring_state)
    head, tail, _ = host(state).tolist()
    assert tail - head == 8 and sorted(host(ring)[(head + np.arange(8)) % 8].tolist()) == list(range(8)) and mx.device_status() == 0


def test_fork_of_a_fork_that_got_no_block(mx):
    """The row that lacked a block, forked again with the length it was meant to have."""
    t, refs, ring = dev([[1, 2], [-9, -9], [-9, -9]]), mx.kv_refs(4), dev([0, 3, -1, -1])
    f = mx.kv_fork(t, dev([0]), dev([1]), dev([20]), refs, ring, dev([2, 2, 0], np.int64), 16)
    assert host(f.lens).tolist() == [16] and host(f.ring_state).tolist() == [2, 2, 1] and host(t)[1].tolist() == [1, -1]
    assert mx.device_status() == 0
    f = mx.kv_fork(t, dev([1]), dev([2]), dev([20]), refs, ring, dev([0, 2, 0], np.int64), 16)
    assert mx.device_status() == 7
    assert host(f.lens).tolist() == [16] and host(f.to_blocks).tolist() == [-1] and host(f.ring_state).tolist() == [0, 2, 0]


def test_fork_many(mx):
    """As many forks as a call takes, most of them with a partial page, some of whose pages are not there."""
    rng = np.random.default_rng(3)
    F, R, page, width = 16384, 40, 16, 4
    blocks = R * width + F
    table = np.concatenate([rng.permutation(R * width).reshape(R, width), np.full((F, width), -1)])
    table[:R][rng.random((R, width)) < 0.1] = -1
    src, lens = rng.integers(0, R, F), rng.integers(0, width * page + 1, F)
    t, refs, ring = dev(table), mx.kv_refs(blocks), dev(R * width + np.arange(blocks) % F)
    f = mx.kv_fork(t, dev(src), dev(R + np.arange(F)), dev(lens), refs, ring, dev([0, F - 5000, 0], np.int64), page)
    assert mx.device_status() == 7
    whole, part = lens // page, lens % page != 0
    old = table[src, np.minimum(whole, width - 1)]
    wants = part & (old >= 0)
    rank = np.cumsum(wants) - wants
    got = wants & (rank < F - 5000)
    assert host(f.from_blocks).tolist() == np.where(got, old, -1).tolist()
    assert host(f.to_blocks).tolist() == np.where(got, R * width + rank, -1).tolist()
    assert host(f.lens).tolist() == np.where(part & ~got, whole * page, lens).tolist()
    assert host(f.ring_state).tolist() == [got.sum(), F - 5000, wants.sum() - got.sum()]
    shared = np.zeros(blocks, int)
    for w in range(width):
        x = table[src[whole > w], w]
        np.add.at(shared, x[x >= 0], 1)
    assert host(refs).tolist() == shared.tolist()


def fork_with_gaps(table, src, dst, lens, gaps, refs, ring, head, tail, page):
    """Fork by fork; table and refs are updated -> (from, to, lens, state)."""
    a, b, kept, want = [], [], [], 0
    for s, d, n, (g0, g1) in zip(src, dst, lens, gaps):
        whole, pair = n // page, (-1, -1)
        for j in range(whole):
            gone = g0 <= j < g1
            table[d][j] = -1 if gone else table[s][j]
            if not gone:
                refs[table[s][j]] += 1
        if n % page:
            if want < tail - head:
                pair = (table[s][whole], ring[(head + want) % len(ring)])
            else:
                n = whole * page
            want += 1
            table[d][whole] = pair[1]
        a.append(pair[0])
        b.append(pair[1])
        kept.append(n)
    took = min(want, tail - head)
    return a, b, kept, [head + took, tail, want - took]


@pytest.mark.parametrize("given_stream", [False, True])
@pytest.mark.parametrize("R,F,page,width,spare", [(2, 1, 16, 3, 1), (9, 7, 32, 7, 3), (30, 25, 16, 3000, 40), (500, 400, 64, 5, 500)])
def test_fork_with_gaps(mx, R, F, page, width, spare, given_stream):
    """Entries in the gap are not looked at, whatever they hold; without a gap the call is the one without it."""
    import torch
    rng = np.random.default_rng(R)
    lens = rng.integers(0, width * page + 1, F)
    src, whole = rng.integers(0, R, F), lens // page
    g0 = rng.integers(0, whole + 1)
    g1 = rng.integers(g0, whole + 1)
    g0[0], g1[0] = 0, whole[0]
    blocks = R * width + spare
    table = np.concatenate([rng.permutation(R * width).reshape(R, width), np.full((F, width), -5)])
    ring = np.concatenate([R * width + rng.permutation(spare), np.full(blocks - spare, -9)])
    wt, wr = table.tolist(), [0] * blocks
    want = fork_with_gaps(wt, src.tolist(), list(range(R, R + F)), lens.tolist(), list(zip(g0, g1)), wr, ring.tolist(), 0, spare, page)
    t, refs, st = dev(table), mx.kv_refs(blocks), torch.cuda.Stream() if given_stream else None
    args = (dev(src), dev(R + np.arange(F)), dev(lens), refs, dev(ring), dev([0, spare, 0], np.int64), page)
    gap = (dev(g0), dev(g1))
    torch.cuda.synchronize()
    got = mx.kv_fork(t, *args, gap=gap, stream=st)
    torch.cuda.synchronize()
    for g, w in zip((got.from_blocks, got.to_blocks, got.lens, got.ring_state), want):
        assert host(g).tolist() == w
    assert host(t).tolist() == wt and host(refs).tolist() == wr and mx.device_status() == 0
    one, two = dev(table), dev(table)
    none = torch.zeros_like(gap[0])
    a, b = mx.kv_fork(one, *args, gap=(none, none)), mx.kv_fork(two, *args)
    assert torch.equal(one, two) and all(torch.equal(getattr(a, n), getattr(b, n)) for n in ("from_blocks", "to_blocks", "lens", "ring_state"))


def test_gaps_outside_their_bounds(mx):
    t, refs, ring = dev([[7, 8, 9], [-5] * 3, [-5] * 3, [-5] * 3, [-5] * 3, [-5] * 3]), mx.kv_refs(10), dev([0, 1, 2, 3, 4, 5, 6, 0, 0, 0])
    gap = (dev([-1, 0, 2, 1, 3]), dev([1, 3, 1, 2, 3]))
    f = mx.kv_fork(t, dev([0] * 5), dev([1, 2, 3, 4, 5]), dev([40, 40, 40, 40, 48]), refs, ring, dev([0, 7, 0], np.int64), 16, gap=gap)
    assert mx.device_status() == 7                          # before the first page, behind the whole ones, end before first
    assert host(f.lens).tolist() == [0, 0, 0, 40, 48] and host(f.to_blocks).tolist() == [-1, -1, -1, 0, -1]
    assert host(t)[1:].tolist() == [[-5] * 3] * 3 + [[7, -1, 0], [7, 8, 9]] and host(f.ring_state).tolist() == [1, 7, 0]
    assert host(refs).tolist() == [0] * 7 + [2, 1, 1]
    t = dev([[7, 1 << 30, 9], [-5] * 3])                     # what was given up may be anything
    f = mx.kv_fork(t, dev([0]), dev([1]), dev([33]), refs, ring, dev([0, 7, 0], np.int64), 16, gap=(dev([1]), dev([2])))
    assert host(t)[1].tolist() == [7, -1, 0] and host(f.lens).tolist() == [33] and mx.device_status() == 0


@pytest.mark.parametrize("fmt,page,window,sinks", [(0, 16, 50, 4), (1, 32, 33, 0), (0, 16, 1, 17)])
def test_window_run_that_gives_pages_up(mx, fmt, page, window, sinks):
    """Pages behind a window go back as requests grow, others take their blocks, a request is forked with the gap and
    both go on; at the end the ring holds every block once."""
    rng = np.random.default_rng(page + window)
    R, width, blocks = 5, 900 // page, 1100 // page
    s = Server(mx, rng, fmt, page, 2, 4, R, width, blocks)
    scale, kept = 128 ** -0.5, -(-sinks // page)             # pages that hold a sink stay
    gone = [kept] * R                                        # entries kept .. gone - 1 of a row were given up

    def give_up():
        first = list(gone)
        for r in range(R):
            # the next query, at position ctx, sees the keys from ctx - window + 1 on
            gone[r] = max(gone[r], (s.ctx[r] - window + 1) // page)
        s.state = mx.kv_free(s.table, dev(range(R)), dev(first), dev(gone), s.refs, s.ring, s.state)

    def step(new):
        inside = lambda qr, p: mx.kv_attention(qr, s.c, p.cu_q, p.kv_lens, s.table, max(new), scale, window=window, sinks=sinks)
        s.check(*s.step(new, inside), window, sinks)
        give_up()

    def ended(rows):
        used = [-(-s.ctx[r] // page) for r in rows]
        whole = [(r, 0, min(kept, u)) for r, u in zip(rows, used)] + [(r, gone[r], max(gone[r], u)) for r, u in zip(rows, used)]
        s.state = mx.kv_free(s.table, *(dev([x[i] for x in whole]) for i in range(3)), s.refs, s.ring, s.state)
        for r in rows:
            s.ctx[r], s.slots[r], gone[r] = 0, [], kept
    for new in ([300, 0, 0, 100, 5], [3, 0, 0, 200, 1], [70, 0, 0, 1, 150], [1, 0, 0, 2, 60]):
        step(new)
    ended([3])
    step([20, 0, 0, 400, 1])
    lens = [s.ctx[0], gone[0] * page + window - 1]           # the whole of it; and the fewest tokens whose window is still there
    gaps = [gone[0]] * 2
    f = mx.kv_fork(s.table, dev([0, 0]), dev([1, 2]), dev(lens), s.refs, s.ring, s.state, page, gap=(dev([kept] * 2), dev(gaps)))
    mx.kv_copy_blocks(s.c, f.from_blocks, f.to_blocks)
    s.state = f.ring_state
    assert mx.device_status() == 0 and host(f.lens).tolist() == lens
    for r, n, g in zip((1, 2), lens, gaps):
        s.ctx[r], gone[r] = n, g
        assert (host(s.table)[r, kept:g] == -1).all() and g > kept
        s.slots[r] = list(s.slots[0][:n])
        for p in range(n // page * page, n):
            s.slots[r][p] = int(host(s.table)[r][p // page]) * page + p % page
    assert lens[1] < lens[0]
    for new in ([1, 1, 1, 0, 1], [4, 6, 2, 1, 1], [30, 1, 5, 200, 1], [1, 40, 1, 1, 90]):
        step(new)
    ended(range(R))
    head, tail, lacked = host(s.state).tolist()
    assert (tail - head, lacked) == (blocks, 0) and not s.refs.any() and mx.device_status() == 0
    assert sorted(host(s.ring)[(head + np.arange(blocks)) % blocks].tolist()) == list(range(blocks))


@pytest.mark.parametrize("share", [True, False, None])
def test_group_of_one_request_short_of_its_prefix(mx, share):
    """A request whose queries do not lie behind its group's prefix is left out and recorded, alone in its group too."""
    import torch
    rng = np.random.default_rng(4)
    for rows, kv_lens, lost in (([1, 1, 1], [70, 64, 90], {1}), ([1, 2, 1], [70, 65, 90], {1}), ([1, 0, 1], [70, 3, 90], set()),
                                ([1, 60, 40], [70, 120, 90], {1}), ([1, 1, 1], [70, 65, 90], set())):
        c, q, cu, kv, table, slots = build(mx, rng, 0, 16, 2, 4, rows, kv_lens)
        o, lse = results(q)
        mx.kv_attention_shared(q, c, cu, kv, table, dev([1, 2, 3]), dev([64, 20]), max(rows), max(rows), 0.1, out=(o, lse), share=share)
        torch.cuda.synchronize()
        assert mx.device_status() == (7 if lost else 0), (rows, kv_lens)
        compare(c, q, cu, slots, o, lse, lambda r, n, k: more_ref.window_mask(n, k, 1 << 30, 0), rows={0, 1, 2} - lost, scale=0.1)
        if lost:
            assert (o[rows[0]: rows[0] + rows[1]].float() == 77.0).all()


def test_capacity_costs_no_time(mx):
    """max_q is a bound that a captured step sets to what it may ever hold: the time goes by the tokens there are."""
    import torch
    rng = np.random.default_rng(5)
    R, H, G = 64, 8, 4
    q_lens = [60] + [1] * (R - 1)
    c, q, cu, kv, table, slots = build(mx, rng, 0, 64, H, G, q_lens, [300] * R)
    out = results(q)
    ws = torch.empty(mx.mxfa_kv_attn_workspace_size(R, 60, table.shape[1] * 64, H * G, H), dtype=torch.uint8, device="cuda")

    def time(max_q):
        call = lambda: mx.kv_attention(q, c, cu, kv, table, max_q, 0.1, out=out, ws=ws)
        g = torch.cuda.CUDAGraph()
        call()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            for _ in range(20):
                call()
        best = 1e9
        for _ in range(5):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            g.replay()
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b) * 1000 / 20)
        return best
    exact, most = time(60), time(1 << 30)
    # 60 ns for each turn of a loop of 2^30 tokens' blocks would be 370 us
    assert most <= 2 * exact + 60, (exact, most)
    compare(c, q, cu, slots, *out, lambda r, n, k: more_ref.window_mask(n, k, 1 << 30, 0), scale=0.1)
    assert mx.device_status() == 0


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("fmt,page,G,groups,behind", [
    (0, 16, 4, [([1] * 9, 1024, [1, 5, 64, 65, 200, 900, 1, 2, 3]), ([1], 40, [5])], [(1, 70)]),
    (1, 64, 8, [([4, 6, 1], 3000, [4, 100, 1]), ([2, 0, 5], 17, [9, 0, 129])], []),
    (0, 32, 2, [([100, 20, 1], 700, [100, 150, 1])], [(1, 2000)]),
    (0, 16, 40, [([2, 1], 700, [100, 150])], [(3, 90)])])
def test_never_shared_in_its_own_workspace(mx, fmt, page, G, groups, behind, given):
    """share=False in a workspace of that mode's bytes, from contents of any kind, and nothing behind it is written."""
    import torch
    rng = np.random.default_rng(G)
    c, q, cu, kv, table, slots, starts, pre, max_q, most, _, _ = shared_case(mx, rng, fmt, page, 2, G, groups, [], behind)
    need = mx.mxfa_kv_attn_shared_workspace_size_mode(kv.numel(), pre.numel(), q.shape[0], max_q, most, table.shape[1] * page, 2 * G, 2, mx.KV_SHARE_NEVER)
    ws = torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device="cuda") if given else None
    o, lse = results(q)
    mx.kv_attention_shared(q, c, cu, kv, table, starts, pre, max_q, most, 0.1, out=(o, lse), share=False, ws=None if ws is None else ws[:need])
    torch.cuda.synchronize()
    assert mx.device_status() == 0
    compare(c, q, cu, slots, o, lse, lambda r, n, k: more_ref.window_mask(n, k, 1 << 30, 0), scale=0.1)
    if given:
        assert (ws[need:] == 0xFF).all()
        with pytest.raises(mx.MxfaError):
            mx.kv_attention_shared(q, c, cu, kv, table, starts, pre, max_q, most, 0.1, out=(o, lse), share=True, ws=ws[:need])


@pytest.mark.parametrize("share", [True, False, None])
def test_shared_after_a_step_that_lacked_blocks(mx, share):
    """The requests that got no block keep their old kv_lens: just behind the prefix they are left out and recorded, and
    the others are as ever; kv_attention computes them all."""
    import torch
    rng = np.random.default_rng(12)
    c, q, cu, kv, table, slots = build(mx, rng, 0, 16, 2, 4, [1, 1, 1, 1], [33, 32, 32, 70], groups=[([0, 1, 2], 32)], extra=3)
    t = table.clone()
    t[0, 2] = -1
    plan = mx.kv_plan(dev([32, 32, 32, 69]), dev([1, 1, 1, 1]), t, table[0, 2:3].clone(), dev([0, 1, 0], np.int64), 16, 4)
    assert host(plan.kv_lens).tolist() == [33, 32, 32, 70] and host(plan.ring_state).tolist() == [1, 1, 2] and torch.equal(t, table)
    o, lse = results(q)
    mx.kv_attention(q, c, plan.cu_q, plan.kv_lens, t, 1, 0.1, out=(o, lse))
    assert mx.device_status() == 0
    o, lse = results(q)
    mx.kv_attention_shared(q, c, plan.cu_q, plan.kv_lens, t, dev([0, 3]), dev([32]), 1, 3, 0.1, out=(o, lse), share=share)
    assert mx.device_status() == 7
    compare(c, q, cu, slots, o, lse, lambda r, n, k: more_ref.window_mask(n, k, 1 << 30, 0), rows={0, 3}, scale=0.1)
    assert (o[1:3].float() == 77.0).all() and (lse[:, 1:3] == 77.0).all()


def test_fork_time_grows_with_the_forks(mx):
    """Eight times the forks take no more than sixteen times as long: no fork looks at all those before it."""
    import torch

    def time(F, R=40, width=64, page=16):
        blocks = R * width + F
        t = torch.cat([torch.arange(R * width, dtype=torch.int32).view(R, width), torch.full((F, width), -1, dtype=torch.int32)]).cuda()
        ring = R * width + torch.arange(blocks, dtype=torch.int32, device="cuda") % F
        args = (t, dev(np.arange(F) % R), dev(R + np.arange(F)), dev([1001] * F), mx.kv_refs(blocks), ring, dev([0, F, 0], np.int64), page)
        mx.kv_fork(*args)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(10):
                mx.kv_fork(*args)
        best = 1e9
        for _ in range(5):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            g.replay()
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b) * 100)
        return best
    few, many = time(2048), time(16384)
    assert many <= 16 * few + 20, (few, many)                # all pairs of forks: 64 times
    assert mx.device_status() == 0


@pytest.mark.parametrize("G,groups", [(4, [([1] * 9, 1024, [1, 5, 64, 65, 200, 900, 1, 2, 3])]), (4, [([100, 20, 1], 700, [100, 150, 1])]),
                                      (40, [([2, 1], 700, [100, 150])])])
def test_every_mode_captured_in_one_workspace(mx, G, groups):
    """Calls of all modes one behind another in one workspace, captured, replayed for other queries and lengths, beside the same
    on another stream with a workspace of its own."""
    import torch
    rng = np.random.default_rng(G)
    c, q, cu, kv, table, slots, starts, pre, max_q, most, q_lens, kv_lens = shared_case(mx, rng, 0, 16, 2, G, groups, [], [(1, 300)])
    n, Hq = q.shape[0], 2 * G
    size = mx.mxfa_kv_attn_shared_workspace_size(kv.numel(), pre.numel(), n, max_q, most, table.shape[1] * 16, Hq, 2)
    modes, sides = (True, False, None), []
    for _ in range(2):
        ws, outs, st = torch.empty(size, dtype=torch.uint8, device="cuda"), [results(q) for _ in modes], torch.cuda.Stream()

        def one():
            for share, out in zip(modes, outs):
                mx.kv_attention_shared(q, c, cu, kv, table, starts, pre, max_q, most, 0.1, out=out, ws=ws, share=share)
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            one()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            one()
        sides.append((g, st, outs, ws))                      # a graph keeps no tensor: its workspace has to live as long
    for shorter in (0, 1, 0):
        q.copy_(torch.randn(q.shape, device="cuda"))
        lens = [k - shorter if r == 0 and k - shorter >= int(pre[0]) + q_lens[0] else k for r, k in enumerate(kv_lens)]
        kv.copy_(dev(lens))
        torch.cuda.synchronize()
        for _ in range(5):
            for g, st, _, _ in sides:
                with torch.cuda.stream(st):
                    g.replay()
        torch.cuda.synchronize()
        assert mx.device_status() == 0
        for _, _, outs, _ in sides:
            for o, lse in outs:
                compare(c, q, cu, [s[:k] for s, k in zip(slots, lens)], o, lse, lambda r, n, k: more_ref.window_mask(n, k, 1 << 30, 0), scale=0.1)


def test_fork_with_gaps_captured(mx):
    """A fork with a gap whose counters are in place, captured once and replayed with other lists."""
    import torch
    table = np.array([[4, 5, 6, 7], [8, 9, 10, 11], [-1] * 4, [-1] * 4])
    t, refs, ring, state = dev(table), mx.kv_refs(20), dev(list(range(12, 20)) + [0] * 12), dev([0, 8, 0], np.int64)
    src, dst, lens, g0, g1 = (dev([0, 0]) for _ in range(5))
    out = mx.KvFork(*(torch.empty(2, dtype=torch.int32, device="cuda") for _ in range(3)), state)
    mx.kv_fork(t.clone(), dev([0]), dev([2]), dev([0]), refs.clone(), ring, state.clone(), 16)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mx.kv_fork(t, src, dst, lens, refs, ring, state, 16, out=out, gap=(g0, g1))
    wt, wr, head = table.tolist(), [0] * 20, 0
    for a, b, n, gaps in (([0, 1], [2, 3], [50, 33], [(1, 2), (0, 0)]), ([1, 0], [3, 2], [64, 17], [(0, 4), (0, 1)]), ([1, 1], [2, 3], [1, 0], [(0, 0), (0, 0)])):
        for x, v in zip((src, dst, lens, g0, g1), (a, b, n, [x for x, _ in gaps], [y for _, y in gaps])):
            x.copy_(dev(v))
        g.replay()
        torch.cuda.synchronize()
        want = fork_with_gaps(wt, a, b, n, gaps, wr, host(ring).tolist(), head, 8, 16)
        head = want[3][0]
        for x, w in zip((out.from_blocks, out.to_blocks, out.lens, state), want):
            assert host(x).tolist() == w
        assert host(t).tolist() == wt and host(refs).tolist() == wr
    assert mx.device_status() == 0
