"""Pages of the 4-bit cache at their edges: entries that are no blocks, as many forks as a call takes."""
import numpy as np
import pytest

from tests.helpers import host
from tests.test_gpu_more_kv import dev, mx  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("inplace", [False, True])
def test_fork_of_a_partial_page_that_is_not_there(mx, inplace):
    """Such a fork takes no place of the ring: the next ones get the blocks, and none is lost."""
    import torch
    table = [[1, -1, -1, -1], [2, 3, -1, -1], [4, 99, -1, -1]] + [[-9] * 4 for _ in range(5)]
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
