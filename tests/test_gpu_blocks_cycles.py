"""Long cycles of a copy list in the order of their blocks, upwards and
downwards, alone and among trees: every block where it belongs, at the same
cost in either direction."""
import numpy as np
import pytest
import torch

from test_gpu_blocks import Blocks, idx

pytestmark = pytest.mark.gpu


def rotate(blocks, by):
    """(sources, destinations): each block takes the one ``by`` places on."""
    return np.roll(blocks, -by), blocks


@pytest.mark.parametrize("nb", [100, 8192, 8193, 16385])
@pytest.mark.parametrize("by", [1, -1, 7])
def test_a_rotation_of_all_blocks(nb, by):
    b = Blocks("lin", nb)
    src, dst = rotate(np.arange(1, nb), by)
    b.pool.copy_blocks(idx(src), idx(dst))
    torch.cuda.synchronize()
    new = np.arange(nb)
    new[dst] = src
    assert b.pool.error_flags() == 0
    assert torch.equal(b.mem, b.before[:, torch.from_numpy(new).cuda()])


@pytest.mark.parametrize("nb", [3000, 9000])
@pytest.mark.parametrize("depth", [1, 20, 100])
def test_rotations_with_trees_hanging_on_them(nb, depth):
    """Cycles of 17 to 1,000 blocks, up and down, each block of some with a
    chain of ``depth`` sources behind it, and chains of their own."""
    rng = np.random.default_rng(nb + depth)
    free = list(rng.permutation(np.arange(1, nb)))
    src, dst = [], []
    for length, by, tails in ((17, 1, 3), (40, -1, 4), (300, 1, 2), (1000, -1, 5), (2, 1, 1)):
        ring = np.sort([free.pop() for _ in range(length)])
        s, d = rotate(ring, by)
        src += s.tolist()
        dst += d.tolist()
        for at in rng.integers(0, length, tails):
            # (a chain's last source is the ring's block; each further block takes its neighbour's)
            chain = [int(ring[at])] + [int(free.pop()) for _ in range(depth)]
            src += chain[:-1]
            dst += chain[1:]
    b = Blocks("lin", nb, seed=depth)
    order = rng.permutation(len(src))
    src, dst = np.array(src)[order], np.array(dst)[order]
    b.pool.copy_blocks(idx(src), idx(dst))
    torch.cuda.synchronize()
    new = np.arange(nb)
    new[dst] = src
    assert b.pool.error_flags() == 0
    assert torch.equal(b.mem, b.before[:, torch.from_numpy(new).cuda()])


def test_either_direction_costs_the_same():
    """(The lowest block of a cycle was looked for from each of its blocks: a
    rotation downwards took a step for every pair of them.)"""
    nb = 40000
    b = Blocks("lin", nb)
    lists = [[idx(x) for x in rotate(np.arange(1, nb), by)] for by in (1, -1)]
    best = [1e9, 1e9]
    for _ in range(6):
        for i, (src, dst) in enumerate(lists):
            t0, t1 = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            torch.cuda.synchronize()
            t0.record()
            b.pool.copy_blocks(src, dst, layer=0)
            t1.record()
            torch.cuda.synchronize()
            best[i] = min(best[i], t0.elapsed_time(t1))
    print("rotations up and down, ms:", best)
    assert max(best) <= 1.5 * min(best), best
