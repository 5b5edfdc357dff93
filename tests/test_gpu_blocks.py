"""The pool's block operations on the GPU: copy lists with every overlap a
beam search makes, free and compaction, against the definitions, bit for bit."""
import numpy as np
import pytest
import torch

from continuous_linear_attention_gb300 import binding
from lin_check import LinRun, check
from oracle import lin as ref

pytestmark = pytest.mark.gpu

# (make the pool, layers): blocks of 2.1 MB, 19 KiB, 4 KiB and 64.25 KiB
POOLS = {
    "gdn": lambda nb, mem=None: binding.Pool(nb, 2, 16, 32, 128, 128, 4, "bf16", memory=mem),
    "gdn_small": lambda nb, mem=None: binding.Pool(nb, 3, 2, 4, 32, 32, 4, "f32", memory=mem),
    "lin": lambda nb, mem=None: binding.LinPool(nb, 5, 1, 32, "f32", memory=mem),
    "ssd": lambda nb, mem=None: binding.SsdPool(nb, 1, 2, 64, 128, 1, 4, "bf16", memory=mem),
}


class Blocks:
    """A pool over a torch tensor of random words, [layers][blocks][words]."""

    def __init__(self, kind, nb, seed=0):
        probe = POOLS[kind](2)
        words, layers = probe.stride // 4, probe.num_layers
        probe.close()
        self.mem = torch.empty(layers, nb, words, dtype=torch.int32, device="cuda")
        self.pool = POOLS[kind](nb, self.mem.view(-1).view(torch.uint8))
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.mem.random_(generator=g)
        self.mem[:, 0] = 0
        self.nb, self.layers = nb, layers
        # blocks are only moved: a few words of each and all its sums say where it went
        self.before = self.mem.clone()

    def check(self, want_of, flags, layer=-1):
        """want_of: {block: source block or None (zeros)} of those that change."""
        assert self.pool.error_flags(layer=max(layer, 0)) == flags
        want = self.before.clone()
        at = slice(None) if layer < 0 else slice(layer, layer + 1)
        for b, s in want_of.items():
            want[at, b] = 0 if s is None else self.before[at, s]
        assert torch.equal(self.mem, want)


def idx(v):
    return torch.tensor(list(v), dtype=torch.int32, device="cuda")


def expect(nb, src, dst):
    """{block: source} by the definition on block numbers."""
    mem = np.arange(nb)[None]
    out, flags = ref.copy_blocks(mem, src, dst)
    return {b: int(out[0, b]) for b in range(nb) if out[0, b] != b}, flags


LISTS = {
    "one": ([3], [7]),
    "fork": ([5, 5, 5, 5], [1, 2, 3, 4]),
    "zero": ([0, 0], [3, 4]),
    "itself": ([4, 4], [4, 6]),
    "swap": ([1, 2], [2, 1]),
    "cycle": ([1, 2, 3, 4, 5], [2, 3, 4, 5, 1]),
    "two_cycles": ([1, 2, 7, 8, 9], [2, 1, 8, 9, 7]),
    "chain": ([1, 2, 3, 4, 5, 6], [2, 3, 4, 5, 6, 7]),
    "chain_down": ([7, 6, 5, 4], [6, 5, 4, 3]),
    "beams": ([2, 1, 3, 3, 5, 5, 6, 8], [1, 2, 3, 4, 5, 6, 7, 8]),
    "cycle_with_trees": ([1, 2, 3, 1, 4, 4, 2, 9], [2, 3, 1, 4, 5, 6, 7, 8]),
    "padding": ([3, -1, 4, -5], [5, 6, -1, -2]),
    "bad": ([3, 99, 4, 5, 5, 6], [7, 8, 99, 0, 9, 9]),
    "all_skipped": ([-1, 99, 2], [4, 3, 0]),
    "twice_itself": ([4, 3], [4, 4]),
}


@pytest.mark.parametrize("kind", ["lin", "gdn_small", "ssd", "gdn"])
@pytest.mark.parametrize("name", LISTS)
def test_copy_lists(kind, name):
    src, dst = LISTS[name]
    b = Blocks(kind, 11)
    b.pool.copy_blocks(idx(src), idx(dst))
    torch.cuda.synchronize()
    b.check(*expect(11, src, dst))


@pytest.mark.parametrize("layer", [0, 2])
def test_one_layer(layer):
    b = Blocks("gdn_small", 9)
    b.pool.copy_blocks(idx([1, 2, 3, 99]), idx([2, 1, 4, 1]), layer=layer)
    torch.cuda.synchronize()
    b.check({1: 2, 2: 1, 4: 3}, ref.BLOCK_RANGE, layer)
    assert b.pool.error_flags() == 0


@pytest.mark.parametrize("kind,nb,seed", [("lin", 300, 0), ("lin", 1500, 1), ("gdn_small", 700, 2),
                                          ("lin", 9000, 3), ("lin", 9000, 4), ("gdn", 40, 5)])
def test_random_functions(kind, nb, seed):
    """Any source for any set of destinations: trees of any depth on roots and
    cycles of any length; above 8192 blocks the plan works in device memory."""
    rng = np.random.default_rng(seed)
    b = Blocks(kind, nb, seed)
    dst = rng.permutation(nb - 1)[: int((nb - 1) * (0.3 + 0.7 * rng.random()))] + 1
    if seed % 2:
        src = rng.permutation(dst)  # a permutation: cycles only
    else:
        src = rng.integers(0, nb, len(dst))
    b.pool.copy_blocks(idx(src), idx(dst))
    torch.cuda.synchronize()
    new = np.arange(nb)
    new[dst] = src
    want = b.before[:, torch.from_numpy(new).cuda()]
    assert b.pool.error_flags() == 0 and torch.equal(b.mem, want)


@pytest.mark.parametrize("nb", [1025, 2500, 8193])
def test_the_longest_chain_and_cycle(nb):
    b = Blocks("lin", nb)
    order = np.random.default_rng(nb).permutation(nb - 1) + 1
    b.pool.copy_blocks(idx(order), idx(np.roll(order, 1)))
    torch.cuda.synchronize()
    new = np.arange(nb)
    new[np.roll(order, 1)] = order
    assert torch.equal(b.mem, b.before[:, torch.from_numpy(new).cuda()])
    b.before.copy_(b.mem)
    b.pool.copy_blocks(idx(order[:-1]), idx(order[1:]))
    torch.cuda.synchronize()
    new = np.arange(nb)
    new[order[1:]] = order[:-1]
    assert torch.equal(b.mem, b.before[:, torch.from_numpy(new).cuda()])


@pytest.mark.parametrize("kind", ["lin", "gdn", "ssd"])
def test_free(kind):
    b = Blocks(kind, 12)
    b.pool.clear_blocks(idx([3, -1, 11, 3, 7]))
    torch.cuda.synchronize()
    b.check({3: None, 11: None, 7: None}, 0)
    b.before.copy_(b.mem)
    b.pool.clear_blocks(idx([0, 5, 12]), layer=0)
    torch.cuda.synchronize()
    b.check({5: None}, ref.TRASH_WRITE | ref.BLOCK_RANGE, 0)


@pytest.mark.parametrize("nb,live", [
    (12, [9, 2, 11, 1]), (12, [1, 2, 3]), (12, [11]), (12, [-1, 0, 8, 8, 3, 40]), (12, list(range(1, 12))),
    (12, [-1, -2]), (3000, 1700), (9000, 40), (9000, 5000),
])
def test_compaction(nb, live):
    if isinstance(live, int):
        live = (np.random.default_rng(nb).permutation(nb - 1)[:live] + 1).tolist()
    for alias in (False, True):
        b = Blocks("gdn_small" if nb < 100 else "lin", nb)
        given = idx(live)
        new = given if alias else torch.full_like(given, -77)
        assert b.pool.compact(given, new) is new
        torch.cuda.synchronize()
        _, want, flags = ref.compact(np.zeros((1, nb)), live)
        assert new.tolist() == want
        moved = {w: a for a, w in zip(live, want) if a != w}
        b.check(moved, flags)
        assert sorted(set(w for w in want if 0 < w < nb)) == list(
            range(1, len({w for w in want if 0 < w < nb}) + 1))


def test_empty_lists_and_refusals():
    b = Blocks("lin", 5)
    none = idx([])
    b.pool.copy_blocks(none, none)
    b.pool.clear_blocks(none)
    b.pool.compact(none)
    lib, one = binding.load(), idx([1])
    p, h = one.data_ptr(), b.pool.handle
    assert lib.gdn_state_pool_copy_blocks(h, 5, p, p, 1, None) == -3
    assert lib.gdn_state_pool_copy_blocks(h, -2, p, p, 1, None) == -3
    assert lib.gdn_state_pool_copy_blocks(h, 0, p, p, -1, None) == -3
    assert lib.gdn_state_pool_copy_blocks(h, 0, p, None, 1, None) == -1
    assert lib.gdn_state_pool_clear_blocks(h, 0, None, 1, None) == -1
    assert lib.gdn_state_pool_clear_blocks(h, 5, p, 1, None) == -3
    assert lib.gdn_state_pool_compact(h, p, None, 1, None) == -1
    with pytest.raises(ValueError):
        b.pool.copy_blocks(idx([1, 2]), one)
    with pytest.raises(ValueError):
        b.pool.clear_blocks(one.long())
    with pytest.raises(ValueError):
        b.pool.compact(idx([1, 2]), one)
    torch.cuda.synchronize()
    b.check({}, 0)


def test_captured_reorder_replays_over_new_lists():
    b = Blocks("gdn_small", 20)
    src, dst = idx([1, 2, 3, -1]), idx([2, 1, 5, -1])
    b.pool.copy_blocks(src, dst)  # loads the kernels
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.pool.copy_blocks(src, dst, stream=torch.cuda.current_stream())
    b.before.copy_(b.mem)
    src.copy_(idx([7, 8, 9, 7]))
    dst.copy_(idx([8, 9, 7, 12]))
    g.replay()
    torch.cuda.synchronize()
    b.check({8: 7, 9: 8, 7: 9, 12: 7}, 0)


def test_a_beam_search_and_its_end():
    """A prompt, its fork into beams, steps with reorders between them, then
    compaction and free: each beam's rows and state equal those of its whole
    token path run alone."""
    H, d, beams = 4, 128, 4
    prompt, steps = 200, 5
    tree = LinRun([prompt + steps * beams], [0], H, 2, d, "bf16", num_blocks=16, blocks=[6], seed=1)
    dev = dict(dtype=torch.int32, device="cuda")
    pool, mem = tree.pool, tree.view

    def forward(rows, cu, blocks, past):
        out = torch.empty(len(rows), H, d, dtype=torch.bfloat16, device="cuda")
        binding.lin_varlen_forward(pool, 0, tree.q[rows], tree.k[rows], tree.v[rows],
                                   torch.tensor(cu, **dev), blocks,
                                   torch.tensor(past, dtype=torch.uint8, device="cuda"),
                                   tree.decay_d, out, len(rows), len(cu) - 1, scale=tree.scale)
        return out

    forward(list(range(prompt)), [0, prompt], idx([6]), [0])
    slots = [6, 9, 3, 12]
    pool.copy_blocks(idx([6, 6, 6]), idx(slots[1:]))
    paths = [list(range(prompt)) for _ in range(beams)]
    parents = [[0, 0, 1, 3], [1, 0, 3, 2], [2, 2, 2, 2], [3, 2, 1, 0], [1, 2, 3, 0]]
    for i, parent in enumerate(parents):
        rows = [prompt + i * beams + j for j in range(beams)]
        last = forward(rows, list(range(beams + 1)), idx(slots), [1] * beams)
        for j in range(beams):
            paths[j].append(rows[j])
        pool.copy_blocks(idx([slots[p] for p in parent]), idx(slots))
        paths = [list(paths[p]) for p in parent]
        last = last[parent]
    table = pool.compact(idx(slots))
    # 3 stays; 6, 9 and 12 move to 1, 2 and 4
    assert table.tolist() == [1, 2, 3, 4]
    pool.clear_blocks(idx([6, 9, 12]))
    torch.cuda.synchronize()
    assert pool.error_flags() == 0
    assert not mem[0, [6, 9, 12]].any()
    for j in range(beams):
        alone = LinRun([len(paths[j])], [0], H, 2, d, "bf16", num_blocks=4, blocks=[1], seed=1,
                       values=lambda x, run, j=j: x.copy_(tree.x[paths[j]]))
        alone.view[0, 1] = mem[0, table[j]]
        alone.out.fill_(0)
        out, states = alone.expected()
        got = mem[0, table[j]].double().cpu().numpy()
        assert np.linalg.norm(got - states[0]) <= 1e-5 * np.linalg.norm(states[0])
        o = last[j].double().cpu().numpy()
        assert np.linalg.norm(o - out[-1]) <= 2.0 ** -7 * np.linalg.norm(out[-1])


def test_block_operations_follow_their_stream():
    """On a stream of their own behind slow work that writes the blocks and the
    lists, while another pool is busy on another stream."""
    a, b = Blocks("gdn", 12, seed=1), Blocks("lin", 40, seed=2)
    first, zero = idx([1, 2, 3]), idx([0, 0, 0])
    src, dst, dead = zero.clone(), zero.clone(), zero.clone()
    lists = idx([2, 1, 1]), idx([1, 2, 5]), idx([7, 7, -1])
    fresh = torch.randint_like(a.mem, 2 ** 31 - 1)
    fresh[:, 0] = 0
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(2_000_000)
        a.mem.copy_(fresh)
        for x, y in zip((src, dst, dead), lists):
            x.copy_(y)
        a.pool.copy_blocks(src, dst)
        a.pool.clear_blocks(dead)
        for x in (src, dst, dead):
            x.copy_(first)
    with torch.cuda.stream(t):
        b.pool.copy_blocks(idx([4, 5]), idx([5, 4]))
    torch.cuda.synchronize()
    a.before = fresh
    a.check({1: 2, 2: 1, 5: 1, 7: None}, 0)
    b.check({5: 4, 4: 5}, 0)


def test_operations_one_after_the_other_without_a_host_wait():
    """Each operation's plan may not overtake the moves before it."""
    b = Blocks("lin", 64, seed=5)
    rng = np.random.default_rng(6)
    where = np.arange(64)
    for _ in range(40):
        dst = rng.permutation(np.arange(1, 64))[:rng.integers(1, 63)]
        src = rng.integers(1, 64, len(dst))
        b.pool.copy_blocks(idx(src), idx(dst))
        where[dst] = where[src]
    torch.cuda.synchronize()
    b.check({x: int(where[x]) for x in range(64)}, 0)


@pytest.mark.parametrize("n", [15, 16, 17, 18, 33])
@pytest.mark.parametrize("shape", ["chain", "cycle", "tail_into_cycle", "tail_into_long_cycle", "tails"])
def test_walks_around_the_length_that_is_walked(n, shape):
    """Chains, cycles and tails of blocks about as long as the plan follows
    them step by step, among short ones."""
    order = np.random.default_rng(n).permutation(np.arange(1, 120)).tolist()
    pairs = [(order[0], order[1]), (order[2], order[3]), (order[3], order[2])]
    line = order[4:4 + n]
    # (source, destination): the last of the line is the one that is read first
    pairs += list(zip(line[1:], line))
    ring = {"cycle": line, "tail_into_cycle": order[60:62], "tail_into_long_cycle": order[60:60 + n]}.get(shape)
    if shape == "cycle":
        pairs.append((line[0], line[-1]))
    elif ring:
        pairs += list(zip(ring[1:], ring)) + [(ring[0], ring[-1]), (ring[0], line[-1])]
    elif shape == "tails":
        other = order[60:60 + n]
        pairs += list(zip(other[1:], other)) + [(line[0], other[-1])]
    src, dst = zip(*pairs)
    b = Blocks("lin", 130, seed=n)
    b.pool.copy_blocks(idx(src), idx(dst))
    want, flags = expect(130, src, dst)
    torch.cuda.synchronize()
    b.check(want, flags)
    assert flags == 0
