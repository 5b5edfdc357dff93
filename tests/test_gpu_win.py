"""GPU parity of gdn_win_varlen_forward (attention with a sliding window and
sinks) with its fp64 definition: types, head layouts, lengths from one token to
many tiles, windows and sinks around the tiles' edges, padding and bad indices,
values that may not leak, streams, graphs and several calls on one pool."""
import numpy as np
import pytest
import torch

from continuous_linear_attention_gb300 import binding
from hybrid_check import SENTINEL, WinRun, bits, win_check

pytestmark = pytest.mark.gpu

FORMS = [("f32", 32), ("f32", 64), ("f32", 128), ("bf16", 32), ("bf16", 64), ("bf16", 128)]


@pytest.mark.parametrize("act,d", FORMS)
def test_short_ragged_batch(act, d):
    win_check([5, 1, 0, 33, 1, 16, 17], [3, 0, 9, 100, 50, 0, 7], 6, 3, d, 24, 3, act, rows_after=3)


@pytest.mark.parametrize("act,d", FORMS)
@pytest.mark.parametrize("H,Hkv", [(1, 1), (8, 1), (5, 5), (14, 2), (40, 1), (70, 1)])
def test_decode_batch(act, d, H, Hkv):
    win_check([1] * 9, [0, 1, 5, 39, 40, 41, 43, 44, 1000], H, Hkv, d, 40, 4, act, hint=1, seed=H)


@pytest.mark.parametrize("act,d", [("f32", 64), ("bf16", 64), ("bf16", 128)])
@pytest.mark.parametrize("past", [0, 1, 6, 90, 2_000_000_000])
@pytest.mark.parametrize("H,Hkv", [(4, 1), (3, 3)])
def test_drafted_tokens(act, d, past, H, Hkv):
    win_check([2, 4, 5, 9, 16, 17], [past] * 6, H, Hkv, d, 70, 5, act, seed=past % 7)


@pytest.mark.parametrize("n", [2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 400])
@pytest.mark.parametrize("past", [0, 77])
def test_prompts_around_the_tile_edges(n, past):
    win_check([n], [past], 4, 2, 128, 60, 4, "bf16", seed=n)


@pytest.mark.parametrize("act,d", [("f32", 32), ("bf16", 64), ("bf16", 128)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 7), (16, 0), (31, 1), (64, 64), (100, 0), (128, 4),
                                          (300, 17), (1000, 3)])
@pytest.mark.parametrize("past", [0, 2, 300])
def test_windows_and_sinks(act, d, window, sinks, past):
    win_check([150, 1, 3, 40], [past] * 4, 2, 1, d, window, sinks, act, seed=window)


@pytest.mark.parametrize("group", [1, 2, 3, 5, 7, 8, 12, 16, 24, 33])
@pytest.mark.parametrize("d", [64, 128])
def test_groups(group, d):
    win_check([130, 1, 7, 20], [50, 60, 0, 3], 2 * group, 2, d, 45, 2, "bf16", seed=group)


def test_one_query_head_per_many():
    win_check([3, 1, 40], [5, 90, 0], 160, 1, 64, 50, 2, "bf16")
    win_check([3, 1, 40], [5, 90, 0], 160, 1, 64, 50, 2, "f32")


def test_layers_pitches_and_scales():
    win_check([40, 1, 3], [10, 200, 0], 4, 2, 128, 64, 4, num_layers=3, layer=1, dense=True, scale=-0.4)
    win_check([40, 1, 3], [10, 200, 0], 4, 2, 64, 64, 4, "f32", num_layers=2, layer=1, scale=0.0)


def test_more_sequences_than_a_cta_lists():
    rng = np.random.default_rng(0)
    win_check(rng.integers(0, 6, 700).tolist(), rng.integers(0, 80, 700), 4, 2, 64, 30, 2)
    win_check([1] * 300, rng.integers(0, 80, 300), 4, 2, 128, 30, 2, hint=1)
    win_check(([1] * 299) + [200], rng.integers(0, 80, 300), 4, 2, 128, 30, 2)


def test_a_long_window():
    win_check([1, 2, 200], [5000, 3000, 2500], 8, 2, 128, 2048, 4)
    win_check([1], [100_000], 8, 1, 128, 4096, 4)


def test_a_long_prompt():
    win_check([1100, 300], [0, 900], 4, 1, 128, 512, 4)
    win_check([600], [0], 2, 2, 64, 256, 16)


@pytest.mark.parametrize("blocks,hint", [([1, 0, 2, 3], 0), ([1, 9, 2, 3], 0), ([1, -1, 2, 3], 0),
                                         ([1, 2, 2, 3], 0), ([4, 5, 6, 1], 4), ([-5, 0, 99, 99], 0)])
def test_bad_indices_leave_their_sequences_out(blocks, hint):
    for n in (4, 300):
        lens = [3, 4, 6, 1] + [0] * (n - 4)
        win_check(lens, [5] * n, 4, 2, 64, 20, 2, blocks=blocks + [-1] * (n - 4), num_blocks=8, hint=hint)


@pytest.mark.parametrize("past", [-1, -2 ** 31, 2 ** 31 - 1, 2 ** 31 - 3])
def test_past_lengths_out_of_range(past):
    for n in (3, 300):
        win_check([3, 4, 1] + [0] * (n - 3), [5, past, 9] + [0] * (n - 3), 4, 2, 64, 20, 2)


def test_the_last_positions():
    win_check([3, 1], [2 ** 31 - 4, 2 ** 31 - 2], 4, 2, 128, 20, 2)
    win_check([40], [2 ** 31 - 41], 4, 2, 128, 20, 2)


@pytest.mark.parametrize("cu", [[1, 3, 6], [0, 4, 3], [0, 3, 7], [0, -1, 6], [0, 7, 6]])
def test_bad_cu_seqlens_leave_the_batch_out(cu):
    for n in (2, 301):
        run = WinRun([3, 3] + [0] * (n - 2), [4] * n, 4, 2, 64, 20, 2)
        run.cu = cu + [cu[-1]] * (n - 2)
        run.cu_d = torch.tensor(run.cu, dtype=torch.int32, device="cuda")
        run.run()
        torch.cuda.synchronize()
        assert run.pool.error_flags() == 1
        assert (run.out == SENTINEL).all() and torch.equal(run.mem, run.before)


def test_nothing_to_do():
    run = win_check([0, 0], [4, 0], 4, 2, 64, 20, 2)
    run.T = run.N = 0
    run.run()
    torch.cuda.synchronize()
    assert torch.equal(run.mem, run.before)


BAD = [float("nan"), float("inf"), -float("inf")]
LEAK = pytest.mark.parametrize("act,d,H,Hkv", [("f32", 64, 4, 2), ("bf16", 64, 4, 2), ("bf16", 128, 8, 2),
                                               ("bf16", 128, 1, 1)])


@LEAK
@pytest.mark.parametrize("value", BAD)
@pytest.mark.parametrize("lens", [[5, 1, 9], [150, 3, 200], [1, 1, 1], [20, 1, 40]])
def test_later_tokens_and_neighbours_do_not_leak(act, d, H, Hkv, value, lens):
    """Keys and values of tokens behind a query, of other sequences and of other
    kv heads: nothing of it changes, to the bit where the form is the same and
    within the roundings else (a form may compute such rows again)."""
    past = [30, 0, 7]

    def put(x, run):
        for s in range(3):
            if lens[s] > 2:
                x[run.cu[s] + lens[s] // 2 + 1, H:] = value  # (queries up to the middle do not see it)
        x[run.cu[1]:run.cu[2], H:] = value

    run = WinRun(lens, past, H, Hkv, d, 64, 4, act, values=put)
    run.run()
    torch.cuda.synchronize()
    for s in (0, 2):
        n = lens[s] // 2 + 1
        assert torch.isfinite(run.out[run.cu[s]:run.cu[s] + n]).all(), s
    run.check()


@LEAK
@pytest.mark.parametrize("value", BAD)
def test_keys_and_values_that_have_left_the_window(act, d, H, Hkv, value):
    def put(rows, pos, s):
        for i, j in enumerate(pos):
            if j == 100:  # position 100 is in the ring until query 140 is there, which does not see it
                rows[i] = value

    for lens in ([1], [3], [60]):
        run = win_check(lens, [140], H, Hkv, d, 40, 4, act, history=put)
        assert torch.isfinite(run.out).all()


@LEAK
@pytest.mark.parametrize("value", BAD)
def test_values_that_are_not_finite_where_they_are_seen(act, d, H, Hkv, value):
    def put(x, run):
        x[run.cu[0] + 2, H + Hkv, 5] = value
        x[run.cu[2] + 10, H + Hkv:, 3] = value

    run = win_check([4, 1, 100], [9, 9, 0], H, Hkv, d, 32, 2, act, values=put)
    assert not torch.isfinite(run.out[run.cu[0] + 2, 0, 5])
    assert torch.isfinite(run.out[run.cu[2]:run.cu[2] + 10]).all()
    assert torch.isfinite(run.out[run.cu[2] + 42:]).all()


@LEAK
def test_infinite_and_nan_scores(act, d, H, Hkv):
    """A key that makes every score of a head -inf leaves the others' softmax as it
    is; one that makes it inf or NaN makes the rows that see it NaN."""
    def put(x, run):
        x[:, :H] = x[:, :H].abs() + 0.1
        x[run.cu[0] + 3, H:H + Hkv] = -float("inf")
        x[run.cu[1] + 3, H:H + Hkv] = float("inf")
        x[run.cu[2] + 3, H:H + Hkv] = float("nan")
        x[run.cu[3], H:H + Hkv] = -float("inf")  # the first query sees nothing else: NaN

    win_check([90, 90, 90, 5], [0, 0, 0, 0], H, Hkv, d, 32, 0, act, values=put)


@pytest.mark.parametrize("act,d", [("f32", 64), ("bf16", 128)])
def test_large_scores(act, d):
    win_check([70, 1], [5, 90], 4, 2, d, 64, 4, act, values=lambda x, run: x.mul_(6), scale=1.0)


@pytest.mark.parametrize("act,d", [("f32", 32), ("bf16", 64), ("bf16", 128)])
def test_a_request_over_many_calls(act, d):
    """A prompt, single tokens, drafted tokens and another prompt on one block."""
    window, sinks = 50, 3
    whole = WinRun([320], [0], 4, 2, d, window, sinks, act, seed=3)
    whole.run()
    parts = WinRun([320], [0], 4, 2, d, window, sinks, act, seed=3)
    at = 0
    for n in (1, 1, 2, 70, 1, 5, 130, 16, 1, 1, 92):
        v = WinRun([n], [at], 4, 2, d, window, sinks, act, seed=3)
        v.pool, v.blk_d = parts.pool, parts.blk_d
        for name in ("q", "k", "v", "out"):
            setattr(v, name, getattr(parts, name)[at:at + n])
        v.run()
        at += n
    torch.cuda.synchronize()
    assert at == 320
    whole.check()
    tol = 2.0 ** -7 if act == "bf16" else 1e-5  # (two roundings of each, of weights and outputs)
    assert ((whole.out - parts.out).float().abs() <= tol * (1 + whole.out.float().abs())).all()
    assert torch.equal(bits(whole.kv[whole.blk[0]]), bits(parts.kv[parts.blk[0]]))


def test_captured_and_replayed_over_other_batches():
    run = WinRun([30, 1, 20, 1], [10, 3, 0, 200], 8, 2, 128, 48, 4, seed=3)
    run.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run.run()
    for lens, past in (([30, 1, 20, 1], [10, 3, 0, 200]), ([1, 50, 0, 1], [47, 1, 0, 9]), ([13] * 4, [0, 1, 100, 5])):
        run.cu_d.copy_(torch.tensor([0] + np.cumsum(lens).tolist(), dtype=torch.int32))
        run.past_d.copy_(torch.tensor(past, dtype=torch.int32))
        run.mem.view(torch.bfloat16).normal_()
        start = run.mem.clone()
        run.out.fill_(SENTINEL)
        graph.replay()
        torch.cuda.synchronize()
        out, mem = run.out.clone(), run.mem.clone()
        run.mem.copy_(start)
        run.out.fill_(SENTINEL)
        run.run()
        torch.cuda.synchronize()
        assert torch.equal(bits(out), bits(run.out)) and torch.equal(mem, run.mem), lens
        assert run.pool.error_flags() == 0


def test_another_stream_and_two_pools_at_once():
    a = WinRun([30, 1, 20], [10, 90, 0], 8, 2, 128, 48, 4, seed=3)
    b = WinRun([1] * 40, [100] * 40, 8, 1, 128, 300, 4, seed=4, hint=1)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):  # (the same tokens again: only single tokens leave the block the same)
        with torch.cuda.stream(t):
            b.run()
    with torch.cuda.stream(s):
        a.run()
    torch.cuda.synchronize()
    a.check()
    b.check()


def test_a_call_right_behind_another():
    """Single tokens of the same requests, call behind call: each reads what the last one wrote."""
    n, steps = 20, 12
    run = WinRun([1] * n, [0] * n, 8, 2, 128, 8, 2, seed=5, hint=1)
    rows = torch.randn(steps, n, 12, 128, generator=torch.Generator().manual_seed(1)).bfloat16()
    dev = rows.cuda()
    outs = torch.zeros(steps, n, 8, 128, dtype=torch.bfloat16, device="cuda")
    pasts = torch.arange(steps, dtype=torch.int32, device="cuda")[:, None].repeat(1, n).contiguous()
    for i in range(steps):
        binding.win_varlen_forward(run.pool, 0, dev[i][:, :8], dev[i][:, 8:10], dev[i][:, 10:], run.cu_d, run.blk_d,
                                   pasts[i], outs[i], n, n, scale=run.scale, max_seqlen_hint=1)
    torch.cuda.synchronize()
    whole = WinRun([steps] * n, [0] * n, 8, 2, 128, 8, 2, seed=5)
    flat = rows.transpose(0, 1).reshape(n * steps, 12, 128)
    whole.x.copy_(flat)
    whole.q.copy_(flat[:, :8]), whole.k.copy_(flat[:, 8:10]), whole.v.copy_(flat[:, 10:])
    whole.run()
    torch.cuda.synchronize()
    whole.check()
    got = outs.transpose(0, 1).reshape(n * steps, 8, 128).float()
    assert ((got - whole.out.float()).abs() <= 2.0 ** -7 * (1 + whole.out.float().abs())).all()


def test_fork_and_compaction_carry_the_window():
    run = WinRun([40, 1], [0, 100], 4, 2, 64, 30, 2, num_blocks=9)
    run.run()
    src = torch.tensor([run.blk[0]], dtype=torch.int32, device="cuda")
    free = [b for b in range(1, 9) if b not in run.blk]
    dst = torch.tensor([free[0]], dtype=torch.int32, device="cuda")
    run.pool.copy_blocks(src, dst)
    torch.cuda.synchronize()
    page = run.mem.view(9, -1)
    assert torch.equal(page[free[0]], page[run.blk[0]])


def test_host_refusals():
    run = WinRun([3, 1], [5, 0], 4, 2, 64, 20, 2)
    lib = binding.load()
    P = lambda t: t.data_ptr()  # noqa: E731

    def go(pool=run.pool, layer=0, q=P(run.q), k=P(run.k), v=P(run.v), ldq=512, ldk=512, ldv=512, H=4,
           cu=P(run.cu_d), past=P(run.past_d), out=P(run.out), ldo=256, T=4, N=2, hint=0):
        return lib.gdn_win_varlen_forward(pool.handle, layer, q, k, v, ldq, ldk, ldv, H, cu, P(run.blk_d), past,
                                          1.0, out, ldo, T, N, hint, None)

    lin = binding.LinPool(4, 1, 2, 32, "bf16")
    assert [go(layer=1), go(layer=-1), go(T=-1), go(N=-1), go(hint=-1), go(N=0), go(ldq=248), go(ldo=1 << 39),
            go(T=2 ** 31 - 1)] == [-3] * 9
    assert [go(q=None), go(out=None), go(cu=None), go(past=None)] == [-1] * 4
    assert [go(q=P(run.q) + 2), go(ldk=516), go(ldo=260)] == [-4] * 3
    assert [go(pool=lin), go(H=3), go(H=0), go(H=8192)] == [-2] * 4 and go(T=0, N=0) == 0
    for f in (lambda: binding.varlen_forward(run.pool, 0, run.q, run.q, run.q, run.cu_d, run.blk_d, run.past_d, run.q,
                                             run.q, run.q, run.out, 4, 2),
              lambda: binding.lin_varlen_forward(run.pool, 0, run.q, run.k, run.v, run.cu_d, run.blk_d, run.past_d,
                                                 run.q, run.out, 4, 2)):
        with pytest.raises((binding.GdnError, ValueError)):
            f()
    torch.cuda.synchronize()
    assert (run.out == SENTINEL).all() and torch.equal(run.mem, run.before)


@LEAK
@pytest.mark.parametrize("value", BAD)
def test_queries_that_are_not_finite_reach_their_own_row_only(act, d, H, Hkv, value):
    def put(x, run):
        for s in range(run.N):
            x[run.cu[s + 1] - 1, 0] = value

    lens = [150, 5, 1]
    a = WinRun(lens, [7, 30, 60], H, Hkv, d, 64, 4, act)
    b = WinRun(lens, [7, 30, 60], H, Hkv, d, 64, 4, act, values=put)
    for r in (a, b):
        r.run()
    torch.cuda.synchronize()
    for s in range(3):
        last = b.cu[s + 1] - 1
        assert torch.isnan(b.out[last, 0]).all()
        assert torch.equal(bits(a.out[b.cu[s]:last]), bits(b.out[b.cu[s]:last]))
        assert torch.equal(bits(a.out[last, 1:]), bits(b.out[last, 1:]))


def test_prompts_in_two_graphs_on_one_pool():
    """Both use the pool's lists and counters, one behind the other, replayed in both orders."""
    a = WinRun([300, 1, 40], [10, 90, 0], 8, 2, 128, 48, 4, seed=3, blocks=[1, 2, 3], num_blocks=8)
    b = WinRun([700, 1], [100, 50], 8, 2, 128, 48, 4, seed=4, blocks=[4, 5], num_blocks=8)
    b.kv[a.blk] = a.kv[a.blk]
    start = b.mem.clone()
    a.pool = b.pool
    graphs, want = [], []
    for r in (a, b):
        b.mem.copy_(start)
        r.run()
        torch.cuda.synchronize()
        want.append(r.out.clone())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            r.run()
        graphs.append(g)
    for order in ((0, 1), (1, 0), (1, 0)):
        b.mem.copy_(start)
        for r in (a, b):
            r.out.fill_(SENTINEL)
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for r, w in zip((a, b), want):
            assert torch.equal(bits(r.out), bits(w)), order
    assert b.pool.error_flags() == 0


def test_more_sequences_than_a_cta_lists_with_long_prompts():
    lens = [0, 1] * 150 + [260, 40, 300]
    win_check(lens, [3] * 303, 4, 2, 128, 50, 2)
    win_check(lens, [3] * 303, 4, 2, 64, 50, 2)


def test_values_that_are_not_finite_in_every_prompt_and_head():
    """More units than the list of those done again holds: all of them are."""
    def put(x, run):
        for s in range(run.N):
            x[run.cu[s] + 30, 130:, 1] = float("inf")

    win_check([33] * 256, [0] * 256, 65, 65, 64, 20, 0, values=put)


def test_scales_that_are_not_finite_are_refused():
    run = WinRun([3, 1], [5, 0], 4, 2, 64, 20, 2)
    for scale in (float("nan"), float("inf"), -float("inf")):
        run.scale = scale
        with pytest.raises(binding.GdnError):
            run.run()
    torch.cuda.synchronize()
    assert (run.out == SENTINEL).all() and torch.equal(run.mem, run.before)
