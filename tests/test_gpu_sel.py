"""GPU parity of gdn_sel_conv_varlen_forward and gdn_sel_scan_varlen_forward
with their fp64 definitions: types, sizes, lengths from none to many tiles,
pitches, padding and bad indices, values that may not leak, streams, graphs."""
import ctypes

import numpy as np
import pytest
import torch

from continuous_linear_attention_gb300 import binding
from hybrid_check import I32, SENTINEL, SelRun, bits, sel_check

pytestmark = pytest.mark.gpu

BOTH = pytest.mark.parametrize("what", ["conv", "scan"])
RAGGED = [5, 1, 0, 33, 2, 1, 16, 3, 65]
PAST = [1, 0, 1, 1, 0, 1, 0, 1, 0]


@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("channels", [8, 72, 1032])
def test_conv_ragged(K, act, channels):
    sel_check("conv", RAGGED, PAST, channels, K=K, act=act, bias=K != 3, rows_after=3)


@pytest.mark.parametrize("N", [16, 32, 64])
@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("channels", [8, 72, 264])
def test_scan_ragged(N, act, channels):
    sel_check("scan", RAGGED, PAST, channels, N=N, act=act, gate=N != 32, rows_after=3)


@BOTH
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 300])
def test_one_sequence_around_the_tiles(what, n):
    sel_check(what, [n], [n % 2], 40, act="f32", seed=n)


@BOTH
@pytest.mark.parametrize("act,N,K", [("bf16", 16, 4), ("f32", 16, 2), ("bf16", 32, 3), ("f32", 64, 4)])
def test_single_tokens(what, act, N, K):
    sel_check(what, [1] * 11, [1, 1, 0, 1, 1, 0, 1, 1, 1, 0, 1], 136, N=N, K=K, act=act, hint=1)


@BOTH
def test_wide_rows_and_other_layers(what):
    sel_check(what, [70, 1, 40], [1, 1, 0], 4096, num_layers=3, layer=1, dense=True)


@pytest.mark.parametrize("what,N,channels", [("conv", 16, 24), ("scan", 16, 24), ("scan", 64, 8)])
def test_more_sequences_than_a_cta_lists(what, N, channels):
    rng = np.random.default_rng(0)
    lens = rng.integers(0, 5, 700).tolist()
    sel_check(what, lens, rng.integers(0, 2, 700), channels, N=N)
    sel_check(what, [1] * 300, [1] * 300, channels, N=N, hint=1, act="f32")


def test_conv_of_many_pieces():
    sel_check("conv", [700, 1, 2000], [1, 0, 0], 264, act="bf16")


@BOTH
def test_without_skip_weight_gate_or_bias(what):
    run = SelRun([20, 1, 3], [1, 0, 1], 16, act="f32", bias=False, gate=False, skip_weight=False)
    run.dt_bias = run.dev[4] = None
    run.run_conv() if what == "conv" else run.run_scan()
    run.check(what)


@BOTH
@pytest.mark.parametrize("blocks,hint", [([1, 0, 2, 3], 0), ([1, 9, 2, 3], 0), ([1, -1, 2, 3], 0),
                                         ([1, 2, 2, 3], 0), ([4, 5, 6, 1], 4), ([-5, 0, 99, 99], 0)])
def test_bad_indices_leave_their_sequences_out(what, blocks, hint):
    for n in (4, 300):  # listed by every CTA, and by the planning kernel
        lens = [3, 4, 6, 1] + [0] * (n - 4)
        sel_check(what, lens, [1] * n, 32, blocks=blocks + [-1] * (n - 4), num_blocks=8, hint=hint)


@BOTH
@pytest.mark.parametrize("cu", [[1, 3, 6], [0, 4, 3], [0, 3, 7], [0, -1, 6], [0, 7, 6]])
def test_bad_cu_seqlens_leave_the_batch_out(what, cu):
    for n in (2, 301):
        run = SelRun([3, 3] + [0] * (n - 2), [1] * n, 32)
        run.cu = cu + [cu[-1]] * (n - 2)
        run.cu_d = torch.tensor(run.cu, dtype=torch.int32, device="cuda")
        run.run_conv() if what == "conv" else run.run_scan()
        torch.cuda.synchronize()
        assert run.pool.error_flags() == 1
        assert (run.out == SENTINEL).all() and torch.equal(run.mem, run.before)


@BOTH
def test_nothing_to_do(what):
    run = SelRun([0, 0], [1, 1], 32)
    run.run_conv() if what == "conv" else run.run_scan()
    run.check(what)
    run.T = run.N = 0
    run.run_conv() if what == "conv" else run.run_scan()
    run.check(what)


@BOTH
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_values_stay_in_their_sequence_and_behind_their_token(what, value):
    lens, past = [40, 37, 1, 3, 1], [1, 0, 1, 0, 1]

    def put(host, run):
        for t in host.values():
            t[run.cu[1] + 20] = value
            t[run.cu[3]] = value
            t[run.cu[-1]:] = value

    a, b = SelRun(lens, past, 48, rows_after=2), SelRun(lens, past, 48, rows_after=2, values=put)
    for r in (a, b):
        r.run_conv() if what == "conv" else r.run_scan()
    torch.cuda.synchronize()
    keep = [slice(a.cu[0], a.cu[1]), slice(a.cu[1], a.cu[1] + 20), slice(a.cu[2], a.cu[3]),
            slice(a.cu[4], a.cu[5])]
    for rows in keep:
        assert torch.isfinite(b.out[rows]).all() and torch.equal(bits(a.out[rows]), bits(b.out[rows]))
    for s in (0, 2, 4):
        assert torch.equal(bits(a.ssm[a.blk[s]]), bits(b.ssm[b.blk[s]]))
    if what == "conv":  # a convolution forgets
        assert torch.equal(bits(a.out[a.cu[1] + 24:a.cu[2]]), bits(b.out[a.cu[1] + 24:a.cu[2]]))


def test_scan_extremes():
    """No decay, total decay, steps from nothing to large, an infinite state."""
    A_log = torch.tensor([-np.inf, -20.0, 0.0, 5.0, 60.0, 88.0, 100.0, -5.0] * 2).float().repeat(16, 1)

    def put(host, run):
        host["dt"][3] = -30.0
        host["dt"][4] = 30.0

    for lens in ([9, 40], [1, 1]):
        sel_check("scan", lens, [1, 1], 16, act="f32", A_log=A_log, values=put if lens[0] > 4 else None)
    run = SelRun([5, 1], [1, 1], 16, act="f32")
    for s in range(2):
        run.past_ssm[s, 3, 5] = float("inf")
        run.ssm[run.blk[s], 3, 5] = float("inf")
    run.before = run.mem.clone()
    run.run_scan()
    torch.cuda.synchronize()
    for s in range(2):
        assert run.ssm[run.blk[s], 3, 5] == float("inf")
        assert torch.isfinite(run.ssm[run.blk[s], 4:]).all()


def test_slow_decay_keeps_the_state_over_many_tokens():
    """Decays within 1e-4 of 1 over 3,000 tokens: the fp32 form's roundings add
    up like a walk (twice its rms: sqrt(n) 2^-24 / sqrt(3) of the state's size for
    the state's own and as much for the decay's), not like their sum."""
    n = 3000
    run = SelRun([n], [1], 64, act="f32", A_log=torch.full((64, 16), 0.0), dt_bias=torch.full((64,), -9.5))
    run.run_scan()
    h = run.past_ssm.double().cpu()[0]
    x = {k: v.double() for k, v in run.host.items()}
    step = torch.nn.functional.softplus(x["dt"] - 9.5)
    for t in range(n):
        h = h * torch.exp(-step[t])[:, None] + (step[t] * x["u"][t])[:, None] * x["B"][t]
    err = (run.ssm[run.blk[0]].double().cpu() - h).norm() / h.norm()
    assert err <= 4 * n ** 0.5 * 2.0 ** -24 / 3 ** 0.5, err


@BOTH
def test_split_calls_equal_one(what):
    """A prompt in two calls and a token after it: as the whole in one."""
    n = 50
    whole = SelRun([n], [0], 40, act="f32", seed=7)
    parts = SelRun([n], [0], 40, act="f32", seed=7)
    go = lambda r: r.run_conv() if what == "conv" else r.run_scan()  # noqa: E731
    go(whole)
    for lo, hi in ((0, 20), (20, 21), (21, 49), (49, 50)):
        v = SelRun([hi - lo], [lo > 0], 40, act="f32", seed=7)
        v.pool, v.blk_d = parts.pool, parts.blk_d
        for name in ("x", "z", "u", "dt", "B", "Cm"):
            setattr(v, name, getattr(parts, name)[lo:hi])
        v.dev, v.out, v.T = parts.dev, parts.out[lo:hi], hi - lo
        go(v)
    torch.cuda.synchronize()
    # the same roundings whatever the split, but for the two forms' order of sums
    tol = 0 if what == "conv" else 2.0 ** -18
    assert (whole.out - parts.out).abs().max() <= tol * whole.out.abs().max()
    assert (whole.ssm[whole.blk[0]] - parts.ssm[parts.blk[0]]).abs().max() <= 2.0 ** -18 * 10


@BOTH
def test_captured_and_replayed(what):
    """One graph over batches of other compositions written into its buffers."""
    run = SelRun([30, 1, 20, 1], [1, 1, 0, 1], 72, seed=3)
    go = lambda: run.run_conv() if what == "conv" else run.run_scan()  # noqa: E731
    go()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    for lens in ([30, 1, 20, 1], [1, 50, 0, 1], [13, 13, 13, 13]):
        cu = torch.tensor([0] + np.cumsum(lens).tolist(), dtype=torch.int32, device="cuda")
        run.cu_d.copy_(cu)
        run.mem.copy_(run.before)
        run.out.fill_(SENTINEL)
        graph.replay()
        torch.cuda.synchronize()
        out, mem = run.out.clone(), run.mem.clone()
        run.mem.copy_(run.before)
        run.out.fill_(SENTINEL)
        go()
        torch.cuda.synchronize()
        assert torch.equal(out, run.out) and torch.equal(mem, run.mem), lens
        assert run.pool.error_flags() == 0


@BOTH
def test_another_stream(what):
    run = SelRun([30, 1, 20], [1, 1, 0], 72, seed=3)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run.run_conv() if what == "conv" else run.run_scan()
    side.synchronize()
    run.check(what)


def test_host_refusals():
    run = SelRun([3, 1], [1, 0], 32)
    lib, w = binding.load(), binding.SelWeights(run.dev[2].data_ptr(), None, None)
    P = lambda t: t.data_ptr()  # noqa: E731

    def conv(layer=0, x=P(run.x), ldx=64, cu=P(run.cu_d), wt=P(run.dev[0]), out=P(run.out), ldo=40, T=4, N=2,
             hint=0, pool=run.pool):
        return lib.gdn_sel_conv_varlen_forward(pool.handle, layer, x, ldx, cu, P(run.blk_d), P(run.past_d), wt,
                                               None, out, ldo, T, N, hint, None)

    def scan(u=P(run.u), ldu=64, B=P(run.B), ldb=40, y=P(run.out), T=4, N=2, weights=w, z=P(run.z), ldz=64):
        return lib.gdn_sel_scan_varlen_forward(
            run.pool.handle, 0, u, ldu, P(run.dt), 64, B, ldb, P(run.Cm), 40, z, ldz, P(run.cu_d), P(run.blk_d),
            P(run.past_d), ctypes.byref(weights) if weights else None, y, 40, T, N, 0, None)

    lin = binding.LinPool(4, 1, 2, 32, "bf16")
    assert [conv(layer=1), conv(layer=-1), conv(T=-1), conv(N=-1), conv(hint=-1), conv(N=0), conv(ldx=24),
            conv(ldo=1 << 39)] == [-3] * 8
    assert [conv(x=None), conv(out=None), conv(cu=None), conv(wt=None)] == [-1] * 4
    assert [conv(x=P(run.x) + 2), conv(ldx=66), conv(ldo=41), conv(wt=P(run.dev[0]) + 2)] == [-4] * 4
    assert conv(pool=lin) == -2 and conv(T=0, N=0) == 0
    assert [scan(u=None), scan(B=None), scan(weights=None), scan(weights=binding.SelWeights(None, None, None))] == [-1] * 4
    assert [scan(u=P(run.u) + 4), scan(ldb=36), scan(ldz=60), scan(y=P(run.out) + 2)] == [-4] * 4
    assert [scan(ldu=24), scan(ldb=8), scan(ldz=16), scan(N=0)] == [-3] * 4
    with pytest.raises(ValueError):
        binding.sel_scan_varlen_forward(run.pool, 0, run.u.float(), run.dt, run.B, run.Cm, None, run.cu_d, run.blk_d,
                                        run.past_d, run.dev[2], None, None, run.out, 4, 2)
    with pytest.raises(ValueError):
        binding.sel_conv_varlen_forward(run.pool, 0, run.x, run.cu_d[:2], run.blk_d, run.past_d, run.dev[0], None,
                                        run.out, 4, 2)
    torch.cuda.synchronize()
    assert (run.out == SENTINEL).all() and torch.equal(run.mem, run.before)


def test_block_operations_move_both_states():
    run = SelRun([1, 1], [1, 1], 32, num_blocks=8)
    src = torch.tensor([run.blk[0]], dtype=torch.int32, device="cuda")
    free = [b for b in range(1, 8) if b not in run.blk]
    run.pool.copy_blocks(src, torch.tensor(free[:1], dtype=torch.int32, device="cuda"))
    run.pool.reserve(100)
    torch.cuda.synchronize()
    page = run.mem.view(8, -1)
    assert torch.equal(page[free[0]], page[run.blk[0]])


# Long sequences of few channels: their segments run side by side, from states that
# a pass before them finds.
SEGMENTED = [([900], [0]), ([900], [1]), ([700, 1, 0, 450, 2, 64, 65], [1, 1, 1, 0, 1, 0, 1]),
             ([1, 1, 230, 1, 640], [0, 1, 0, 1, 1])]


@pytest.mark.parametrize("lens,past", SEGMENTED)
@pytest.mark.parametrize("act,N", [("f32", 16), ("bf16", 16), ("f32", 32), ("bf16", 64)])
@pytest.mark.parametrize("channels", [8, 136])
def test_segments_of_long_sequences(lens, past, act, N, channels):
    run = sel_check("scan", lens, past, channels, N=N, act=act, gate=N != 32, skip_weight=N != 64, seed=N,
                    rows_after=2, segment=64)
    assert run.pool.error_flags() == 0


def test_segments_with_other_layers_and_a_long_sequence():
    sel_check("scan", [5000, 300], [1, 0], 264, act="bf16", num_layers=2, layer=1, segment=192)


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_values_reach_no_segment_before_them_and_no_other_sequence(value):
    lens = [700, 300, 1]

    def put(host, run):
        for t in host.values():
            t[500] = value
        host["u"][700 + 299] = value

    a, b = SelRun(lens, [1, 0, 1], 48), SelRun(lens, [1, 0, 1], 48, values=put)
    for r in (a, b):
        r.run_scan()
    torch.cuda.synchronize()
    for rows in (slice(0, 500), slice(700, 999), slice(1000, 1001)):
        assert torch.isfinite(b.out[rows]).all() and torch.equal(bits(a.out[rows]), bits(b.out[rows]))
    assert torch.equal(bits(a.ssm[a.blk[2]]), bits(b.ssm[b.blk[2]]))
    assert not torch.isfinite(b.out[500:564]).any()


def test_segments_in_two_graphs_on_one_pool():
    """Both use the pool's room for states, one behind the other."""
    runs = [SelRun([800, 1, 300], [1, 1, 0], 72, seed=3, blocks=[3, 1, 2]), SelRun([260, 640], [0, 1], 72, seed=4)]
    first, second = runs
    second.pool, second.blk_d = first.pool, torch.tensor([4, 5], dtype=torch.int32, device="cuda")
    graphs = []
    for r in runs:
        r.run_scan()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            r.run_scan()
        graphs.append(g)
    start = first.before.clone()
    start.view(6, -1)[4:] = start.view(6, -1)[1:3].flip(0)
    want = []
    for r in runs:
        first.mem.copy_(start)
        r.run_scan()
        torch.cuda.synchronize()
        want.append(r.out.clone())
    first.mem.copy_(start)
    for r in runs:
        r.out.fill_(SENTINEL)
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    for r, w in zip(runs, want):
        assert torch.equal(bits(r.out), bits(w))


@pytest.mark.parametrize("n", [79_030, 77_824, 77_825])
def test_lengths_whose_segments_just_fit(n):
    """A share of the tokens that is no whole number of segments: every token is in one."""
    run = SelRun([n], [1], 8, act="f32", seed=1, gate=False)
    run.run_scan()
    other, out = 2 if run.blk[0] != 2 else 1, run.out.clone()
    run.ssm[other] = run.past_ssm[0].cuda()
    for lo, hi in ((0, n // 2), (n // 2, n)):
        part = SelRun([hi - lo], [1], 8, act="f32", seed=1, gate=False)
        part.pool, part.blk_d, part.dev, part.T = run.pool, torch.tensor([other], **I32), run.dev, hi - lo
        for name in ("u", "dt", "B", "Cm"):
            setattr(part, name, getattr(run, name)[lo:hi])
        part.out = out[lo:hi]
        part.run_scan()
    torch.cuda.synchronize()
    # (the same sums in another order)
    assert (run.out - out).abs().max() <= 2.0 ** -16 * run.out.abs().max()
    a, b = run.ssm[run.blk[0]], run.ssm[other]
    assert (a - b).abs().max() <= 2.0 ** -16 * a.abs().max()
