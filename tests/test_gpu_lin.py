"""GPU parity of gdn_lin_varlen_forward (linear attention with a decay per
head) with the fp64 recurrence: types, head layouts, lengths from none to many
chunks, pitches, decays from none to total, padding and bad indices, values
that may not leak, streams, graphs and several calls on one pool."""
import ctypes

import numpy as np
import pytest
import torch

from continuous_linear_attention_gb300 import binding
from lin_check import SENTINEL, LinRun, check, run_and_check

pytestmark = pytest.mark.gpu

FORMS = [("f32", 32), ("f32", 64), ("f32", 128), ("bf16", 32), ("bf16", 64), ("bf16", 128)]


@pytest.mark.parametrize("act,d", FORMS)
def test_short_ragged_batch(act, d):
    run_and_check([5, 1, 0, 33, 1, 16, 17], [1, 0, 1, 1, 1, 0, 0], 6, 3, d, act,
                  tensor_cores=act == "bf16" and d == 128)


@pytest.mark.parametrize("act,d", FORMS)
@pytest.mark.parametrize("H,Hkv", [(1, 1), (8, 1), (5, 5)])
def test_decode_batch(act, d, H, Hkv):
    run_and_check([1] * 9, [1, 1, 0, 1, 1, 0, 1, 1, 1], H, Hkv, d, act, hint=1, seed=H)


@pytest.mark.parametrize("lens", [[1], [2], [31], [32], [33], [64], [65], [127], [128], [129],
                                  [255], [256], [257], [300, 1, 129, 64], [700]])
@pytest.mark.parametrize("past", [0, 1])
def test_prompts_around_the_chunk_edges(lens, past):
    run_and_check(lens, [past] * len(lens), 4, 2, 128, "bf16", tensor_cores=True, seed=len(lens))


@pytest.mark.parametrize("act,d", [("bf16", 128), ("f32", 64)])
def test_decays_from_none_to_total(act, d):
    decay = [0.0, -1e-5, -0.02, -0.3, -2.0, -30.0, -200.0, -float("inf")]
    run, _ = run_and_check([150, 40, 1], [1, 0, 1], 8, 4, d, act, log_decay=decay,
                           tensor_cores=act == "bf16")
    # a head without memory answers with its own token alone
    x = run.x.double()
    q, k, v = (p.unflatten(1, (-1, d)) for p in x.split([8 * d, 4 * d, 4 * d], 1))
    want = (q[:, 7] * k[:, 3]).sum(1, keepdim=True) * v[:, 3] * run.scale
    got = run.out[:, 7].double().cpu()
    assert (got - want).norm() <= (2e-6 if act == "f32" else 2.0 ** -7) * want.norm()


def fp32_walk(n):
    """Twice the rms of n fp32 roundings of a slowly changing value: each is
    uniform in half a step, at most 2^-24 relative, so 2^-24 / sqrt(3) rms, and
    n independent ones add as sqrt(n).  (n = 2100: 3.2e-6.  A decay held as one
    fp32 number alone would be off by up to n 2^-25 = 6e-5.)"""
    return 2 * n ** 0.5 * 2.0 ** -24 / 3 ** 0.5


def test_slow_decay_keeps_the_state_over_many_chunks():
    """e^g within 1e-4 of 1: the past and everything since stay in the state."""
    _, errs = run_and_check([2100, 700], [1, 1], 2, 1, 128, "bf16", log_decay=[-1e-4, -1e-6],
                            tensor_cores=True)
    assert errs["state"] <= fp32_walk(2100), errs


def test_slow_decay_in_the_serial_form():
    _, errs = run_and_check([1500], [1], 2, 2, 64, "f32", log_decay=[-1e-4, -3e-3])
    assert errs["state"] <= fp32_walk(1500) and errs["out"] <= fp32_walk(1500), errs


@pytest.mark.parametrize("lens", [[1] * 5, [140, 3, 40]])
def test_dense_tensors_and_wider_rows_give_the_same_bits(lens):
    a = LinRun(lens, [1] * len(lens), 4, 4, 128, "bf16", seed=5)
    b = LinRun(lens, [1] * len(lens), 4, 4, 128, "bf16", seed=5, dense=True)
    wide = torch.full((a.T, 4 * 128 + 64), SENTINEL, dtype=torch.bfloat16, device="cuda")
    b.out = wide[:, 32:32 + 512].unflatten(1, (4, 128))
    a.run()
    b.run()
    torch.cuda.synchronize()
    assert torch.equal(a.out, b.out) and torch.equal(a.mem, b.mem)
    assert (wide[:, :32] == SENTINEL).all() and (wide[:, 544:] == SENTINEL).all()
    check(a, tensor_cores=True)


@pytest.mark.parametrize("act,d", [("f32", 32), ("bf16", 128)])
@pytest.mark.parametrize("blocks,hint", [
    ([3, 9, 5, 1], 0), ([3, 0, 5, 1], 0), ([3, 5, 5, 1], 0), ([3, -1, 5, -7], 0), ([3, 2, 5, 1], 40),
])
def test_padding_and_bad_indices(act, d, blocks, hint):
    run_and_check([4, 60, 3, 1], [1, 1, 0, 1], 2, 1, d, act, blocks=blocks, num_blocks=8, hint=hint,
                  rows_after=3, tensor_cores=act == "bf16")


@pytest.mark.parametrize("cu", [[1, 5, 8], [0, 9, 8], [0, 5, 7]])
def test_bad_cu_seqlens_skip_the_batch(cu):
    run = LinRun([5, 3], [1, 1], 2, 2, 64, "bf16")
    before = run.mem.clone()
    run.cu = cu
    run.cu_d.copy_(torch.tensor(cu, dtype=torch.int32))
    run.run()
    torch.cuda.synchronize()
    check(run)
    assert torch.equal(run.mem, before)


@pytest.mark.parametrize("act,d", [("f32", 32), ("bf16", 128)])
def test_many_sequences_take_the_scheduler(act, d):
    """More sequences than the kernels check by themselves, with empty ones,
    padding, one block named twice and a few prompts."""
    rng = np.random.default_rng(1)
    lens = rng.choice([0, 1, 1, 1, 2], 700).tolist()
    lens[11], lens[500] = 70, 40
    lens[3] = lens[4] = 1
    blocks = (rng.permutation(900)[:700] + 1).tolist()
    blocks[4] = blocks[3]
    blocks[20] = -1
    run_and_check(lens, rng.integers(0, 2, 700).tolist(), 1, 1, d, act, blocks=blocks,
                  num_blocks=901, tensor_cores=act == "bf16")


@pytest.mark.parametrize("act,d", [("f32", 64), ("bf16", 128)])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_values_of_later_tokens_and_neighbours_do_not_leak(act, d, value):
    """A non-finite v, k or q of one token reaches no earlier row of its
    sequence and no row of another one."""
    at = 150

    def put(x, run):
        w, kv = run.H * run.d, run.Hkv * run.d
        x[at, w + kv:] = value           # v, in the middle of the first sequence
        x[260, w:w + kv] = value         # k of the second one's last token
        x[261, :w] = value               # q of the third one's first token

    run = LinRun([200, 61, 40, 1], [1, 1, 1, 1], 4, 2, d, act, values=put, seed=8)
    run.run()
    torch.cuda.synchronize()
    out, states = run.expected()
    got = run.out.double().cpu().numpy()
    tol = 1e-5 if act == "f32" else 2.0 ** -7
    for rows in (slice(0, at), slice(200, 260), slice(262, 302)):
        assert np.isfinite(got[rows]).all()
        assert np.linalg.norm(got[rows] - out[rows]) <= tol * np.linalg.norm(out[rows])
    for rows in (slice(at, 200), slice(260, 261), slice(261, 262)):
        assert not np.isfinite(got[rows]).any(), rows
    view = run.view[0].cpu().double().numpy()
    for s, fine in enumerate((False, False, True, True)):
        st = view[run.blk[s]]
        assert np.isfinite(st).all() == fine
        if fine:
            assert np.linalg.norm(st - states[s]) <= 1e-5 * np.linalg.norm(states[s])
    assert run.pool.error_flags() == 0


@pytest.mark.parametrize("size", [1e-30, 1e4, 1e15])
def test_values_of_any_size(size):
    """bf16 has fp32's range: products of 1e15 have to come out as they are."""
    def put(x, run):
        x *= size if size < 1 else size ** 0.5

    run = LinRun([200, 3], [0, 0], 2, 1, 128, "bf16", values=put)
    run.run()
    torch.cuda.synchronize()
    check(run, tensor_cores=True)


def test_empty_calls():
    run = LinRun([0, 0], [1, 1], 2, 2, 64, "bf16")
    before = run.mem.clone()
    run.run()
    binding.lin_varlen_forward(run.pool, 0, run.q, run.k, run.v, run.cu_d[:1], run.blk_d[:0],
                               run.past_d[:0], run.decay_d, run.out, 0, 0)
    torch.cuda.synchronize()
    assert torch.equal(run.mem, before) and run.pool.error_flags() == 0


def test_requests_over_several_calls_equal_one_pass():
    """Prompts, drafted tokens and single tokens of four requests over six
    calls on one pool, against one pass over the whole sequences."""
    rng = np.random.default_rng(5)
    H, d, n = 4, 128, 4
    calls = [[300, 5, 1, 40], [1, 1, 1, 1], [130, 0, 4, 1], [1, 64, 1, 33], [0, 1, 1, 129], [2, 2, 2, 2]]
    whole = LinRun(np.sum(calls, axis=0).tolist(), [0] * n, H, 2, d, "bf16", seed=9)
    outs = [[] for _ in range(n)]
    at = [whole.cu[s] for s in range(n)]
    for i, lens in enumerate(calls):
        rows = np.concatenate([np.arange(at[s], at[s] + lens[s]) for s in range(n)]).tolist()
        cu = torch.tensor([0] + np.cumsum(lens).tolist(), dtype=torch.int32, device="cuda")
        out = torch.empty(len(rows), H, d, dtype=torch.bfloat16, device="cuda")
        past = torch.tensor([int(at[s] > whole.cu[s]) for s in range(n)], dtype=torch.uint8, device="cuda")
        binding.lin_varlen_forward(whole.pool, 0, whole.q[rows], whole.k[rows], whole.v[rows], cu,
                                   whole.blk_d, past, whole.decay_d, out, len(rows), n,
                                   scale=whole.scale, max_seqlen_hint=max(lens))
        for s, part in enumerate(out.split(lens)):
            outs[s].append(part)
            at[s] += lens[s]
    whole.out = torch.cat([p for s in range(n) for p in outs[s]])
    torch.cuda.synchronize()
    check(whole, tensor_cores=True)


@pytest.mark.parametrize("lens", [[1] * 6, [300, 1, 40, 2]])
def test_captured_calls_replay_over_new_batches(lens):
    """One graph, replayed over another composition written into its inputs,
    gives the bits of an eager call."""
    a = LinRun(lens, [1] * len(lens), 4, 2, 128, "bf16", seed=2)
    b = LinRun(lens[::-1], [0, 1] * (len(lens) // 2), 4, 2, 128, "bf16", seed=3, blocks=a.blk)
    a.run()  # loads the kernels
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.run(torch.cuda.current_stream())
    for x, y in ((a.q._base, b.q._base), (a.cu_d, b.cu_d), (a.past_d, b.past_d)):
        x.copy_(y)
    mem = b.mem.clone()
    a.mem.copy_(mem)
    graph.replay()
    b.run()
    torch.cuda.synchronize()
    assert torch.equal(a.out, b.out) and torch.equal(a.mem, b.mem)
    check(b, tensor_cores=True)


def test_another_stream_and_its_order():
    """A call on a stream of its own reads inputs that stream's earlier work
    has written."""
    run = LinRun([1] * 4, [1] * 4, 4, 4, 128, "bf16", seed=6)
    good = run.q._base.clone()
    run.q._base.zero_()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(2_000_000)
        run.q._base.copy_(good)
        run.run()
        run.q._base.zero_()
    torch.cuda.synchronize()
    check(run)


def test_layers_have_their_own_blocks_and_error_words():
    run = LinRun([40, 1], [1, 1], 2, 1, 128, "bf16", blocks=[1, 9], num_blocks=4, num_layers=3, layer=2)
    before = run.view.clone()
    run.run()
    torch.cuda.synchronize()
    assert torch.equal(before[:2], run.view[:2])
    assert run.pool.error_flags(layer=1) == 0 and run.pool.error_flags(layer=2, reset=False) == 0x2
    check(run, tensor_cores=True, before=before)


def test_equal_calls_give_equal_bits():
    runs = [LinRun([513, 1, 70], [1, 1, 0], 8, 2, 128, "bf16", seed=4) for _ in range(2)]
    for r in runs:
        r.run()
    torch.cuda.synchronize()
    assert torch.equal(runs[0].out, runs[1].out) and torch.equal(runs[0].mem, runs[1].mem)


def test_offsets_past_32_bits():
    """Rows whose element offset passes 2^32: a pitch of 2^31 elements would
    need too much memory, so the pool's last block lies 9 GB into it."""
    H, d, nb = 64, 128, 2200
    run = LinRun([1, 40], [1, 1], H, 1, d, "bf16", blocks=[nb - 1, nb - 2], num_blocks=nb)
    run.run()
    torch.cuda.synchronize()
    check(run, tensor_cores=True)


def test_refusals():
    lib = binding.load()
    run = LinRun([3, 1], [1, 1], 4, 2, 64, "bf16")
    q, k, v, o = (t.data_ptr() for t in (run.q, run.k, run.v, run.out))
    ld = run.q.stride(0)

    def call(layer=0, q=q, k=k, v=v, ldq=ld, ldk=ld, ldv=ld, kv=2, cu=run.cu_d.data_ptr(),
             decay=run.decay_d.data_ptr(), o=o, ldo=256, T=4, N=2, hint=0):
        return lib.gdn_lin_varlen_forward(run.pool.handle, layer, q, k, v, ldq, ldk, ldv, kv, cu,
                                          run.blk_d.data_ptr(), run.past_d.data_ptr(), decay, 1.0, o,
                                          ldo, T, N, hint, None)

    before = run.mem.clone()
    assert call(layer=1) == call(layer=-1) == call(T=-1) == call(N=-1) == call(hint=-1) == -3
    assert call(kv=0) == call(kv=3) == call(kv=8) == -2
    assert call(q=None) == call(v=None) == call(cu=None) == call(decay=None) == call(o=None) == -1
    assert call(q=q + 2) == call(k=k + 8) == call(o=o + 4) == call(ldv=ld + 1) == call(ldo=257) == -4
    assert call(ldq=248) == call(ldo=248) == call(ldk=120) == call(T=1, N=0) == -3
    gdn = binding.Pool(4, 1, 2, 4, 64, 64, 4, "bf16")
    assert lib.gdn_lin_varlen_forward(gdn.handle, 0, q, k, v, ld, ld, ld, 2, run.cu_d.data_ptr(),
                                      run.blk_d.data_ptr(), run.past_d.data_ptr(),
                                      run.decay_d.data_ptr(), 1.0, o, 256, 4, 2, 0, None) == -2
    w = binding.Weights(q, q, q)
    assert lib.gdn_varlen_forward(run.pool.handle, 0, q, q, q, run.cu_d.data_ptr(),
                                  run.blk_d.data_ptr(), run.past_d.data_ptr(), ctypes.byref(w), o, 4,
                                  2, 0, None) == -2
    ws = binding.SsdWeights(q, q, q, q)
    assert lib.gdn_ssd_varlen_forward(run.pool.handle, 0, q, q, run.cu_d.data_ptr(),
                                      run.blk_d.data_ptr(), run.past_d.data_ptr(), ctypes.byref(ws), o,
                                      4, 2, 0, None) == -2
    run.pool.reserve(100)
    torch.cuda.synchronize()
    assert torch.equal(run.mem, before) and (run.out == SENTINEL).all()
    for bad in (dict(q=run.q.float()), dict(k=run.k[:, :, :32]), dict(out=run.out[:, :2]),
                dict(v=run.v.transpose(0, 1)), dict(q=run.q[:3])):
        kw = dict(q=run.q, k=run.k, v=run.v, out=run.out) | bad
        with pytest.raises(ValueError):
            binding.lin_varlen_forward(run.pool, 0, kw["q"], kw["k"], kw["v"], run.cu_d, run.blk_d,
                                       run.past_d, run.decay_d, kw["out"], 4, 2)


@pytest.mark.parametrize("act,d", FORMS[:-1])
@pytest.mark.parametrize("lens,H,Hkv", [([700], 2, 1), ([3, 900, 1, 0, 64, 385], 3, 3), ([257, 260], 1, 1)])
def test_long_sequences_of_few_heads_are_split(act, d, lens, H, Hkv):
    """The token-serial form over segments side by side: their own states
    first, then the outputs from the states at their starts."""
    _, errs = run_and_check(lens, [1, 0] * (len(lens) // 2) + [1] * (len(lens) % 2), H, Hkv, d, act,
                            log_decay=[-1e-3, -0.05, 0.0][:H], seed=d)
    if act == "f32":
        assert errs["out"] <= fp32_walk(max(lens)) and errs["state"] <= fp32_walk(max(lens)), errs


def test_a_split_call_skips_what_it_should():
    run_and_check([400, 300, 2, 350], [1, 1, 0, 1], 2, 1, 64, "f32", blocks=[3, 9, -1, 3], num_blocks=8,
                  rows_after=2)
    run_and_check([400, 30, 2, 350], [1, 1, 0, 1], 2, 1, 32, "bf16", blocks=[3, 2, -1, 5], num_blocks=8,
                  hint=380)


@pytest.mark.parametrize("act,d", [("f32", 64), ("bf16", 128)])
@pytest.mark.parametrize("n", [6, 600])
def test_a_hint_of_one_flags_what_is_longer(act, d, n):
    """Few sequences check themselves, many are listed; either way one of two
    tokens, a padding entry and a block named twice are left out."""
    lens = [1] * n
    lens[2], lens[4] = 2, 0
    blocks = list(range(n + 1, 1, -1))
    blocks[1], blocks[5] = -1, blocks[0]
    run_and_check(lens, [1, 0] * (n // 2), 2, 1, d, act, blocks=blocks, num_blocks=n + 2, hint=1, rows_after=1)


@pytest.mark.parametrize("lens,H,Hkv", [([1030], 1, 1), ([1500, 1, 0, 40, 1153], 3, 1), ([4000, 1024], 2, 2)])
@pytest.mark.parametrize("past", [0, 1])
def test_long_prompts_of_few_heads_are_split(lens, H, Hkv, past):
    """The chunked form over segments side by side, with decays from none to
    more than a segment remembers."""
    run_and_check(lens, [past] * len(lens), H, Hkv, 128, "bf16", log_decay=[-0.004, 0.0, -3.0][:H],
                  tensor_cores=True, seed=H)


@pytest.mark.parametrize("blocks,hint", [([3, 9, 5, 1], 0), ([3, -1, 5, 3], 0), ([3, 0, 5, 1], 1200)])
def test_a_split_prompt_batch_skips_what_it_should(blocks, hint):
    run_and_check([1100, 1300, 3, 1150], [1, 1, 0, 1], 2, 1, 128, "bf16", blocks=blocks, num_blocks=8,
                  hint=hint, rows_after=2, tensor_cores=True)


@pytest.mark.parametrize("act,d,at", [("bf16", 128, 700), ("bf16", 128, 1410), ("f32", 32, 700)])
def test_values_that_are_not_finite_in_a_split_sequence(act, d, at):
    """Earlier rows of every segment and the other columns come out as if the
    value were a number."""
    col = 5  # of v

    def put(x, run):
        x[at, (run.H + run.Hkv) * d + col] = float("inf")

    run = LinRun([1420, 3], [1, 1], 2, 1, d, act, values=put, log_decay=[-0.01, -0.2], dense=True)
    run.run()
    torch.cuda.synchronize()
    assert run.pool.error_flags() == 0
    run.x[at, (run.H + run.Hkv) * d + col] = 0.0
    out, states = run.expected()
    got = run.out.double().cpu().numpy()
    view = run.view[0].cpu().double().numpy()[run.blk[0]]
    tol, st_tol = (1e-5, 1e-5) if act == "f32" else (2.0 ** -7, 1e-5)
    fine = np.ones(d, bool)
    fine[col] = False
    n = np.linalg.norm
    assert n(got[:at] - out[:at]) <= tol * n(out[:at])
    assert n(got[at:, :, fine] - out[at:, :, fine]) <= tol * n(out[at:, :, fine])
    assert n(view[..., fine] - states[0][..., fine]) <= st_tol * n(states[0][..., fine])
    assert not np.isfinite(got[at:1420, :, col]).any() and not np.isfinite(view[..., col]).any()


@pytest.mark.parametrize("act,d,lens", [("bf16", 128, [1500, 1, 40, 3]), ("f32", 32, [900, 1, 40, 3])])
def test_a_captured_split_call_replays_over_a_batch_that_is_not_split(act, d, lens):
    a = LinRun(lens, [1, 0, 1, 1], 2, 1, d, act, seed=2)
    short = [len_ for len_ in (a.T // 4,) * 3] + [a.T - 3 * (a.T // 4)]
    b = LinRun(short, [0, 1, 0, 1], 2, 1, d, act, seed=3, blocks=a.blk)
    before = b.mem.clone()
    a.run()
    torch.cuda.synchronize()
    check(a, tensor_cores=act == "bf16")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.run(torch.cuda.current_stream())
    for x, y in ((a.q._base, b.q._base), (a.cu_d, b.cu_d), (a.past_d, b.past_d), (a.mem, before)):
        x.copy_(y)
    graph.replay()
    b.run()
    torch.cuda.synchronize()
    assert torch.equal(a.out, b.out) and torch.equal(a.mem, b.mem)
    check(b, tensor_cores=act == "bf16")


def test_two_pools_on_two_streams_at_once():
    runs = [LinRun([1300, 1, 200], [1, 1, 0], 2, 2, 128, "bf16", seed=11),
            LinRun([700, 2, 90], [0, 1, 1], 3, 1, 64, "f32", seed=12)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    for r, s in zip(runs, streams):
        r.run(s)
    torch.cuda.synchronize()
    for r in runs:
        check(r, tensor_cores=r.act == "bf16")


@pytest.mark.parametrize("lens", [[1, 39], [20] * 2])
def test_row_offsets_past_32_bits(lens):
    """q, k, v and out as columns of rows of 2^28 elements: the last row starts
    beyond 2^33 elements."""
    run = LinRun(lens, [1] * len(lens), 2, 1, 128, "bf16", seed=7)
    wide = torch.empty(run.T, 2 ** 28, dtype=torch.bfloat16, device="cuda")
    for name, x, at in (("q", run.q, 0), ("k", run.k, 2 ** 27), ("v", run.v, 2 ** 28 - 512),
                        ("out", run.out, 2 ** 28 - 256)):
        cols = wide[:, at:at + x.shape[1] * 128]
        cols.copy_(x.flatten(1))
        setattr(run, name, cols.unflatten(1, (-1, 128)))
    run.run()
    torch.cuda.synchronize()
    check(run, tensor_cores=True)


def test_has_past_is_any_value_but_zero():
    run = LinRun([1, 40, 3], [1, 1, 0], 2, 1, 128, "bf16")
    run.past_d.copy_(torch.tensor([255, 2, 0], dtype=torch.uint8))
    run.run()
    torch.cuda.synchronize()
    check(run, tensor_cores=True)


@pytest.mark.parametrize("act,d", [("f32", 64), ("bf16", 128)])
@pytest.mark.parametrize("n", [3, 700])
def test_bad_cu_seqlens_whose_differences_wrap(act, d, n):
    """No difference of these is negative in 32 bits."""
    lens = [300, 300, 300] + [0] * (n - 3)
    run = LinRun(lens, [1] * n, 1, 1, d, act, num_blocks=n + 1)
    before = run.mem.clone()
    run.cu = [0, 2_000_000_000, -2_000_000_000] + [run.T] * (n - 2)
    run.cu_d.copy_(torch.tensor(run.cu, dtype=torch.int32))
    run.run()
    torch.cuda.synchronize()
    check(run)
    assert torch.equal(run.mem, before)


@pytest.mark.parametrize("hint", [0, 1])
def test_slow_decay_keeps_the_state_over_many_single_tokens(hint):
    """One token per call, in the kernel for single tokens and in the one for
    any length."""
    run = LinRun([1200], [1], 2, 1, 64, "f32", log_decay=[-1e-4, -1e-6])
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    for t in range(run.T):
        binding.lin_varlen_forward(run.pool, 0, run.q[t:], run.k[t:], run.v[t:], cu, run.blk_d, run.past_d,
                                   run.decay_d, run.out[t:], 1, 1, scale=run.scale, max_seqlen_hint=hint)
    torch.cuda.synchronize()
    errs = check(run)
    assert errs["state"] <= fp32_walk(1200) and errs["out"] <= fp32_walk(1200), errs


def many_long(short):
    """2,100 sequences that are all long, one of them long enough to be split,
    which is done only for lists that are sorted."""
    lens = [short] * 2100
    lens[1234] = 1300
    return lens


def test_more_long_sequences_than_are_put_in_order():
    run_and_check(many_long(20), [1, 0] * 1050, 1, 1, 32, "f32", log_decay=[-0.03])


def test_more_long_prompts_than_are_put_in_order_equal_two_calls():
    """(The half with the long one splits it: other roundings.)"""
    run = LinRun(many_long(19), [1, 0] * 1050, 1, 1, 128, "bf16", log_decay=[-0.03])
    before = run.mem.clone()
    run.run()
    out, mem = run.out.clone(), run.view.clone()
    run.mem.copy_(before)
    for lo, hi in ((0, 1050), (1050, 2100)):
        rows = slice(run.cu[lo], run.cu[hi])
        binding.lin_varlen_forward(run.pool, 0, run.q[rows], run.k[rows], run.v[rows],
                                   run.cu_d[lo:hi + 1] - run.cu[lo], run.blk_d[lo:hi], run.past_d[lo:hi],
                                   run.decay_d, run.out[rows], run.cu[hi] - run.cu[lo], hi - lo,
                                   scale=run.scale)
    torch.cuda.synchronize()
    assert run.pool.error_flags() == 0
    long_rows, long_block = slice(run.cu[1234], run.cu[1235]), run.blk[1234]
    for a, b, at, tol in ((out, run.out, long_rows, 2.0 ** -7), (mem[0], run.view[0], long_block, 1e-5)):
        assert (a[at].double() - b[at].double()).norm() <= tol * b[at].double().norm()
        a[at] = b[at]
        assert torch.equal(a, b)


@pytest.mark.parametrize("act,d", [("f32", 64), ("bf16", 128)])
def test_batches_padded_far_beyond_the_pool(act, d):
    """4,000 sequences on a pool of seven blocks: padding, empty ones that name
    any block, and six with tokens."""
    n = 4000
    rng = np.random.default_rng(3)
    lens, blocks = [0] * n, rng.integers(-3, 40, n).tolist()
    at = rng.permutation(n)[:6].tolist()
    for b, s in enumerate(at):
        lens[s], blocks[s] = [1, 300, 17, 64, 1, 2][b], b + 1
    lens[(at[0] + 1) % n or 1] = 5
    blocks[(at[0] + 1) % n or 1] = -2
    run_and_check(lens, [1] * n, 2, 1, d, act, blocks=blocks, num_blocks=7, tensor_cores=act == "bf16")


@pytest.mark.parametrize("n", [256, 257, 512, 513])
@pytest.mark.parametrize("hint", [0, 1, 2])
def test_the_number_of_sequences_that_check_themselves(n, hint):
    lens = [1] * n
    lens[7] = 0
    run_and_check(lens, [1] * n, 1, 1, 32, "f32", hint=hint, num_blocks=n + 1)


def test_lists_of_another_type_size_or_place_are_refused():
    run = LinRun([3, 1], [1, 1], 2, 1, 64, "f32")
    kw = dict(q=run.q, k=run.k, v=run.v, cu_seqlens=run.cu_d, state_block_idx=run.blk_d,
              has_past=run.past_d, log_decay=run.decay_d, out=run.out, T=4, N=2)
    for bad in (dict(cu_seqlens=run.cu_d.long()), dict(cu_seqlens=run.cu_d[:2]),
                dict(cu_seqlens=run.cu_d.cpu()), dict(state_block_idx=run.blk_d[:1]),
                dict(state_block_idx=torch.stack([run.blk_d, run.blk_d], 1)[:, 0]),
                dict(has_past=run.past_d.int()), dict(log_decay=run.decay_d.double()),
                dict(log_decay=run.decay_d[:1]), dict(q=run.q.cpu()), dict(N=3)):
        with pytest.raises(ValueError):
            binding.lin_varlen_forward(run.pool, 0, **(kw | bad))
    torch.cuda.synchronize()
    assert (run.out == SENTINEL).all() and run.pool.error_flags() == 0
