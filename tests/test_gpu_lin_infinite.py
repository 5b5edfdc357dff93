"""Infinite values in decayed linear attention on the GPU: where the recurrence
gives an infinity, every form does, and NaN only where it gives NaN (a decay
leaves an infinity what it is, and so does adding a finite product)."""
import numpy as np
import pytest
import torch

from lin_check import LinRun

pytestmark = pytest.mark.gpu

INF = float("inf")
# log decays on both sides of where the rounding of e^g is corrected, and none
DECAY = [-0.3, 0.0, -0.7, -1e-3]
FORMS = [
    ("f32", 32, [1, 1], 1), ("f32", 128, [1, 1], 0), ("bf16", 64, [1, 1], 1), ("bf16", 128, [1, 1], 1),
    ("f32", 64, [5, 18], 0), ("bf16", 128, [5, 18], 0), ("bf16", 32, [16, 33], 0),
    ("f32", 32, [900, 3], 0), ("bf16", 64, [900, 3], 0), ("f32", 128, [700, 40], 0),   # segments
    ("bf16", 128, [200, 90], 0), ("bf16", 128, [1500, 70], 0),                         # chunks, segments of them
]


def check_infinities(run, out, states):
    got = run.out[:run.T].double().cpu().numpy()
    view = run.view[0].double().cpu().numpy()[run.blk]
    for name, g, w in (("out", got, out), ("state", view, states)):
        for kind in (np.isnan, np.isposinf, np.isneginf):
            bad = kind(g) != kind(w)
            assert not bad.any(), (name, kind.__name__, np.argwhere(bad)[:4], g[bad][:4], w[bad][:4])
        fine = np.isfinite(w)
        # (values that others of their sums do not dwarf: the forms' own tests hold their errors)
        tol = 2.0 ** -7 if name == "out" and run.act == "bf16" else 1e-5
        assert np.linalg.norm(g[fine] - w[fine]) <= tol * np.linalg.norm(w[fine]), name
    assert run.pool.error_flags() == 0


@pytest.mark.parametrize("act,d,lens,hint", FORMS)
def test_an_infinite_past(act, d, lens, hint):
    """One entry of a state's column is infinite: so are the column's outputs,
    with the sign of q, and the entry for good."""
    run = LinRun(lens, [1, 1], 4, 2, d, act, log_decay=DECAY, hint=hint, seed=1)
    for h, (k, v, x) in enumerate([(3, 5, INF), (0, d - 1, -INF), (d - 1, 17, INF), (11, 0, -INF)]):
        run.states[0, h, k, v] = x
    run.view[0, run.blk[0]] = run.states[0].cuda()
    with np.errstate(invalid="ignore"):
        out, states = run.expected()
    assert np.isinf(out).any() and not np.isnan(out).any()
    run.run()
    torch.cuda.synchronize()
    check_infinities(run, out, states)


@pytest.mark.parametrize("act,d,lens,hint", [f for f in FORMS if f[3] == 0 and f[2][0] > 1])
@pytest.mark.parametrize("of", ["k", "v"])
def test_an_infinite_token(act, d, lens, hint, of):
    """An infinite entry of k or v makes a row or a column of the state
    infinite, with the other one's signs; its outputs are sums of both signs."""
    at = lens[0] // 2

    def put(x, run):
        x[at, run.H * d + (0 if of == "k" else run.Hkv * d) + 7] = INF  # kv head 0: q heads 0 and 1

    run = LinRun(lens, [1, 1], 4, 2, d, act, log_decay=DECAY, values=put, seed=2)
    with np.errstate(invalid="ignore"):
        out, states = run.expected()
    assert np.isinf(states[0, :2]).any() and not np.isnan(states).any()
    run.run()
    torch.cuda.synchronize()
    check_infinities(run, out, states)


def test_a_head_without_memory_forgets_no_infinity():
    """e^g = 0 times an infinity is NaN, as the recurrence has it."""
    for act, d, lens in (("f32", 64, [5]), ("f32", 32, [900]), ("bf16", 128, [200])):
        run = LinRun(lens, [1], 2, 1, d, act, log_decay=[-INF, -0.5], seed=3)
        run.states[0, :, 2, 3] = INF
        run.view[0, run.blk[0]] = run.states[0].cuda()
        with np.errstate(invalid="ignore"):
            out, states = run.expected()
        assert np.isnan(out[:, 0, 3]).all() and np.isinf(out[:, 1, 3]).all()
        run.run()
        torch.cuda.synchronize()
        check_infinities(run, out, states)
