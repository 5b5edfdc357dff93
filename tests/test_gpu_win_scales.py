"""Scales at the ends of their range: the smallest ones with scores that fp32
just holds, the largest ones with scores of 0."""
import pytest
import torch

from continuous_linear_attention_gb300 import binding
from hybrid_check import SENTINEL, WinRun, win_check

pytestmark = pytest.mark.gpu

FORMS = pytest.mark.parametrize("act,d", [("bf16", 128), ("bf16", 64), ("f32", 64)])


@FORMS
@pytest.mark.parametrize("scale", [0.0, 1e-38, -1e-38, 2.0 ** -101, 2.0 ** -99, -2.0 ** -99])
def test_small_scales_of_large_scores(act, d, scale):
    def put(x, run):
        x[:, :6] *= 2.0 ** 59  # (q and k: scores of 2^118 d^1/2 or so)

    def held(rows, pos, s):
        rows[:, 0] *= 2.0 ** 59

    win_check([140, 1, 3, 60], [0, 90, 7, 30], 4, 2, d, 60, 4, act, values=put, history=held, scale=scale)


@FORMS
def test_the_largest_scale_of_scores_of_0(act, d):
    def put(x, run):
        x[:, :4] = 0.0

    for scale in (2.0 ** 127, -2.0 ** 127):
        win_check([140, 1, 3], [0, 90, 7], 4, 2, d, 60, 4, act, values=put, scale=scale)


@FORMS
def test_scales_beyond_the_largest_are_refused(act, d):
    run = WinRun([140, 1], [0, 9], 4, 2, d, 60, 4, act)
    for scale in (1.8e38, -3.4e38):
        run.scale = scale
        with pytest.raises(binding.GdnError):
            run.run()
    torch.cuda.synchronize()
    assert (run.out == SENTINEL).all() and torch.equal(run.mem, run.before)
