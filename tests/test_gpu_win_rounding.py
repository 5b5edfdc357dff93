"""How far windowed attention's outputs may be off in each of its forms: element
by element with the roundings that this form makes, and in the 2-norm, where a
key too many or too few shows.

Weights: the form for few tokens cuts a weight off at bf16 (what is left is below
2^-7 of it) and rounds the rest to bf16 (2^-8 of that): 2^-15; the prompts'
form rounds it to bf16: 2^-8; the form for any shape keeps fp32."""
import numpy as np
import pytest
import torch

from hybrid_check import EPS, ULP, WinRun, close, f64
from oracle import hybrid as ref

pytestmark = pytest.mark.gpu

WEIGHT = {"few": 2.0 ** -15, "prompts": 2.0 ** -8, "any": 0.0}


def form_of(run, s):
    group = run.H // run.Hkv
    if run.act == "f32" or run.d == 32 or group > 128:
        return "any"
    return "few" if run.lens[s] <= 32 // group else "prompts"


def expected(run, window=None):
    x, H, Hkv = f64(run.x), run.H, run.Hkv
    return ref.win_forward(x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:], run.cu, run.past,
                           [dict(h) for h in run.history], window or run.window, run.sinks, run.scale)


def one_sign(x, run):
    x[:, run.H + run.Hkv:] = x[:, run.H + run.Hkv:].abs() + 0.5


def one_sign_held(rows, pos, s):
    rows[:, 1] = rows[:, 1].abs() + 0.5


def run_and_compare(run, forms):
    """Element by element: the same bounds as everywhere, with the form's weights."""
    assert {form_of(run, s) for s in range(run.N)} == set(forms)
    out, mag, score = expected(run)
    run.run()
    torch.cuda.synchronize()
    got = f64(run.out)
    for s in range(run.N):
        rows = slice(run.cu[s], run.cu[s + 1])
        keys = min(run.window, run.past[s] + run.lens[s]) + run.sinks
        weight = 2 * (run.d + 8) * EPS * score[rows][..., None] + 16 * EPS + WEIGHT[form_of(run, s)]
        tol = (2 * weight + 2 * (keys + 16) * EPS) * mag[rows] + ULP[run.act] * np.abs(out[rows])
        close(got[rows], out[rows], tol + 2.0 ** -126, (form_of(run, s), s))
    return got, out


@pytest.mark.parametrize("d,H,Hkv", [(64, 8, 2), (128, 8, 2), (128, 4, 4), (128, 32, 1)])
@pytest.mark.parametrize("n", [1, 64])  # (windows cut over CTAs, and whole ones)
def test_single_tokens_with_values_of_one_sign(d, H, Hkv, n):
    past = [i % 9 if i % 3 else 40 + 7 * i for i in range(n)]
    run_and_compare(WinRun([1] * n, past, H, Hkv, d, 120, 4, values=one_sign, history=one_sign_held), ["few"])


@pytest.mark.parametrize("d,H,Hkv,k", [(64, 8, 2, 8), (128, 8, 2, 4), (128, 4, 4, 32), (128, 32, 1, 1)])
def test_drafted_tokens_with_values_of_one_sign(d, H, Hkv, k):
    lens = [max(1, k - i % 3) for i in range(12)]
    run_and_compare(WinRun(lens, [0, 1, 2, 5, 30, 119, 120, 130, 1000, 0, 3, 64], H, Hkv, d, 120, 4, values=one_sign,
                           history=one_sign_held), ["few"])


@pytest.mark.parametrize("act,d,H,Hkv", [("bf16", 32, 8, 2), ("f32", 64, 4, 2), ("bf16", 64, 160, 1)])
def test_the_form_for_any_shape_with_values_of_one_sign(act, d, H, Hkv):
    run_and_compare(WinRun([1, 3, 20, 1], [0, 2, 30, 200], H, Hkv, d, 60, 4, act, values=one_sign,
                           history=one_sign_held), ["any"])


def test_prompts_with_values_of_one_sign():
    run_and_compare(WinRun([140, 40], [0, 90], 8, 2, 128, 60, 4, values=one_sign, history=one_sign_held), ["prompts"])


# 2-norm: outputs are rounded by 2^-8 at most; with values that are independent and of mean 0
# roundings of the weights add what they add to the squares, 2^-8 at most in the prompts'
# form; 2^-12 is beyond all of fp32's
@pytest.mark.parametrize("act,d,H,Hkv,lens,past,form,bound", [
    ("bf16", 128, 8, 2, [1, 1, 1], [5000, 4096, 9000], "few", 2.0 ** -8 + 2.0 ** -12),
    ("bf16", 64, 8, 2, [3, 1], [5000, 4500], "few", 2.0 ** -8 + 2.0 ** -12),
    ("bf16", 128, 8, 2, [40], [5000], "prompts", 2.0 ** -7 + 2.0 ** -12),
    ("bf16", 32, 8, 2, [2, 1], [5000, 4500], "any", 2.0 ** -8 + 2.0 ** -12),
    ("f32", 64, 4, 2, [2, 1], [5000, 4500], "any", 2.0 ** -12)])
def test_a_long_window_to_the_key(act, d, H, Hkv, lens, past, form, bound):
    run = WinRun(lens, past, H, Hkv, d, 4096, 4, act, seed=5)
    got, out = run_and_compare(run, [form])
    size = np.linalg.norm(out)
    assert np.linalg.norm(got - out) <= bound * size, np.linalg.norm(got - out) / size
    # and a window of one key less would not pass
    assert np.linalg.norm(expected(run, 4095)[0] - out) > 1.2 * bound * size
