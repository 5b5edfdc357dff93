"""The outputs of decayed linear attention's chunked form on the GPU are as
close to the fp64 recurrence as their type allows: P = Q K^T and the state
enter their products with 16 significant bits, so that an output is off by its
own rounding, as in the recurrent form of a few tokens."""
import numpy as np
import pytest
import torch

from continuous_linear_attention_gb300 import binding
from lin_check import LinRun

pytestmark = pytest.mark.gpu


def last_path(pool):
    import ctypes
    v = ctypes.c_int()
    assert binding.load().gdn_pool_last_prefill_path(pool.handle, ctypes.byref(v)) == 0
    return v.value


def check_rounding(run):
    """Element by element: the output's rounding to bf16 (2^-8 of the value),
    and of the same forward over absolute values, A, what else is rounded.  A
    weight of P or an entry of the state as two bf16 terms is off by 2^-8 of
    2^-8 of it, which adds up to at most 2^-16 of A.  fp32: at most 3 n + d + 4
    roundings of 2^-24 in a recurrence of n tokens, or 32 accumulations of
    2^-23 per chunk, should the tensor cores truncate, and twice that for the
    second terms.

    And as a whole: the roundings beside the output's own are 2^-8 times as
    large as it and independent of it, so the relative error is the one that
    rounding the exact outputs gives, within 5% (one bf16 rounding more, of P
    or of the state, would make it 20% larger at least, both 41%)."""
    out, _ = run.expected()
    mag, _ = run.expected(magnitude=True)
    got = run.out[:run.T].double().cpu().numpy()
    worst = 0.0
    for lo, hi in zip(run.cu, run.cu[1:]):
        if lo == hi:
            continue
        n = hi - lo
        fp32 = max((3 * n + run.d + 4) * 2.0 ** -24, 64 * (n // 128 + 1) * 2.0 ** -23)
        want = out[lo:hi]
        tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -16 + fp32) * mag[lo:hi] * (1 + 2.0 ** -7)
        bad = np.abs(got[lo:hi] - want) > tol
        assert not bad.any(), (bad.mean(), np.argwhere(bad)[:4], got[lo:hi][bad][:4], want[bad][:4])
        rounded = torch.from_numpy(want).bfloat16().double().numpy()
        norm = np.linalg.norm
        worst = max(worst, norm(got[lo:hi] - want) / norm(rounded - want))
    assert worst <= 1.05, worst


@pytest.mark.parametrize("lens,H,Hkv,past", [
    ([700], 4, 2, 1), ([700], 4, 4, 0), ([128, 65, 257, 129], 4, 1, 1),
    ([19, 40, 127, 1, 300, 64, 33, 0, 130, 25, 90], 20, 5, 1),  # enough heads: 19 tokens are chunked
])
def test_prompts(lens, H, Hkv, past):
    run = LinRun(lens, [past] * len(lens), H, Hkv, 128, "bf16", seed=len(lens))
    run.run()
    torch.cuda.synchronize()
    assert run.pool.error_flags() == 0 and last_path(run.pool) == 2
    check_rounding(run)


@pytest.mark.parametrize("lens,H,decay", [
    ([2100, 700], 2, [-1e-4, -1e-6]),       # everything since the start counts
    ([400, 90], 8, [0.0, -1e-5, -0.02, -0.3, -2.0, -30.0, -200.0, -float("inf")]),
    ([4000, 1024], 2, [-0.004, -3.0]),      # cut into segments
])
def test_decays(lens, H, decay):
    run = LinRun(lens, [1, 0], H, 1, 128, "bf16", log_decay=decay, seed=3)
    run.run()
    torch.cuda.synchronize()
    assert run.pool.error_flags() == 0 and last_path(run.pool) == 2
    check_rounding(run)


def test_a_prompt_and_the_same_prompt_in_calls_of_a_few_tokens():
    """The chunked form and the recurrent one differ by their outputs'
    rounding at most where they agree on everything else."""
    n = 160
    run = LinRun([n], [1], 4, 2, 128, "bf16", seed=12)
    start = run.mem.clone()
    run.run()
    whole = run.out.clone()
    run.mem.copy_(start)
    for t in range(0, n, 16):
        cu = torch.tensor([0, 16], dtype=torch.int32, device="cuda")
        rows = slice(t, t + 16)
        binding.lin_varlen_forward(run.pool, 0, run.q[rows], run.k[rows], run.v[rows], cu, run.blk_d,
                                   run.past_d, run.decay_d, run.out[rows], 16, 1, scale=run.scale,
                                   max_seqlen_hint=16)
    torch.cuda.synchronize()
    check_rounding(run)
    # both are the exact values' roundings but where those lie near a border
    assert (whole != run.out).double().mean() < 0.02
