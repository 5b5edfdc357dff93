"""One sequence that is longer than its hint: no form takes it, but a kernel has
to look at the batch and say so."""
import pytest
import torch

from hybrid_check import SENTINEL, WinRun, win_check

pytestmark = pytest.mark.gpu

HINT, SEQLENS = 0x20, 0x1


@pytest.mark.parametrize("act,d,H,Hkv", [("bf16", 64, 8, 2), ("bf16", 128, 1, 1), ("bf16", 32, 4, 2), ("f32", 64, 4, 2)])
@pytest.mark.parametrize("n", [9, 33, 34, 200])
@pytest.mark.parametrize("hint", [1, 8])
def test_one_sequence_longer_than_its_hint(act, d, H, Hkv, n, hint):
    run = WinRun([n], [5], H, Hkv, d, 20, 2, act, hint=hint)
    run.run()
    torch.cuda.synchronize()
    assert run.pool.error_flags() == HINT
    assert (run.out == SENTINEL).all() and torch.equal(run.mem, run.before)
    win_check([n], [5], H, Hkv, d, 20, 2, act, hint=n)  # (as long as the hint: taken)


@pytest.mark.parametrize("cu", [[0, 30], [1, 40], [0, -1], [0, 41]])
def test_bad_cu_seqlens_of_one_sequence_with_a_small_hint(cu):
    run = WinRun([40], [5], 8, 2, 64, 20, 2, hint=2)
    run.cu_d = torch.tensor(cu, dtype=torch.int32, device="cuda")
    run.run()
    torch.cuda.synchronize()
    assert run.pool.error_flags() == SEQLENS
    assert (run.out == SENTINEL).all() and torch.equal(run.mem, run.before)
