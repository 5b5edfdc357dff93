"""Calls of decayed linear attention that leave sequences out, with others
right behind them on the stream: what a left-out sequence had begun to load
has to have landed before its shared memory is anyone else's."""
import pytest
import torch

from lin_check import LinRun, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act,d", [("f32", 64), ("f32", 128), ("bf16", 32), ("bf16", 128)])
def test_left_out_sequences_and_calls_right_behind(act, d):
    """Every sequence of the first call names one block (all are left out),
    the second one's batch is bad as a whole, the third one is fine."""
    lens = [3, 16, 2, 7] * 12
    runs = [LinRun(lens, [1] * 48, 4, 4, d, act, seed=s, blocks=blocks)
            for s, blocks in ((1, [5] * 48), (2, None), (3, None))]
    runs[1].cu[0] = 1
    runs[1].cu_d[:1] = 1
    states = [r.mem.clone() for r in runs]
    torch.cuda.synchronize()
    for i in range(3):
        runs[2].mem.copy_(states[2])
        for r in runs:
            r.run()
    torch.cuda.synchronize()
    for r in runs:
        check(r)
    assert torch.equal(runs[0].mem, states[0]) and torch.equal(runs[1].mem, states[1])
