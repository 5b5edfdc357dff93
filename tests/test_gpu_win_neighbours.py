"""What lies next to a sequence's keys and values in memory - slots without a
position, another head's or another block's slots, another sequence's tokens -
is no part of its attention: its outputs are the same to the bit, whatever is
there.  (The prompts' form loads keys in whole boxes, beyond a run's end.)"""
import pytest
import torch

from hybrid_check import WinRun, bits

pytestmark = pytest.mark.gpu

BAD = [float("nan"), float("inf"), -float("inf")]
SHAPES = pytest.mark.parametrize("d,H,Hkv", [(64, 4, 2), (128, 8, 2), (128, 3, 3), (128, 64, 1)])
# tokens and past: rings that have wrapped, rings that have not, runs of no whole number of boxes
CASES = pytest.mark.parametrize("lens,past", [([150, 201, 40], [30, 0, 7]), ([300, 35, 90], [900, 20, 3]),
                                              ([130], [101])])


def outputs(run):
    run.run()
    torch.cuda.synchronize()
    assert run.pool.error_flags() == 0
    return run.out.clone()


@SHAPES
@CASES
@pytest.mark.parametrize("value", BAD)
def test_slots_without_a_position(d, H, Hkv, lens, past, value):
    a, b = (WinRun(lens, past, H, Hkv, d, 70, 5) for _ in range(2))
    a.mem.view(torch.bfloat16).nan_to_num_(nan=0.75)
    free = torch.isnan(b.mem.view(torch.bfloat16))
    b.mem.view(torch.bfloat16)[free] = value
    a.before.copy_(a.mem), b.before.copy_(b.mem)
    assert torch.equal(bits(outputs(a)), bits(outputs(b)))
    a.check()


@SHAPES
@CASES
@pytest.mark.parametrize("value", BAD)
def test_other_blocks(d, H, Hkv, lens, past, value):
    a, b = (WinRun(lens, past, H, Hkv, d, 70, 5, num_blocks=2 * len(lens) + 2,
                   blocks=[2 * i + 1 for i in range(len(lens))]) for _ in range(2))
    for run, x in ((a, 0.5), (b, value)):
        run.mem.view(torch.bfloat16).nan_to_num_(nan=0.75)
        run.kv[2::2] = x
        run.before.copy_(run.mem)
    assert torch.equal(bits(outputs(a)), bits(outputs(b)))
    a.check()


@SHAPES
@pytest.mark.parametrize("value", BAD)
@pytest.mark.parametrize("what", ["q", "k", "v", "qkv"])
def test_other_sequences_tokens(d, H, Hkv, value, what):
    """The sequences between, of one token and of many, hold the value in every row."""
    lens, past = [150, 60, 40, 1, 97], [30, 9, 7, 100, 0]

    def put(x, run):
        for s in (1, 3):
            rows = x[run.cu[s]:run.cu[s + 1]]
            for part, heads in (("q", slice(0, H)), ("k", slice(H, H + Hkv)), ("v", slice(H + Hkv, None))):
                if part in what:
                    rows[:, heads] = value

    a, b = WinRun(lens, past, H, Hkv, d, 70, 5), WinRun(lens, past, H, Hkv, d, 70, 5, values=put)
    for run in (a, b):
        run.mem.view(torch.bfloat16).nan_to_num_(nan=0.75)
        run.before.copy_(run.mem)
    x, y = outputs(a), outputs(b)
    for s in (0, 2, 4):
        rows = slice(a.cu[s], a.cu[s + 1])
        assert torch.equal(bits(x[rows]), bits(y[rows])), s


@pytest.mark.parametrize("value", BAD)
@pytest.mark.parametrize("d,H,Hkv", [(64, 4, 2), (128, 8, 2), (128, 3, 3)])
def test_another_head(value, d, H, Hkv):
    """The second kv head's keys and values, held and new, and its queries."""
    group = H // Hkv

    def put(x, run):
        x[:, group:2 * group] = value
        x[:, H + 1] = value
        x[:, H + Hkv + 1] = value

    lens, past = [150, 201, 1], [130, 0, 50]
    a = WinRun(lens, past, H, Hkv, d, 70, 5)
    b = WinRun(lens, past, H, Hkv, d, 70, 5, values=put, history=lambda rows, pos, s: rows[:, :, 1].fill_(value))
    free = torch.isnan(a.mem.view(torch.bfloat16))
    for run in (a, b):
        run.mem.view(torch.bfloat16)[free] = 0.75
        run.before.copy_(run.mem)
    x, y = outputs(a), outputs(b)
    heads = [h for h in range(H) if h // group != 1]
    assert torch.equal(bits(x[:, heads]), bits(y[:, heads]))
