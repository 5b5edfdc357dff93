"""What no value of a neighbour or a later token may change in decayed linear
attention's chunked form on the GPU, bit for bit.  (The form computes columns
with values that are not finite again token by token, which gives other
roundings: equal bits show that a chunk that need not be was not.)"""
import numpy as np
import pytest
import torch

from lin_check import LinRun

pytestmark = pytest.mark.gpu

BAD = [float("nan"), float("inf"), -float("inf")]
# (lens, heads, kv heads): alone, with enough heads that 19 tokens are chunked,
# and cut into segments
CHUNKED = [([200, 90, 70], 4, 2), ([40, 129, 25, 60, 20, 33, 130, 19, 90, 64], 20, 5), ([1500, 1100, 70], 2, 2)]


def bits(t):
    return t.contiguous().view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)


def pair(lens, H, Hkv, put, **kw):
    """The same batch as it is and with ``put`` on its rows; both run."""
    runs = [LinRun(lens, [1, 0] * (len(lens) // 2) + [1] * (len(lens) % 2), H, Hkv, 128, "bf16", seed=4,
                   values=v, **kw) for v in (None, put)]
    for r in runs:
        r.run()
    torch.cuda.synchronize()
    assert all(r.pool.error_flags() == 0 and r.pool.last_prefill_path() == 2 for r in runs)
    return runs


@pytest.mark.parametrize("lens,H,Hkv", CHUNKED)
@pytest.mark.parametrize("value", BAD)
@pytest.mark.parametrize("part", ["q", "k", "v", "all"])
def test_the_next_sequence_in_a_chunks_tail(lens, H, Hkv, value, part):
    """The tile of a sequence's last chunk goes on into the next sequence's
    rows: whatever is there, nothing of the sequence changes."""
    victims = [s for s in range(len(lens) - 1) if lens[s] % 128 and s % 2 == 0]

    def put(x, run):
        cols = {"q": slice(0, H * 128), "k": slice(H * 128, (H + Hkv) * 128),
                "v": slice((H + Hkv) * 128, None), "all": slice(None)}[part]
        for s in victims:
            x[run.cu[s + 1]:run.cu[s + 1] + 6, cols] = value

    fine, run = pair(lens, H, Hkv, put)
    for s in victims:
        rows = slice(run.cu[s], run.cu[s + 1])
        assert torch.isfinite(run.out[rows]).all()
        assert torch.equal(bits(run.out[rows]), bits(fine.out[rows])), s
        assert torch.equal(bits(run.view[0, run.blk[s]]), bits(fine.view[0, fine.blk[s]])), s


@pytest.mark.parametrize("lens,H,Hkv", CHUNKED)
@pytest.mark.parametrize("value", BAD)
def test_a_query_reaches_its_own_row_alone(lens, H, Hkv, value):
    def put(x, run):
        for s in range(len(lens)):
            x[run.cu[s] + lens[s] // 2, :H * 128] = value

    fine, run = pair(lens, H, Hkv, put)
    rows = torch.ones(run.T, dtype=torch.bool, device="cuda")
    for s in range(len(lens)):
        rows[run.cu[s] + lens[s] // 2] = False
    assert not torch.isfinite(run.out[~rows]).any()
    assert torch.equal(bits(run.out[rows]), bits(fine.out[rows]))
    assert torch.equal(bits(run.mem.view(torch.float32)), bits(fine.mem.view(torch.float32)))


@pytest.mark.parametrize("lens,H,Hkv", CHUNKED)
@pytest.mark.parametrize("value", BAD)
def test_a_value_reaches_its_own_columns_slice_alone(lens, H, Hkv, value):
    """One column of v: the other 96 columns that are not computed with it, and
    every other sequence, keep their bits, earlier rows their values."""
    s, col = len(lens) // 2, 37
    at = lens[s] // 2

    def put(x, run):
        x[run.cu[s] + at, (H + Hkv) * 128 + col] = value  # kv head 0

    fine, run = pair(lens, H, Hkv, put)
    group = H // Hkv
    other = torch.ones(H, 128, dtype=torch.bool, device="cuda")
    other[:group, 32:64] = False
    mine = slice(run.cu[s], run.cu[s + 1])
    for r in range(len(lens)):
        rows = slice(run.cu[r], run.cu[r + 1])
        keep = other if r == s else torch.ones_like(other)
        assert torch.equal(bits(run.out[rows])[:, keep], bits(fine.out[rows])[:, keep]), r
        a, b = (bits(x.view[0, x.blk[r]]).transpose(1, 2)[keep] for x in (run, fine))
        assert torch.equal(a, b), r
    # the slice itself: earlier rows and its other columns as if it were a number
    got, want = run.out[mine].double(), fine.out[mine].double()
    assert not torch.isfinite(got[at:, :group, col]).any()
    keep = torch.arange(128, device="cuda") != col
    assert torch.equal(torch.isfinite(got), ~((torch.arange(lens[s], device="cuda") >= at)[:, None, None] &
                                              ~keep[None, None] & (torch.arange(H, device="cuda") < group)[None, :, None]))
    for x, y in ((got[:at], want[:at]), (got[at:, :, keep], want[at:, :, keep])):
        assert (x - y).norm() <= 2.0 ** -8 * y.norm()


@pytest.mark.parametrize("lens,H,Hkv", CHUNKED)
@pytest.mark.parametrize("value", BAD)
def test_a_key_reaches_later_rows_of_its_head_alone(lens, H, Hkv, value):
    """In the middle of a chunk: earlier rows are those of a number, other kv
    heads and sequences keep their bits."""
    s = len(lens) // 2
    at = min(lens[s] // 2 + 3, lens[s] - 1)

    def put(x, run):
        x[run.cu[s] + at, H * 128 + 11] = value  # kv head 0

    fine, run = pair(lens, H, Hkv, put)
    group = H // Hkv
    for r in range(len(lens)):
        rows = slice(run.cu[r], run.cu[r + 1])
        heads = slice(group if r == s else 0, H)
        assert torch.equal(bits(run.out[rows, heads]), bits(fine.out[rows, heads])), r
        assert torch.equal(bits(run.view[0, run.blk[r], heads]), bits(fine.view[0, fine.blk[r], heads])), r
    before = slice(run.cu[s], run.cu[s] + at)
    got, want = run.out[before, :group].double(), fine.out[before, :group].double()
    assert torch.isfinite(got).all() and (got - want).norm() <= 2.0 ** -8 * want.norm()
    assert not torch.isfinite(run.out[run.cu[s] + at:run.cu[s + 1], :group]).any()
