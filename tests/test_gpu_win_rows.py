"""A row's running maximum, and so the rounding of its weights, is its own,
whatever the scores of the rows that share its tile."""
import pytest
import torch

from hybrid_check import WinRun, bits
from test_gpu_win_neighbours import outputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,H,Hkv", [(64, 4, 2), (128, 8, 2), (128, 3, 3), (128, 64, 1)])
def test_larger_scores_of_other_rows_do_not_change_a_rows_rounding(d, H, Hkv):
    """Queries of other heads and of the next sequence with scores far above."""
    lens, past = [150, 201], [130, 0]

    def put(x, run):
        x[run.cu[1]:, :H] *= 40
        if H // Hkv > 1:
            x[:, H // Hkv - 1] *= 40

    a, b = WinRun(lens, past, H, Hkv, d, 70, 5), WinRun(lens, past, H, Hkv, d, 70, 5, values=put)
    for run in (a, b):
        run.mem.view(torch.bfloat16).nan_to_num_(nan=0.75)
        run.before.copy_(run.mem)
    x, y = outputs(a), outputs(b)
    heads = [h for h in range(H) if H // Hkv == 1 or h != H // Hkv - 1]
    assert torch.equal(bits(x[:150, heads]), bits(y[:150, heads]))
