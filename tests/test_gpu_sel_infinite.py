"""An infinite state in a sequence that is cut into segments: it stays infinite,
as it does step by step (a segment's whole decay may be too small for fp32)."""
import numpy as np
import pytest
import torch

from hybrid_check import SelRun, bits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens", [[900], [700, 1, 450]])
@pytest.mark.parametrize("N", [16, 32, 64])
@pytest.mark.parametrize("value", [float("inf"), -float("inf")])
def test_an_infinite_state_stays_infinite(lens, N, value):
    kw = dict(N=N, act="f32", gate=False, seed=N, dt_bias=torch.zeros(8))
    a, b = SelRun(lens, [1] * len(lens), 8, **kw), SelRun(lens, [1] * len(lens), 8, **kw)
    # decays of e^-10 a token or so at most: each is far from 0, those of 64 tokens are not
    a_log = torch.log(torch.linspace(0.01, 4.0, N)).repeat(8, 1).cuda()
    a.dev[2], b.dev[2] = a_log, a_log
    for s in range(len(lens)):
        b.ssm[b.blk[s], 3, 1] = b.ssm[b.blk[s], 3, N - 1] = value
    for run in (a, b):
        run.run_scan()
    torch.cuda.synchronize()
    others = [c for c in range(8) if c != 3]
    assert torch.equal(bits(a.out[:, others]), bits(b.out[:, others]))
    for s in range(len(lens)):
        h, was = b.ssm[b.blk[s]], a.ssm[a.blk[s]]
        assert h[3, 1] == value and h[3, N - 1] == value, (h[3, 1], h[3, N - 1])
        h[3, 1], h[3, N - 1] = was[3, 1], was[3, N - 1]
        assert torch.equal(bits(h), bits(was))
        # an output is infinite, or NaN where the two infinite terms differ in sign
        rows = slice(b.cu[s], b.cu[s + 1])
        c = b.Cm[rows][:, [1, N - 1]].double().cpu().numpy()
        with np.errstate(invalid="ignore"):
            want = (c * value).sum(1)
        np.testing.assert_array_equal(b.out[rows, 3].double().cpu().numpy(), want)
