"""The operators as a hybrid model uses them together: a windowed attention
layer (norms and rotation, then attention over its pool) and a selective scan
layer (convolution, then the scan over its pool) over a request's prompt and
tokens, forked in between, against one pass over the whole."""
import pytest
import torch

from continuous_linear_attention_gb300 import binding

pytestmark = pytest.mark.gpu

I32 = dict(dtype=torch.int32, device="cuda")


class Layers:
    """Two layers on their pools, fed with given projections of each token."""

    def __init__(self, act, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.H, self.Hkv, self.d, self.C, self.N = 4, 2, 64, 64, 16
        self.dt = torch.float32 if act == "f32" else torch.bfloat16
        r = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
        self.qkv = r(2, 90, self.H + 2 * self.Hkv, self.d).to(self.dt)  # two continuations
        self.x, self.z, self.step = (r(2, 90, self.C).to(self.dt) for _ in range(3))
        self.bc = r(2, 90, 2 * self.N).to(self.dt)
        self.norm = [1 + 0.1 * r(self.d), 1 + 0.1 * r(self.d)]
        self.freq = 1e4 ** (-torch.arange(0, self.d, 2).cuda() / self.d)
        self.w, self.b = r(self.C, 4).to(self.dt), r(self.C).to(self.dt)
        self.A_log, self.D, self.bias = r(self.C, self.N), r(self.C), r(self.C) - 2
        for t in (self.qkv, self.x, self.z, self.step, self.bc):
            t[1, :60] = t[0, :60]  # the prompt is the same
        self.win = binding.WinPool(6, 1, self.Hkv, self.d, 24, 3, act)
        self.sel = binding.SelPool(6, 1, self.C, self.N, 4, act)

    def go(self, beams, blocks, lo, hi):
        """Tokens lo..hi of the given beams, continued in their blocks."""
        n, m = len(beams), hi - lo
        pick = lambda t: torch.cat([t[b, lo:hi] for b in beams])  # noqa: E731
        cu = torch.arange(0, (n + 1) * m, m, **I32)
        blk, past = torch.tensor(blocks, **I32), torch.full((n,), lo, **I32)
        qkv = pick(self.qkv)
        pos = torch.arange(lo, hi, **I32).repeat(n)
        q, k = binding.qk_norm_rope(qkv[:, :self.H], qkv[:, self.H:self.H + self.Hkv], pos, self.freq, *self.norm)
        o = torch.empty_like(qkv[:, :self.H])
        binding.win_varlen_forward(self.win, 0, q, k, qkv[:, self.H + self.Hkv:], cu, blk, past, o, n * m, n,
                                   scale=self.d ** -0.5, max_seqlen_hint=m)
        has = (past > 0).to(torch.uint8)
        x = pick(self.x)
        u, y = torch.empty_like(x), torch.empty_like(x)
        binding.sel_conv_varlen_forward(self.sel, 0, x, cu, blk, has, self.w, self.b, u, n * m, n, max_seqlen_hint=m)
        bc = pick(self.bc)
        binding.sel_scan_varlen_forward(self.sel, 0, u, pick(self.step), bc[:, :self.N], bc[:, self.N:], pick(self.z),
                                        cu, blk, has, self.A_log, self.D, self.bias, y, n * m, n, max_seqlen_hint=m)
        return o.view(n, m, -1).float(), y.view(n, m, -1).float()


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_prompt_fork_and_tokens_as_one_pass(act):
    whole, parts = Layers(act), Layers(act)
    want = whole.go([0, 1], [1, 2], 0, 90)
    first = parts.go([0], [3], 0, 60)
    for pool in (parts.win, parts.sel):  # the prompt's block forked
        pool.copy_blocks(torch.tensor([3, 3], **I32), torch.tensor([4, 5], **I32))
    got = [first]
    for t in range(60, 80):
        got.append(parts.go([0, 1], [4, 5], t, t + 1))
    got.append(parts.go([0, 1], [4, 5], 80, 90))  # drafted tokens
    torch.cuda.synchronize()
    assert not (parts.win.error_flags() or parts.sel.error_flags())
    for i in (0, 1):
        have = torch.cat([torch.cat([g[i]] * (2 // len(g[i]))) for g in got], 1)
        # the same roundings up to the order of sums; bf16: a step of each side's rounding (the
        # convolution's among them, which the scan carries on)
        tol = 1e-4 if act == "f32" else 2.0 ** -5
        assert ((have - want[i]).abs() <= tol * (1 + want[i].abs())).all(), i


def test_two_layers_in_one_graph():
    a, b = Layers("bf16", 1), Layers("bf16", 1)
    a.go([0, 1], [1, 2], 0, 60), b.go([0, 1], [1, 2], 0, 60)
    pos = 60
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = b.go([0, 1], [1, 2], pos, pos + 1)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    qkv = a.qkv[:, pos].contiguous()
    n, cu, blk = 2, torch.arange(3, **I32), torch.tensor([1, 2], **I32)
    past, has = torch.full((2,), pos, **I32), torch.ones(2, dtype=torch.uint8, device="cuda")
    o, x = torch.empty_like(qkv[:, :a.H]), a.x[:, pos].contiguous()
    u, y, z, step, bc = torch.empty_like(x), torch.empty_like(x), *(t[:, pos].contiguous() for t in (a.z, a.step, a.bc))
    qo, ko = torch.empty_like(qkv[:, :a.H]), torch.empty_like(qkv[:, a.H:a.H + a.Hkv])
    with torch.cuda.graph(graph):
        binding.qk_norm_rope(qkv[:, :a.H], qkv[:, a.H:a.H + a.Hkv], past, a.freq, *a.norm, q_out=qo, k_out=ko)
        binding.win_varlen_forward(a.win, 0, qo, ko, qkv[:, a.H + a.Hkv:], cu, blk, past, o, n, n,
                                   scale=a.d ** -0.5, max_seqlen_hint=1)
        binding.sel_conv_varlen_forward(a.sel, 0, x, cu, blk, has, a.w, a.b, u, n, n, max_seqlen_hint=1)
        binding.sel_scan_varlen_forward(a.sel, 0, u, step, bc[:, :a.N], bc[:, a.N:], z, cu, blk, has, a.A_log, a.D,
                                        a.bias, y, n, n, max_seqlen_hint=1)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o.view(2, 1, -1).float(), want[0]) and torch.equal(y.view(2, 1, -1).float(), want[1])
