"""Helpers of the decayed linear attention tests: stage a packed batch on the
GPU, run it through the binding and compare every output with the oracle."""
import numpy as np
import torch

from continuous_linear_attention_gb300 import binding
from oracle import lin as ref

SENTINEL = 12.5
ULP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}  # half a step, relative to the value


class LinRun:
    """A packed batch: q, k, v as views of one fused projection's rows (or,
    ``dense``, tensors of their own), states of the named blocks, and every
    other pool byte a pattern."""

    def __init__(self, lens, past, H, Hkv, d, act, seed=0, blocks=None, num_blocks=None,
                 log_decay=None, scale=None, dense=False, rows_after=0, values=None, hint=0,
                 num_layers=1, layer=0):
        g = torch.Generator().manual_seed(seed)
        self.N, self.T = len(lens), sum(lens)
        self.H, self.Hkv, self.d, self.act, self.hint = H, Hkv, d, act, hint
        self.cu = [0] + np.cumsum(lens).tolist()
        self.num_blocks = num_blocks or len(lens) + 3
        self.blk = (torch.randperm(self.num_blocks - 1, generator=g)[:self.N] + 1).tolist() \
            if blocks is None else list(blocks)
        self.has_past = [int(p) for p in past]
        self.scale = d ** -0.5 if scale is None else scale
        dtype = torch.float32 if act == "f32" else torch.bfloat16
        T = self.T + rows_after
        w = (H + 2 * Hkv) * d
        x = torch.randn(T, w, generator=g).to(dtype)
        if values is not None:
            values(x, self)
        self.x = x
        heads = [H, Hkv, Hkv]
        dev = x.cuda()
        parts = [p.unflatten(1, (-1, d)) for p in dev.split([n * d for n in heads], 1)]
        if dense:
            parts = [p.contiguous() for p in parts]
        self.q, self.k, self.v = parts
        if log_decay is None:
            log_decay = -(2.0 ** (-8.0 * torch.arange(1, H + 1) / H)) * 0.7
        self.log_decay = torch.as_tensor(log_decay, dtype=torch.float32)
        self.states = torch.randn(self.N, H, d, d, generator=g) * 0.5
        stride, total = binding.lin_layout_for(self.num_blocks, num_layers, H, d, act)
        assert stride == H * d * d * 4
        self.mem = torch.empty(total, dtype=torch.uint8, device="cuda")
        self.pool = binding.LinPool(self.num_blocks, num_layers, H, d, act, memory=self.mem)
        self.layer = layer
        self.view = self.mem.view(torch.float32).view(num_layers, self.num_blocks, H, d, d)
        self.view.copy_(torch.randn(self.view.shape[1:], generator=g).expand(self.view.shape))
        self.view[:, 0] = 0
        # (a block may be named by empty sequences too: theirs first)
        for s in sorted(range(self.N), key=lambda s: lens[s] > 0):
            if 0 < self.blk[s] < self.num_blocks:
                self.view[layer, self.blk[s]] = self.states[s].cuda()
        self.out = torch.full((T, H, d), SENTINEL, dtype=dtype, device="cuda")
        i32 = dict(dtype=torch.int32, device="cuda")
        self.cu_d = torch.tensor(self.cu, **i32)
        self.blk_d = torch.tensor(self.blk, **i32)
        self.past_d = torch.tensor(self.has_past, dtype=torch.uint8, device="cuda")
        self.decay_d = self.log_decay.cuda()
        torch.cuda.synchronize()

    def run(self, stream=None):
        binding.lin_varlen_forward(self.pool, self.layer, self.q, self.k, self.v, self.cu_d,
                                   self.blk_d, self.past_d, self.decay_d, self.out, self.T, self.N,
                                   scale=self.scale, max_seqlen_hint=self.hint, stream=stream)

    def expected(self, magnitude=False):
        H, Hkv, d = self.H, self.Hkv, self.d
        x = self.x.double().numpy()
        q, k, v = (p.reshape(len(x), -1, d) for p in np.split(x, [H * d, (H + Hkv) * d], axis=1))
        past = self.states.double().numpy() * np.array(self.has_past)[:, None, None, None]
        return ref.lin_forward(q, k, v, self.cu, past, self.log_decay.double().numpy(),
                               self.scale, magnitude)


def check(run, tensor_cores=False, before=None):
    """Compare a finished run with the oracle.

    Tolerances, element by element, from the roundings made: with A the same
    forward over absolute values, the fp32 recurrence of a sequence of n
    tokens makes at most 3 roundings per step on a state term and d + 4 in the
    output's sum (2^-24 each, relative to A), and the output is rounded once
    to its type (relative to the value).  The tensor-core form adds one bf16
    rounding (2^-8) of the weights (q k^T with the decay) and of the state as
    operands, each relative to its own part of A, and keeps the state itself
    as fp32: four bf16 terms per decayed operand (2^-27) and fp32
    accumulation, at most 32 steps per chunk (2^-23 each, should the unit
    truncate).  Below fp32's range a rounding is off by up to 2^-126 whatever
    the value, in a state term once more times q in the output."""
    skip, flags = ref.lin_skip(run.cu, run.blk, run.num_blocks, run.T, run.hint)
    got_flags = run.pool.error_flags()
    assert got_flags == flags, f"flags {got_flags:#x}, expected {flags:#x}"
    got = run.out.double().cpu().numpy()
    if flags == ref.SEQLENS:
        assert (got == SENTINEL).all(), "rows of a skipped batch written"
        return {}
    out, states = run.expected()
    mag_out, mag_states = run.expected(magnitude=True)
    view = run.view[run.layer].cpu()
    errs = {"out": 0.0, "state": 0.0}
    for s in range(run.N):
        lo, hi = run.cu[s], run.cu[s + 1]
        if skip[s]:
            assert (got[lo:hi] == SENTINEL).all(), f"rows of skipped sequence {s} written"
            continue
        n = hi - lo
        fp32 = (3 * n + run.d + 4) * 2.0 ** -24
        if tensor_cores:
            fp32 = max(fp32, 32 * (n // 128 + 1) * 2.0 ** -23)
        tol = ULP[run.act] * np.abs(out[lo:hi]) + (fp32 + (2.0 ** -8 if tensor_cores else 0.0)) \
            * mag_out[lo:hi] * (1 + 2.0 ** -7)
        tiny = (3 * n + run.d + 4) * 2.0 ** -126
        tol = tol + tiny * (1 + run.scale * run.d * np.nanmax(np.abs(run.x.double().numpy())))
        bad = np.abs(got[lo:hi] - out[lo:hi]) > tol
        assert not bad.any(), (s, np.argwhere(bad)[:4], got[lo:hi][bad][:4], out[lo:hi][bad][:4])
        st = view[run.blk[s]].double().numpy()
        bad = np.abs(st - states[s]) > fp32 * mag_states[s] + tiny
        assert not bad.any(), (s, np.argwhere(bad)[:4], st[bad][:4], states[s][bad][:4])
        nrm = np.linalg.norm
        if nrm(out[lo:hi]):
            errs["out"] = max(errs["out"], nrm(got[lo:hi] - out[lo:hi]) / nrm(out[lo:hi]))
        if nrm(states[s]):
            errs["state"] = max(errs["state"], nrm(st - states[s]) / nrm(states[s]))
    assert (got[run.T:] == SENTINEL).all(), "rows behind the last sequence written"
    if before is not None:
        same = before.clone()
        for s in range(run.N):
            if not skip[s]:
                same[run.layer, run.blk[s]] = run.view[run.layer, run.blk[s]]
        assert torch.equal(same.view(torch.int32), run.view.view(torch.int32)), \
            "blocks of no active sequence changed"
    return errs


def run_and_check(*args, tensor_cores=False, **kw):
    run = LinRun(*args, **kw)
    before = run.view.clone()
    run.run()
    torch.cuda.synchronize()
    errs = check(run, tensor_cores, before)
    return run, errs
