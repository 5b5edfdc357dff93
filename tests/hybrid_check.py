"""Helpers of the tests of windowed attention, the selective scan, its
convolution and the query/key norms: stage a packed batch on the GPU, run it
through the binding and compare every output with the oracle.

Tolerances are element by element, from the roundings made (ULP: half a step,
relative to the value)."""
import numpy as np
import torch

from continuous_linear_attention_gb300 import binding
from oracle import hybrid as ref
from oracle.lin import SEQLENS, lin_skip

SENTINEL = 12.5
ULP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
EPS = 2.0 ** -24
I32 = dict(dtype=torch.int32, device="cuda")


def dtype_of(act):
    return torch.float32 if act == "f32" else torch.bfloat16


def bits(t):
    return t.contiguous().view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)


def f64(t):
    return t.detach().double().cpu().numpy()


def close(got, want, tol, what):
    """|got - want| <= tol where want is finite; the same infinities and NaN elsewhere."""
    got, want, tol = (np.asarray(a, np.float64) for a in (got, want, tol))
    fine = np.isfinite(want)
    bad = np.where(fine, ~(np.abs(got - np.where(fine, want, 0)) <= tol),
                   ~((got == want) | (np.isnan(got) & np.isnan(want))))
    assert not bad.any(), (what, np.argwhere(bad)[:4], got[bad][:4], want[bad][:4],
                           np.broadcast_to(tol, bad.shape)[bad][:4])


class Packed:
    """What the packed batches share: lengths, blocks, and rows wider than they need be."""

    def batch(self, lens, num_blocks, blocks, g, T=None, rows_after=0):
        self.lens, self.N = list(lens), len(lens)
        self.T = sum(lens) if T is None else T
        self.rows = sum(lens) + rows_after
        self.cu = [0] + np.cumsum(lens).tolist()
        self.num_blocks = num_blocks or len(lens) + 3
        self.blk = (torch.randperm(self.num_blocks - 1, generator=g)[:self.N] + 1).tolist() \
            if blocks is None else list(blocks)
        self.cu_d, self.blk_d = torch.tensor(self.cu, **I32), torch.tensor(self.blk, **I32)

    def pool_memory(self, total, g):
        """Every byte of the pool a pattern, the trash blocks zeros."""
        self.mem = torch.empty(total, dtype=torch.uint8, device="cuda")
        return self.mem

    def untouched(self, before, skip):
        """Blocks of no active sequence, and other layers, as they were."""
        now = self.mem.view(self.num_layers, self.num_blocks, -1)
        then = before.view(self.num_layers, self.num_blocks, -1).clone()
        for s in range(self.N):
            if not skip[s]:
                then[self.layer, self.blk[s]] = now[self.layer, self.blk[s]]
        assert torch.equal(then, now), "blocks of no active sequence changed"


class SelRun(Packed):
    """A batch of the selective scan's convolution and scan (separate inputs)."""

    def __init__(self, lens, past, channels, N=16, K=4, act="bf16", seed=0, blocks=None, num_blocks=None,
                 bias=True, gate=True, skip_weight=True, hint=0, rows_after=0, values=None, num_layers=1,
                 layer=0, A_log=None, dt_bias=None, dense=False, segment=0):
        g = torch.Generator().manual_seed(seed)
        self.batch(lens, num_blocks, blocks, g, rows_after=rows_after)
        self.segment = segment
        C, dt = channels, dtype_of(act)
        self.C, self.n, self.K, self.act, self.hint = C, N, K, act, hint
        self.num_layers, self.layer = num_layers, layer
        rand = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        xz, low, wide = rand(self.rows, 2 * C), rand(self.rows, 8 + 2 * N), rand(self.rows, 2 * C)
        self.host = dict(x=xz[:, :C], z=xz[:, C:], B=low[:, 8:8 + N], C=low[:, 8 + N:],
                         u=wide[:, :C], dt=wide[:, C:] * 0.5)
        if values is not None:
            values(self.host, self)
        self.host = {k: v.to(dt) for k, v in self.host.items()}
        full = {"xz": torch.cat([self.host["x"], self.host["z"]], 1).cuda(),
                "low": torch.cat([low[:, :8].to(dt), self.host["B"], self.host["C"]], 1).cuda(),
                "wide": torch.cat([self.host["u"], self.host["dt"]], 1).cuda()}
        part = (lambda t: t.contiguous()) if dense else (lambda t: t)
        self.x, self.z = part(full["xz"][:, :C]), part(full["xz"][:, C:]) if gate else None
        self.B, self.Cm = part(full["low"][:, 8:8 + N]), part(full["low"][:, 8 + N:])
        self.u, self.dt = part(full["wide"][:, :C]), part(full["wide"][:, C:])
        self.w = (rand(C, K) * 0.5).to(dt)
        self.b = (rand(C) * 0.3).to(dt) if bias else None
        self.A_log = torch.log(torch.arange(1, N + 1).float()) + 0.1 * rand(C, N) if A_log is None else A_log
        self.D = 1 + 0.1 * rand(C) if skip_weight else None
        self.dt_bias = rand(C) - 3 if dt_bias is None else dt_bias
        stride, _, off, total = binding.sel_layout_for(self.num_blocks, num_layers, C, N, K, act)
        self.mem = torch.empty(total, dtype=torch.uint8, device="cuda")
        self.pool = binding.SelPool(self.num_blocks, num_layers, C, N, K, act, memory=self.mem)
        self.mem.copy_(torch.randint(0, 60, (total,), dtype=torch.uint8, generator=g))
        page = self.mem.view(num_layers, self.num_blocks, stride)
        page[:, 0] = 0
        size = 4 if act == "f32" else 2
        self.conv = page[layer, :, :(K - 1) * C * size].view(dt).unflatten(1, (K - 1, C))
        self.ssm = page[layer, :, off:off + C * N * 4].view(torch.float32).unflatten(1, (C, N))
        self.has_past = [int(p) for p in past]
        self.past_conv, self.past_ssm = rand(self.N, K - 1, C).to(dt), rand(self.N, C, N)
        for s in sorted(range(self.N), key=lambda s: lens[s] > 0):
            if 0 < self.blk[s] < self.num_blocks:
                self.conv[self.blk[s]], self.ssm[self.blk[s]] = self.past_conv[s].cuda(), self.past_ssm[s].cuda()
        self.past_d = torch.tensor(self.has_past, dtype=torch.uint8, device="cuda")
        self.out = torch.full((self.rows, C + 8), SENTINEL, dtype=dt, device="cuda")[:, :C]
        self.dev = [None if t is None else t.cuda() for t in (self.w, self.b, self.A_log, self.D, self.dt_bias)]
        self.before = self.mem.clone()
        torch.cuda.synchronize()

    def run_conv(self, stream=None):
        binding.sel_conv_varlen_forward(self.pool, self.layer, self.x, self.cu_d, self.blk_d, self.past_d,
                                        self.dev[0], self.dev[1], self.out, self.T, self.N,
                                        max_seqlen_hint=self.hint, stream=stream)

    def run_scan(self, stream=None):
        binding.sel_scan_varlen_forward(self.pool, self.layer, self.u, self.dt, self.B, self.Cm, self.z,
                                        self.cu_d, self.blk_d, self.past_d, self.dev[2], self.dev[3],
                                        self.dev[4], self.out, self.T, self.N, max_seqlen_hint=self.hint,
                                        stream=stream)

    def _rows(self, skip, got):
        for s in range(self.N):
            if skip[s]:
                assert (got[self.cu[s]:self.cu[s + 1]] == SENTINEL).all(), f"rows of skipped sequence {s} written"
        assert (got[self.cu[-1]:] == SENTINEL).all(), "rows behind the last sequence written"

    def check(self, what):
        skip, flags = lin_skip(self.cu, self.blk, self.num_blocks, self.T, self.hint)
        seen = self.pool.error_flags()
        assert seen == flags, f"flags {seen:#x}, expected {flags:#x}"
        got = f64(self.out)
        self.untouched(self.before, skip)
        if flags == SEQLENS:
            assert (got == SENTINEL).all()
            return
        self._rows(skip, got)
        live = [s for s in range(self.N) if not skip[s]]
        h = {k: f64(v) for k, v in self.host.items()}
        has = np.array(self.has_past)
        with np.errstate(all="ignore"):
            if what == "conv":
                past = f64(self.past_conv) * has[:, None, None]
                out, mag, states = ref.conv_forward(h["x"], f64(self.w), None if self.b is None else f64(self.b),
                                                    self.cu, past)
                # K products and sums, SiLU's slope of 1.1 at most, its exponential and quotient
                tol = 1.1 * (self.K + 1) * EPS * mag + np.abs(out) * (8 + 4 * mag) * EPS + ULP[self.act] * np.abs(out)
                for s in live:
                    rows = slice(self.cu[s], self.cu[s + 1])
                    close(got[rows], out[rows], tol[rows] + 2.0 ** -126, ("out", s))
                    st = self.conv[self.blk[s]].cpu()
                    want = torch.tensor(states[s]).to(st.dtype)
                    assert torch.equal(torch.nan_to_num(st), torch.nan_to_num(want)), ("conv state", s)
            else:
                past = f64(self.past_ssm) * has[:, None, None]
                y, ey, hs, eh = ref.scan_forward(
                    h["u"], h["dt"], h["B"], h["C"], h["z"] if self.z is not None else None, self.cu, past,
                    f64(self.A_log), None if self.D is None else f64(self.D),
                    None if self.dt_bias is None else f64(self.dt_bias))
                # a start of a segment decays by e^x, x the sum of its tokens' in fp32: off by
                # segment EPS |x| e^x, which is segment EPS / e at most, and as much again
                # from the starts before it
                far = 2 * self.segment * EPS / np.e * max(np.abs(past).max(), np.abs(hs).max())
                if far:
                    gate = 1 if self.z is None else np.abs(ref.silu(h["z"]))
                    ey = ey + far * np.abs(h["C"]).sum(1, keepdims=True) * gate
                    eh = eh + far
                for s in live:
                    rows = slice(self.cu[s], self.cu[s + 1])
                    close(got[rows], y[rows], ey[rows] + ULP[self.act] * np.abs(y[rows]) + 2.0 ** -126, ("y", s))
                    close(f64(self.ssm[self.blk[s]]), hs[s], eh[s], ("state", s))


def sel_check(what, *args, **kw):
    run = SelRun(*args, **kw)
    run.run_conv() if what == "conv" else run.run_scan()
    torch.cuda.synchronize()
    run.check(what)
    return run


class WinRun(Packed):
    """A batch of windowed attention: q, k and v as views of one projection's rows."""

    def __init__(self, lens, past, H, Hkv, d, window, sinks, act="bf16", seed=0, blocks=None, num_blocks=None,
                 hint=0, rows_after=0, values=None, history=None, num_layers=1, layer=0, scale=None, dense=False):
        g = torch.Generator().manual_seed(seed)
        self.batch(lens, num_blocks, blocks, g, rows_after=rows_after)
        self.H, self.Hkv, self.d, self.window, self.sinks = H, Hkv, d, window, sinks
        self.act, self.hint, self.past = act, hint, [int(p) for p in past]
        self.num_layers, self.layer = num_layers, layer
        self.scale = d ** -0.5 if scale is None else scale
        dt = dtype_of(act)
        x = torch.randn(self.rows, H + 2 * Hkv, d, generator=g)
        if values is not None:
            values(x, self)
        self.x = x.to(dt)
        dev = self.x.cuda()
        self.q, self.k, self.v = dev[:, :H], dev[:, H:H + Hkv], dev[:, H + Hkv:]
        if dense:
            self.q, self.k, self.v = (t.contiguous() for t in (self.q, self.k, self.v))
        stride, v_off, total = binding.win_layout_for(self.num_blocks, num_layers, Hkv, d, window, sinks, act)
        self.mem = torch.empty(total, dtype=torch.uint8, device="cuda")
        self.pool = binding.WinPool(self.num_blocks, num_layers, Hkv, d, window, sinks, act, memory=self.mem)
        # what no position holds is NaN
        self.mem.view(dt).fill_(float("nan"))
        page = self.mem.view(num_layers, self.num_blocks, stride)
        page[:, 0] = 0
        self.kv = page[layer, :, :2 * v_off].view(dt).unflatten(1, (2, Hkv, sinks + window, d))
        ring = ref.Ring(window, sinks)
        self.history = []
        for s in range(self.N):
            held = {}
            if 0 <= self.past[s] < 2 ** 31 - 1:
                pos = ring.held(self.past[s])
                rows = torch.randn(len(pos), 2, Hkv, d, generator=g).to(dt)
                if history is not None:
                    history(rows, pos, s)
                held = {j: (f64(r[0]), f64(r[1])) for j, r in zip(pos, rows)}
                if 0 < self.blk[s] < self.num_blocks and lens[s] > 0 and pos:
                    at = torch.tensor([ring.slot(j) for j in pos], device="cuda")
                    self.kv[self.blk[s]][:, :, at] = rows.permute(1, 2, 0, 3).cuda()
            self.history.append(held)
        self.out = torch.full((self.rows, H, d), SENTINEL, dtype=dt, device="cuda")
        self.past_d = torch.tensor(self.past, **I32)
        self.before = self.mem.clone()
        torch.cuda.synchronize()

    def run(self, stream=None):
        binding.win_varlen_forward(self.pool, self.layer, self.q, self.k, self.v, self.cu_d, self.blk_d,
                                   self.past_d, self.out, self.T, self.N, scale=self.scale,
                                   max_seqlen_hint=self.hint, stream=stream)

    def check(self):
        skip, flags = ref.win_skip(self.cu, self.blk, self.past, self.num_blocks, self.T, self.hint)
        seen = self.pool.error_flags()
        assert seen == flags, f"flags {seen:#x}, expected {flags:#x}"
        got = f64(self.out)
        self.untouched(self.before, skip)
        if flags == SEQLENS:
            assert (got == SENTINEL).all()
            return
        H, Hkv = self.H, self.Hkv
        x = f64(self.x)
        with np.errstate(all="ignore"):
            out, mag, score = ref.win_forward(x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:], self.cu, self.past,
                                              self.history, self.window, self.sinks, self.scale, skip)
        ring = ref.Ring(self.window, self.sinks)
        for s in range(self.N):
            rows = slice(self.cu[s], self.cu[s + 1])
            if skip[s]:
                assert (got[rows] == SENTINEL).all(), f"rows of skipped sequence {s} written"
                continue
            # a score's sum of d products and its scaling, in a weight twice over (its own and the
            # maximum's); a weight's exponential, its rounding to bf16 (in that form) and the sums
            # over the keys, in numerator and denominator
            keys = min(self.window, self.past[s] + self.lens[s]) + self.sinks
            weight = 2 * (self.d + 8) * EPS * score[rows][..., None] + 16 * EPS + \
                (2.0 ** -8 if self.act == "bf16" else 0)
            tol = (2 * weight + 2 * (keys + 16) * EPS) * mag[rows] + ULP[self.act] * np.abs(out[rows])
            close(got[rows], out[rows], tol + 2.0 ** -126, ("out", s))
            total = self.past[s] + self.lens[s]
            at = torch.tensor([ring.slot(j) for j in ring.held(total)], device="cuda")
            kv = f64(self.kv[self.blk[s]][:, :, at])
            want = np.stack([np.stack(self.history[s][j]) for j in ring.held(total)]).transpose(1, 2, 0, 3)
            np.testing.assert_array_equal(kv, want, err_msg=f"ring of sequence {s}")
            # slots that hold no position are as they were
            free = [i for i in range(self.sinks + self.window) if i not in set(at.tolist())]
            if free:
                was = self.before.view(self.num_layers, self.num_blocks, -1)[self.layer, self.blk[s]]
                was = was[:self.kv[0].numel() * self.kv.element_size()].view(self.kv.dtype).view(self.kv[0].shape)
                assert torch.equal(bits(was[:, :, free]), bits(self.kv[self.blk[s]][:, :, free]))
        assert (got[self.cu[-1]:] == SENTINEL).all(), "rows behind the last sequence written"


def win_check(*args, **kw):
    run = WinRun(*args, **kw)
    run.run()
    torch.cuda.synchronize()
    run.check()
    return run
