"""fp64 definitions of the operators of the layers beside the linear ones
(numpy; TEST INFRASTRUCTURE ONLY, shares nothing with the CUDA path).

  * ``norm_rope``    -- RMS norm per head and the position rotation;
  * ``conv_forward`` -- causal depthwise convolution and SiLU over a packed batch;
  * ``scan_forward`` -- the selective scan, token by token, with a bound of the
                        fp32 form's roundings carried along the same recursion;
  * ``win_forward``  -- windowed attention with sinks, query by query, from the
                        keys and values of each request in order of position;
  * ``Ring``         -- what a block of the windowed pool keeps.
The rules for bad input are ``lin.lin_skip``'s, with ``win_skip`` for past lengths.
"""
from __future__ import annotations

import numpy as np

from .lin import lin_skip

RANGE = 0x40
EPS = 2.0 ** -24  # half a step of fp32, relative


def norm_rope(x, positions, inv_freq, weight=None, offset=0.0, eps=1e-6, interleaved=False):
    """x [T][heads][d] -> (y, magnitude): the magnitude is what the rotation's
    roundings are relative to, |y_a| + |y_b| before it for both of a pair."""
    y = np.array(x, dtype=np.float64)
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * (np.asarray(weight, np.float64) + offset)
    mag = np.abs(y)
    if inv_freq is None or len(inv_freq) == 0:
        return y, mag
    n = len(inv_freq)
    a, b = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    # the angle in long double: its error stays far below the bounds
    turn = np.asarray(positions, np.longdouble)[:, None] * np.asarray(inv_freq, np.float64).astype(np.longdouble)
    turn = np.fmod(turn, 2 * np.longdouble("3.14159265358979323846264338327950288"))
    cos, sin = np.cos(turn).astype(np.float64)[:, None], np.sin(turn).astype(np.float64)[:, None]
    ya, yb = y[..., a].copy(), y[..., b].copy()
    y[..., a], y[..., b] = ya * cos - yb * sin, yb * cos + ya * sin
    mag[..., a] = mag[..., b] = np.abs(ya) + np.abs(yb)
    return y, mag


def silu(x):
    return x / (1 + np.exp(-np.clip(x, -700, None)))


def conv_forward(x, w, bias, cu, past):
    """x [T][C], w [C][K], past [N][K-1][C] (zeros: no past).  Returns (out,
    pre-activations' magnitude, new states)."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    K = w.shape[1]
    out, mag, states = np.zeros_like(x), np.zeros_like(x), np.array(past, np.float64)
    for s in range(len(cu) - 1):
        line = np.concatenate([states[s], x[cu[s]:cu[s + 1]]])
        for t in range(cu[s], cu[s + 1]):
            rows = line[t - cu[s]:t - cu[s] + K]
            acc = (rows * w.T).sum(0)
            mag[t] = np.abs(rows * w.T).sum(0)
            if bias is not None:
                acc, mag[t] = acc + bias, mag[t] + np.abs(bias)
            out[t] = silu(acc)
        states[s] = line[len(line) - (K - 1):]
    return out, mag, states


def scan_forward(u, dt, B, C, z, cu, past, A_log, D=None, dt_bias=None):
    """u, dt, z (or None) [T][C], B, C [T][N], past [N][C][N].  Returns (y, its
    bound, states, their bound): how far fp32 arithmetic of the definition may
    be off, with exponentials of 2^-22 and a softplus of (4 + 3 |raw|) 2^-23
    relative, a rounding for each product and sum, and SiLU to 2^-21 + |z| 2^-22."""
    u, dt, B, C = (np.asarray(a, np.float64) for a in (u, dt, B, C))
    A = -np.exp(np.asarray(A_log, np.float64))
    y, ey = np.zeros_like(u), np.zeros_like(u)
    h = np.array(past, np.float64)
    eh = np.zeros_like(h)
    for s in range(len(cu) - 1):
        for t in range(cu[s], cu[s + 1]):
            raw = dt[t] + (0 if dt_bias is None else dt_bias)
            step = np.logaddexp(0, raw)
            e_step = (4 + 3 * np.abs(raw)) * 2 * EPS
            with np.errstate(invalid="ignore"):
                x = step[:, None] * A
            a = np.exp(x)
            e_a = 4 * EPS + np.where(a > 0, np.abs(x), 0) * (4 * EPS + e_step[:, None])
            add = (step * u[t])[:, None] * B[t]
            eh[s] = a * (eh[s] * (1 + e_a) + np.abs(h[s]) * e_a) + np.abs(add) * (e_step[:, None] + 3 * EPS)
            h[s] = a * h[s] + add
            eh[s] += EPS * np.abs(h[s]) + 2.0 ** -126
            y[t] = (h[s] * C[t]).sum(1)
            ey[t] = (eh[s] * np.abs(C[t])).sum(1) + (B.shape[1] + 2) * EPS * np.abs(h[s] * C[t]).sum(1)
            if D is not None:
                y[t] += D * u[t]
                ey[t] += EPS * (np.abs(D * u[t]) + np.abs(y[t]))
            if z is not None:
                g = silu(np.asarray(z[t], np.float64))
                ey[t] = ey[t] * np.abs(g) + np.abs(y[t] * g) * (8 + 4 * np.abs(z[t])) * EPS
                y[t] *= g
    return y, ey, h, eh


class Ring:
    """A request's keys or values as its block keeps them: [heads][sinks + window][d]."""

    def __init__(self, window, sinks):
        self.window, self.sinks = window, sinks

    def slot(self, j):
        return j if j < self.sinks else self.sinks + (j - self.sinks) % self.window

    def held(self, total):
        """The positions that are in the block after `total` tokens."""
        return list(range(min(self.sinks, total))) + list(range(max(self.sinks, total - self.window), total))


def win_skip(cu, blk, past, num_blocks, T, hint=0):
    """(skip flag per sequence, error flags) with the past lengths' rule."""
    skip, flags = lin_skip(cu, blk, num_blocks, T, hint)
    if all(skip) and flags == 0x1:
        return skip, flags
    for i, p in enumerate(past):
        length = cu[i + 1] - cu[i]
        if not skip[i] and (p < 0 or p + length > 2 ** 31 - 1):
            skip[i], flags = True, flags | RANGE
    return skip, flags


def win_forward(q, k, v, cu, past, history, window, sinks, scale, skip=None):
    """q [T][H][d], k and v [T][Hkv][d]; history[s]: {position: (key, value)}
    ([Hkv][d] each) of what the block holds, which is updated.  Returns (out, mean
    of |v| under the weights, a score's magnitude (scaled))."""
    q, k, v = (np.asarray(a, np.float64) for a in (q, k, v))
    T, H, d = q.shape
    group = H // k.shape[1]
    out, mag, score_mag = np.zeros(q.shape), np.zeros(q.shape), np.zeros((T, H))
    for s in range(len(cu) - 1):
        if skip is not None and skip[s]:
            continue
        held = history[s]
        for t in range(cu[s], cu[s + 1]):
            pos = past[s] + t - cu[s]
            held[pos] = (k[t], v[t])
            seen = [j for j in held if j <= pos and (j > pos - window or j < sinks)]
            kk = np.stack([held[j][0] for j in seen]).repeat(group, axis=1)  # [keys][H][d]
            vv = np.stack([held[j][1] for j in seen]).repeat(group, axis=1)
            score = np.einsum("hd,khd->kh", q[t], kk) * scale
            score_mag[t] = np.einsum("hd,khd->kh", np.abs(q[t]), np.abs(kk)).max(0) * abs(scale)
            w = np.exp(score - score.max(0))
            w /= w.sum(0)
            out[t] = np.einsum("kh,khd->hd", w, vv)
            mag[t] = np.einsum("kh,khd->hd", w, np.abs(vv))
        total = past[s] + cu[s + 1] - cu[s]
        keep = set(Ring(window, sinks).held(total))
        for j in [j for j in held if j not in keep]:
            del held[j]
    return out, mag, score_mag
