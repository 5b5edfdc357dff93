"""fp64 definitions of the decayed linear attention forward and of the pool's
block operations (numpy; TEST INFRASTRUCTURE ONLY, shares nothing with the
CUDA path).

  * ``lin_forward``  -- the recurrence, token by token and sequence by sequence;
  * ``lin_quadratic``-- one sequence as one masked product, an independent
                        restatement used only to pin the token loop;
  * ``lin_skip``     -- which sequences the rules for bad input skip, and why;
  * ``copy_blocks`` / ``clear_blocks`` / ``compact`` -- the block operations on
                        an array whose second axis is the blocks.
"""
from __future__ import annotations

import numpy as np

SEQLENS, BLOCK_RANGE, TRASH_WRITE, DUPLICATE, HINT = 0x1, 0x2, 0x4, 0x8, 0x20


def lin_skip(cu, blk, num_blocks, T, hint=0):
    """(skip flag per sequence, error flags) of a packed batch."""
    n = len(blk)
    if cu[0] != 0 or cu[n] != T or any(cu[i + 1] < cu[i] for i in range(n)):
        return [True] * n, SEQLENS
    skip, flags = [False] * n, 0
    named = [b for i, b in enumerate(blk) if cu[i + 1] > cu[i] and 0 < b < num_blocks]
    for i, b in enumerate(blk):
        length = cu[i + 1] - cu[i]
        if b < 0 or length == 0:
            skip[i] = True
        elif b >= num_blocks:
            skip[i], flags = True, flags | BLOCK_RANGE
        elif b == 0:
            skip[i], flags = True, flags | TRASH_WRITE
        elif named.count(b) > 1:
            skip[i], flags = True, flags | DUPLICATE
        elif hint and length > hint:
            skip[i], flags = True, flags | HINT
    return skip, flags


def lin_forward(q, k, v, cu, past, log_decay, scale, magnitude=False):
    """q [T][H][d], k and v [T][Hkv][d], past [N][H][d][d] (zeros: no past).
    Returns (out [T][H][d], states [N][H][d][d]).  With ``magnitude`` every
    product is of absolute values: what rounding errors are relative to."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    states = np.array(past, dtype=np.float64)
    if magnitude:
        q, k, v, states = np.abs(q), np.abs(k), np.abs(v), np.abs(states)
    H = q.shape[1]
    head = np.arange(H) // (H // k.shape[1])
    alpha = np.exp(np.asarray(log_decay, dtype=np.float64))[:, None, None]
    out = np.zeros_like(q)
    for s in range(len(cu) - 1):
        for t in range(cu[s], cu[s + 1]):
            states[s] = alpha * states[s] + k[t, head][:, :, None] * v[t, head][:, None, :]
            out[t] = scale * np.einsum("hk,hkv->hv", q[t], states[s])
    return out, states


def lin_quadratic(q, k, v, past, log_decay, scale):
    """One sequence and one head: o = ((q k^T) . decay) v + the past's part."""
    n = q.shape[0]
    gap = np.arange(n)[:, None] - np.arange(n)
    decay = np.where(gap >= 0, np.exp(log_decay * np.maximum(gap, 0)), 0.0)
    ages = np.arange(1, n + 1)[:, None]
    return scale * (((q @ k.T) * decay) @ v + np.exp(log_decay * ages) * (q @ past))


def copy_blocks(mem, src, dst):
    """mem [layers][blocks][...]; (new mem, flags).  All reads come first."""
    nb, flags, out = mem.shape[1], 0, mem.copy()
    ok = []
    for s, d in zip(src, dst):
        if s < 0 or d < 0:
            continue
        if s >= nb or d >= nb:
            flags |= BLOCK_RANGE
        elif d == 0:
            flags |= TRASH_WRITE
        else:
            ok.append((s, d))
    named = [d for _, d in ok]
    for s, d in ok:
        if named.count(d) > 1:
            flags |= DUPLICATE
        else:
            out[:, d] = mem[:, s]
    return out, flags


def clear_blocks(mem, idx):
    out, flags = mem.copy(), 0
    for b in idx:
        if b < 0:
            continue
        if b == 0:
            flags |= TRASH_WRITE
        elif b >= mem.shape[1]:
            flags |= BLOCK_RANGE
        else:
            out[:, b] = 0
    return out, flags


def compact(mem, idx):
    """(new mem, new indices, flags); blocks that are neither live nor moved
    into keep their contents here."""
    nb = mem.shape[1]
    live = sorted({b for b in idx if 0 < b < nb})
    m = len(live)
    holes = [b for b in range(1, m + 1) if b not in live]
    to = dict(zip([b for b in live if b > m], holes))
    out = mem.copy()
    for a, b in to.items():
        out[:, b] = mem[:, a]
    return out, [to.get(b, b) for b in idx], BLOCK_RANGE if any(b >= nb for b in idx) else 0
