"""The rotation's angle at far positions and for frequencies above 1: it is off
by its rounding to fp32 alone."""
import numpy as np
import pytest
import torch

from continuous_linear_attention_gb300 import binding
from hybrid_check import EPS, close, f64
from oracle import hybrid as ref

POSITIONS = [0, 1, 77_777, 1_000_001, 16_777_217, 123_456_789, 987_654_321, 2 ** 31 - 2, 2 ** 31 - 1]


def pi_over(position, f):
    """(sin, cos) of position * f in integers: the angle modulo 2 pi to 2^-120 of
    a turn, from 1 / 2 pi to 400 bits (Machin's formula for pi)."""
    bits = 400

    def arctan_inv(x):
        total, term, k = 0, (1 << bits) // x, 0
        while term:
            total += (-term if k & 1 else term) // (2 * k + 1)
            term //= x * x
            k += 1
        return total

    pi = 4 * (4 * arctan_inv(5) - arctan_inv(239))
    num, den = float(f).as_integer_ratio()
    turns = (int(position) * num << 2 * bits) // (2 * den * pi)  # of 2^bits to a turn
    part = (turns % (1 << bits)) >> (bits - 80)
    angle = 2 * np.longdouble("3.14159265358979323846264338327950288") * np.longdouble(part) / np.longdouble(2 ** 80)
    return float(np.sin(angle)), float(np.cos(angle))


@pytest.mark.gpu
@pytest.mark.parametrize("base", [10000.0, 1.0, 0.001, 1e-6])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("sign", [1, -1])
def test_far_positions_and_high_frequencies(base, inter, sign):
    d = 64
    g = torch.Generator().manual_seed(0)
    x = torch.randn(len(POSITIONS), 2, d, generator=g)
    f = torch.tensor(sign * base ** (-np.arange(0, d, 2) / d) * (1 + 1e-3 * np.arange(d // 2)), dtype=torch.float32)
    q = x.cuda()
    out = torch.zeros_like(q)
    binding.qk_norm_rope(q, None, torch.tensor(POSITIONS, dtype=torch.int32, device="cuda"), f.cuda(), q_out=out,
                         interleaved=inter)
    torch.cuda.synchronize()
    y = f64(x)
    a, b = (slice(0, d, 2), slice(1, d, 2)) if inter else (slice(0, d // 2), slice(d // 2, d))
    sc = np.array([[pi_over(p, v) for v in f.tolist()] for p in POSITIONS])  # [T][d/2][2]
    sin, cos = sc[:, None, :, 0], sc[:, None, :, 1]
    want, mag = y.copy(), y.copy()
    want[..., a], want[..., b] = y[..., a] * cos - y[..., b] * sin, y[..., b] * cos + y[..., a] * sin
    mag[..., a] = mag[..., b] = np.abs(y[..., a]) + np.abs(y[..., b])
    # sine and cosine to 2^-22 and 6 roundings, the angle rounded to 24 bits of half a turn at
    # most (pi 2^-24), and 2^-32 of a turn cut off before
    tol = (4 * EPS + 6 * EPS + np.pi * EPS + 2 * np.pi * 2.0 ** -31) * mag + 2.0 ** -126
    close(f64(out), want, tol, "rows")


def test_the_integers_agree_with_the_oracle_at_near_positions():
    y, _ = ref.norm_rope(np.array([[[1.0, 0.0]]] * 3), [1, 5, 4000], np.array([0.37], np.float32))
    for row, p in zip(y[:, 0], [1, 5, 4000]):
        sin, cos = pi_over(p, np.float32(0.37))
        assert abs(row[0] - cos) < 1e-12 and abs(row[1] - sin) < 1e-12
