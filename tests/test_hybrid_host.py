"""Windowed attention, the selective scan, its convolution and the query/key
norms without a GPU: the oracle's definitions against independent restatements,
pool layouts, and the argument checks that come before any device work."""
import ctypes

import numpy as np
import pytest
import torch

from continuous_linear_attention_gb300 import binding
from oracle import hybrid as ref

NULL, DIMS, RANGE, ALIGN, NOMEM = -1, -2, -3, -4, -6


def test_rotation_is_a_complex_product_and_keeps_norms():
    rng = np.random.default_rng(0)
    x, f = rng.standard_normal((5, 2, 12)), np.array([1.0, 0.3, 0.01], np.float32)
    pos = [0, 1, 7, 100_000, 2 ** 31 - 1]
    for inter in (False, True):
        y, _ = ref.norm_rope(x, pos, f, interleaved=inter)
        a, b = (x[..., 0:6:2], x[..., 1:6:2]) if inter else (x[..., :3], x[..., 3:6])
        ya, yb = (y[..., 0:6:2], y[..., 1:6:2]) if inter else (y[..., :3], y[..., 3:6])
        turn = np.exp(1j * (np.array(pos)[:, None] * f.astype(np.float64)))[:, None]
        np.testing.assert_allclose(ya + 1j * yb, (a + 1j * b) * turn, atol=2e-6)
        np.testing.assert_allclose((y ** 2).sum(-1), (x ** 2).sum(-1), rtol=1e-12)
        np.testing.assert_array_equal(y[..., 6:], x[..., 6:])
        np.testing.assert_array_equal(y[0], x[0])
    n, _ = ref.norm_rope(x, pos, None, weight=np.full(12, 0.5), offset=1.0)
    np.testing.assert_allclose((n ** 2).mean(-1), 2.25, rtol=1e-4)


def test_convolution_is_torchs():
    rng = np.random.default_rng(1)
    x, w, bias = rng.standard_normal((9, 4)), rng.standard_normal((4, 3)), rng.standard_normal(4)
    out, _, st = ref.conv_forward(x, w, bias, [0, 9], np.zeros((1, 2, 4)))
    y = torch.nn.functional.conv1d(torch.tensor(x.T)[None], torch.tensor(w)[:, None], torch.tensor(bias),
                                   padding=2, groups=4)[0, :, :9].T
    np.testing.assert_allclose(out, torch.nn.functional.silu(y).numpy(), rtol=1e-12)
    np.testing.assert_array_equal(st[0], x[7:])
    a, _, s1 = ref.conv_forward(x[:1], w, bias, [0, 1], np.zeros((1, 2, 4)))
    b, _, s2 = ref.conv_forward(x[1:], w, bias, [0, 8], s1)
    np.testing.assert_allclose(np.concatenate([a, b]), out, rtol=1e-13)
    np.testing.assert_array_equal(s2, st)


def test_scan_is_the_sum_over_earlier_tokens():
    rng = np.random.default_rng(2)
    T, C, N = 11, 3, 4
    u, dt, z = (rng.standard_normal((T, C)) for _ in range(3))
    B, Cm = rng.standard_normal((T, N)), rng.standard_normal((T, N))
    A_log, D, bias = rng.standard_normal((C, N)), rng.standard_normal(C), rng.standard_normal(C)
    past = rng.standard_normal((1, C, N))
    y, _, h, _ = ref.scan_forward(u, dt, B, Cm, z, [0, T], past, A_log, D, bias)
    step = np.log1p(np.exp(dt + bias))
    upto = np.cumsum(step, 0)
    want = np.zeros((T, C))
    for t in range(T):
        for s in range(t + 1):
            a = np.exp(-(upto[t] - upto[s])[:, None] * np.exp(A_log))
            want[t] += (a * B[s] * Cm[t]).sum(1) * step[s] * u[s]
        want[t] += (np.exp(-upto[t][:, None] * np.exp(A_log)) * past[0] * Cm[t]).sum(1) + D * u[t]
    np.testing.assert_allclose(y, want * z / (1 + np.exp(-z)), rtol=1e-10, atol=1e-12)
    y1, _, h1, _ = ref.scan_forward(u[:4], dt[:4], B[:4], Cm[:4], z[:4], [0, 4], past, A_log, D, bias)
    y2, _, h2, _ = ref.scan_forward(u[4:], dt[4:], B[4:], Cm[4:], z[4:], [0, T - 4], h1, A_log, D, bias)
    np.testing.assert_allclose(np.concatenate([y1, y2]), y, rtol=1e-12)
    np.testing.assert_allclose(h2, h, rtol=1e-12)


@pytest.mark.parametrize("window,sinks", [(1, 0), (3, 2), (5, 0), (100, 4)])
def test_windowed_attention_is_torchs_and_splits(window, sinks):
    rng = np.random.default_rng(3)
    T, H, Hkv, d = 17, 4, 2, 8
    q, k, v = rng.standard_normal((T, H, d)), rng.standard_normal((T, Hkv, d)), rng.standard_normal((T, Hkv, d))
    out, _, _ = ref.win_forward(q, k, v, [0, T], [0], [{}], window, sinks, 0.3)
    i = np.arange(T)
    mask = (i[None] <= i[:, None]) & ((i[None] > i[:, None] - window) | (i[None] < sinks))
    t = lambda a: torch.tensor(a).transpose(0, 1)[None]  # noqa: E731
    want = torch.nn.functional.scaled_dot_product_attention(
        t(q), t(k.repeat(2, 1)), t(v.repeat(2, 1)), attn_mask=torch.tensor(mask), scale=0.3)
    np.testing.assert_allclose(out, want[0].transpose(0, 1).numpy(), rtol=1e-10, atol=1e-12)
    held = [{}]
    a, _, _ = ref.win_forward(q[:6], k[:6], v[:6], [0, 6], [0], held, window, sinks, 0.3)
    assert sorted(held[0]) == ref.Ring(window, sinks).held(6)
    b, _, _ = ref.win_forward(q[6:], k[6:], v[6:], [0, T - 6], [6], held, window, sinks, 0.3)
    np.testing.assert_allclose(np.concatenate([a, b]), out, rtol=1e-12)


def test_ring_slots():
    r = ref.Ring(4, 2)
    assert [r.slot(j) for j in range(11)] == [0, 1, 2, 3, 4, 5, 2, 3, 4, 5, 2]
    for total in range(12):
        assert len({r.slot(j) for j in r.held(total)}) == len(r.held(total))


@pytest.mark.parametrize("args", [(5, 2, 64, 16, 4, "bf16", 0), (3, 1, 8, 32, 2, "f32", 0),
                                  (3, 1, 1000, 64, 3, "bf16", 4096)])
def test_sel_layout(args):
    stride, conv, ssm, total = binding.sel_layout_for(*args)
    C, N, K = args[2:5]
    size = 4 if args[5] == "f32" else 2
    off = -(-(K - 1) * C * size // 128) * 128
    align = max(128, args[6])
    assert (conv, ssm) == (0, off)
    assert stride == -(-(off + C * N * 4) // align) * align and total == stride * args[0] * args[1]


@pytest.mark.parametrize("args", [(5, 2, 8, 128, 1024, 4, "bf16", 0), (2, 1, 1, 32, 1, 0, "bf16", 0),
                                  (4, 3, 3, 64, 77, 9, "f32", 8192)])
def test_win_layout(args):
    stride, v_off, total = binding.win_layout_for(*args)
    nb, nl, Hkv, d, w, s, act, align = args
    assert v_off == Hkv * (w + s) * d * (4 if act == "f32" else 2)
    align = max(128, align)
    assert stride == -(-2 * v_off // align) * align and total == stride * nb * nl


@pytest.mark.parametrize("args,status", [
    ((1, 1, 64, 16, 4, 0, 0), RANGE), ((4, 0, 64, 16, 4, 0, 0), RANGE), ((4, 1, 0, 16, 4, 0, 0), DIMS),
    ((4, 1, 12, 16, 4, 0, 0), DIMS), ((4, 1, 65544, 16, 4, 0, 0), DIMS), ((4, 1, 64, 8, 4, 0, 0), DIMS),
    ((4, 1, 64, 128, 4, 0, 0), DIMS), ((4, 1, 64, 16, 1, 0, 0), DIMS), ((4, 1, 64, 16, 5, 0, 0), DIMS),
    ((4, 1, 64, 16, 4, 2, 0), DIMS), ((4, 1, 64, 16, 4, 1, 64), DIMS), ((4, 1, 64, 16, 4, 1, 384), DIMS),
    ((1 << 20, 1 << 10, 64, 16, 4, 1, 0), RANGE),
])
def test_sel_pool_refusals(args, status):
    lib, out = binding.load(), ctypes.c_void_p()
    assert lib.gdn_sel_pool_layout_for(*args, None, None, None, None) == status
    assert lib.gdn_sel_pool_create(ctypes.byref(out), *args, None, 0) == status and not out.value


@pytest.mark.parametrize("args,status", [
    ((1, 1, 4, 64, 8, 0, 0, 0), RANGE), ((4, 0, 4, 64, 8, 0, 0, 0), RANGE), ((4, 1, 0, 64, 8, 0, 0, 0), DIMS),
    ((4, 1, 1025, 64, 8, 0, 0, 0), DIMS), ((4, 1, 4, 96, 8, 0, 0, 0), DIMS), ((4, 1, 4, 256, 8, 0, 0, 0), DIMS),
    ((4, 1, 4, 64, 0, 4, 0, 0), DIMS), ((4, 1, 4, 64, (1 << 20) + 1, 4, 0, 0), DIMS),
    ((4, 1, 4, 64, 8, -1, 0, 0), DIMS), ((4, 1, 4, 64, 8, 4097, 0, 0), DIMS), ((4, 1, 4, 64, 8, 4, 2, 0), DIMS),
    ((4, 1, 4, 64, 8, 4, 1, 100), DIMS), ((1 << 20, 1 << 10, 4, 64, 8, 4, 1, 0), RANGE),
])
def test_win_pool_refusals(args, status):
    lib, out = binding.load(), ctypes.c_void_p()
    assert lib.gdn_win_pool_layout_for(*args, None, None, None) == status
    assert lib.gdn_win_pool_create(ctypes.byref(out), *args, None, 0) == status and not out.value


def test_memory_too_small_or_not_aligned_is_refused_before_any_device_work():
    lib, out = binding.load(), ctypes.c_void_p()
    total = binding.sel_layout_for(4, 1, 64, 16, 4, "f32")[3]
    create = lib.gdn_sel_pool_create
    assert create(ctypes.byref(out), 4, 1, 64, 16, 4, 0, 0, 4096, total - 1) == NOMEM
    assert create(ctypes.byref(out), 4, 1, 64, 16, 4, 0, 0, 4096 + 128, total) == ALIGN
    assert create(None, 4, 1, 64, 16, 4, 0, 0, None, 0) == NULL
    total = binding.win_layout_for(4, 1, 2, 64, 8, 1, "f32")[2]
    create = lib.gdn_win_pool_create
    assert create(ctypes.byref(out), 4, 1, 2, 64, 8, 1, 0, 0, 4096, total - 1) == NOMEM
    assert create(ctypes.byref(out), 4, 1, 2, 64, 8, 1, 0, 0, 4096 + 128, total) == ALIGN
    assert create(None, 4, 1, 2, 64, 8, 1, 0, 0, None, 0) == NULL


def test_forwards_without_a_pool():
    lib = binding.load()
    w = binding.SelWeights(None, None, None)
    assert lib.gdn_sel_conv_varlen_forward(None, 0, None, 0, *[None] * 6, 0, 0, 0, 0, None) == NULL
    assert lib.gdn_sel_scan_varlen_forward(None, 0, *[None, 0] * 5, None, None, None, ctypes.byref(w),
                                           None, 0, 0, 0, 0, None) == NULL
    assert lib.gdn_win_varlen_forward(None, 0, None, None, None, 0, 0, 0, 1, None, None, None, 1.0, None, 0,
                                      0, 0, 0, None) == NULL


def rope_status(**kw):
    """A call's status with the given arguments wrong; the addresses are never followed."""
    a = dict(q=4096, k=8192, ldq=256, ldk=128, positions=4096, inv_freq=4096, rot=64, inter=0, qw=None, kw=None,
             offset=0.0, eps=1e-6, T=3, H=4, Hkv=2, d=64, act=1, qo=4096, ko=8192, ldqo=256, ldko=128)
    assert set(kw) <= set(a)
    a.update(kw)
    return binding.load().gdn_qk_norm_rope(
        a["q"], a["k"], a["ldq"], a["ldk"], a["positions"], a["inv_freq"], a["rot"], a["inter"], a["qw"], a["kw"],
        a["offset"], a["eps"], a["T"], a["H"], a["Hkv"], a["d"], a["act"], a["qo"], a["ko"], a["ldqo"], a["ldko"],
        None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), RANGE), (dict(eps=-1.0), RANGE), (dict(eps=float("nan")), RANGE), (dict(H=-1), DIMS),
    (dict(H=0, Hkv=0), DIMS), (dict(H=4097, ldq=1 << 20, ldqo=1 << 20), DIMS), (dict(d=96), DIMS),
    (dict(d=16), DIMS), (dict(rot=63), DIMS), (dict(rot=66), DIMS), (dict(rot=-2), DIMS), (dict(act=2), DIMS),
    (dict(q=None), NULL), (dict(ko=None), NULL), (dict(positions=None), NULL), (dict(inv_freq=None), NULL),
    (dict(q=4104), ALIGN), (dict(ko=8200), ALIGN), (dict(ldq=260), ALIGN), (dict(ldko=132), ALIGN),
    (dict(ldq=248), RANGE), (dict(ldk=120), RANGE), (dict(ldqo=1 << 39), RANGE), (dict(T=0, q=None), 0),
])
def test_rope_refusals(kw, status):
    assert rope_status(**kw) == status


def test_binding_refuses_what_it_cannot_pass_on():
    t = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype)  # noqa: E731
    with pytest.raises(ValueError):
        binding.qk_norm_rope(t(3, 256), t(3, 2, 64), t(3, dtype=torch.int32), None)
    with pytest.raises(ValueError):  # tensors of the host
        binding.qk_norm_rope(t(3, 4, 64), t(3, 2, 64), t(3, dtype=torch.int32), None)

    class Pool:
        dims, dtype, device, handle = (4, 1, 2, 64, 8, 1), torch.bfloat16, 0, None

    i32 = dict(dtype=torch.int32)
    for q, k in ((t(3, 256), t(3, 2, 64)), (t(3, 4, 64), t(3, 3, 64)), (t(2, 4, 64), t(3, 2, 64)),
                 (t(3, 4, 64), t(3, 2, 64))):
        with pytest.raises(ValueError):
            binding.win_varlen_forward(Pool, 0, q, k, t(3, 2, 64), t(2, **i32), t(1, **i32), t(1, **i32),
                                       t(3, 4, 64), 3, 1)

    class Sel:
        dims, dtype, device, handle = (4, 1, 64, 16, 4), torch.bfloat16, 0, None

    with pytest.raises(ValueError):
        binding.sel_conv_varlen_forward(Sel, 0, t(3, 60), t(2, **i32), t(1, **i32), t(1, dtype=torch.uint8),
                                        t(64, 4), None, t(3, 64), 3, 1)
