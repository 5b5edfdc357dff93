"""Decayed linear attention and the block operations without a GPU: the
oracle's definitions against independent restatements, pool layouts, and the
argument checks that come before any device work."""
import ctypes

import numpy as np
import pytest

from continuous_linear_attention_gb300 import binding
from oracle import lin as ref

NULL, DIMS, RANGE, ALIGN = -1, -2, -3, -4


@pytest.mark.parametrize("log_decay", [0.0, -0.003, -1.0, -40.0, -np.inf])
def test_recurrence_is_the_masked_product(log_decay):
    rng = np.random.default_rng(3)
    q, k, v = (rng.standard_normal((37, 1, 8)) for _ in range(3))
    past = rng.standard_normal((1, 1, 8, 8))
    out, _ = ref.lin_forward(q, k, v, [0, 37], past, [log_decay], 0.3)
    g = max(log_decay, -1e30)
    want = ref.lin_quadratic(q[:, 0], k[:, 0], v[:, 0], past[0, 0], g, 0.3)
    np.testing.assert_allclose(out[:, 0], want, rtol=1e-12, atol=1e-12)


def test_recurrence_split_equals_whole_and_heads_share_keys():
    rng = np.random.default_rng(4)
    q, k, v = rng.standard_normal((20, 4, 8)), *(rng.standard_normal((20, 2, 8)) for _ in range(2))
    g = [-0.1, -0.2, 0.0, -3.0]
    past = rng.standard_normal((1, 4, 8, 8))
    out, st = ref.lin_forward(q, k, v, [0, 20], past, g, 1.0)
    o1, s1 = ref.lin_forward(q[:7], k[:7], v[:7], [0, 7], past, g, 1.0)
    o2, s2 = ref.lin_forward(q[7:], k[7:], v[7:], [0, 13], s1, g, 1.0)
    np.testing.assert_allclose(np.concatenate([o1, o2]), out, rtol=1e-13)
    np.testing.assert_allclose(s2, st, rtol=1e-13)
    for h in range(4):
        want = ref.lin_quadratic(q[:, h], k[:, h // 2], v[:, h // 2], past[0, h], g[h], 1.0)
        np.testing.assert_allclose(out[:, h], want, rtol=1e-11, atol=1e-12)


def test_copy_lists_read_before_they_write():
    mem = np.arange(12.0).reshape(2, 6)
    out, flags = ref.copy_blocks(mem, [1, 2, 3, 3], [2, 3, 1, 5])
    assert flags == 0
    np.testing.assert_array_equal(out[0], [0, 3, 1, 2, 4, 3])
    assert ref.copy_blocks(mem, [1, 2], [3, 3])[1] == ref.DUPLICATE
    assert ref.compact(mem, [5, 2, 5])[1] == [1, 2, 1]


@pytest.mark.parametrize("H,d,act,align,stride", [
    (16, 128, "bf16", 0, 16 * 65536), (1, 32, "f32", 0, 4096), (3, 64, "bf16", 1 << 16, 1 << 16),
])
def test_layout(H, d, act, align, stride):
    assert binding.lin_layout_for(5, 2, H, d, act, align) == (stride, stride * 10)


@pytest.mark.parametrize("args,status", [
    ((1, 1, 4, 64, 0, 0), RANGE), ((4, 0, 4, 64, 0, 0), RANGE), ((4, 1, 0, 64, 0, 0), DIMS),
    ((4, 1, 4097, 64, 0, 0), DIMS), ((4, 1, 4, 96, 0, 0), DIMS), ((4, 1, 4, 64, 2, 0), DIMS),
    ((4, 1, 4, 64, 1, 64), DIMS), ((4, 1, 4, 64, 1, 384), DIMS), ((1 << 20, 1 << 11, 4, 64, 1, 0), RANGE),
])
def test_layout_refusals(args, status):
    assert binding.load().gdn_lin_pool_layout_for(*args, None, None) == status


def test_null_arguments_are_refused_without_device_work():
    lib = binding.load()
    out = ctypes.c_void_p()
    assert lib.gdn_lin_pool_create(None, 4, 1, 4, 64, 0, 0, None, 0) == NULL
    assert lib.gdn_lin_pool_create(ctypes.byref(out), 4, 1, 4, 65, 0, 0, None, 0) == DIMS
    assert lib.gdn_lin_pool_create(ctypes.byref(out), 4, 1, 4, 64, 0, 0, 256, 8) == -6
    assert lib.gdn_lin_pool_create(ctypes.byref(out), 4, 1, 1, 32, 0, 0, 16, 1 << 20) == ALIGN
    assert not out.value
    assert lib.gdn_lin_varlen_forward(None, 0, *[None] * 3, 0, 0, 0, 1, *[None] * 4, 1.0, None, 0,
                                      0, 0, 0, None) == NULL
    assert lib.gdn_state_pool_copy_blocks(None, 0, None, None, 0, None) == NULL
    assert lib.gdn_state_pool_clear_blocks(None, 0, None, 0, None) == NULL
    assert lib.gdn_state_pool_compact(None, None, None, 0, None) == NULL


def test_binding_refuses_index_lists_it_cannot_pass():
    import torch
    for bad in (torch.zeros(3, dtype=torch.int64), torch.zeros(3, dtype=torch.int32)):
        with pytest.raises(ValueError):
            binding._index(bad)
