"""Tensors of decayed linear attention and of the block operations that lie on
another device than the pool are refused by the binding (no GPU needed: stand-ins
with a tensor's attributes)."""
import types

import pytest
import torch

from continuous_linear_attention_gb300 import binding


class OnDevice:
    """A dense tensor's attributes, on a CUDA device of one's choice."""

    def __init__(self, shape, dtype, device):
        self._like = torch.empty(shape, dtype=dtype)
        self.shape, self.dtype, self.is_cuda = self._like.shape, dtype, True
        self.device = torch.device("cuda", device)

    def get_device(self):
        return self.device.index

    def data_ptr(self):
        return 4096

    def __len__(self):
        return len(self._like)

    def __getattr__(self, name):  # dim, numel, stride, is_contiguous
        return getattr(self._like, name)


class Library:
    """Takes the place of the library; counts the calls that got there."""
    calls = 0

    def __getattr__(self, name):
        def entry(*args):
            self.calls += 1
            return 0
        return entry


@pytest.fixture
def library(monkeypatch):
    lib = Library()
    monkeypatch.setattr(binding, "load", lambda: lib)
    return lib


def pool(cls, **kw):
    p = cls.__new__(cls)
    p.__dict__.update(handle=types.SimpleNamespace(value=None), device=0, **kw)
    return p


@pytest.mark.parametrize("wrong", ["", "q", "k", "v", "out", "cu_seqlens", "state_block_idx", "has_past",
                                   "log_decay"])
def test_forward(library, wrong):
    f, i = torch.float32, torch.int32
    shapes = dict(q=((3, 4, 64), f), k=((3, 2, 64), f), v=((3, 2, 64), f), out=((3, 4, 64), f),
                  cu_seqlens=((3,), i), state_block_idx=((2,), i), has_past=((2,), torch.uint8),
                  log_decay=((4,), f))
    kw = {n: OnDevice(s, t, 1 if n == wrong else 0) for n, (s, t) in shapes.items()}
    p = pool(binding.LinPool, dims=(3, 1, 4, 64), dtype=f)
    if not wrong:
        binding.lin_varlen_forward(p, 0, T=3, N=2, stream=7, **kw)
        assert library.calls == 1
        return
    with pytest.raises(ValueError, match="cuda:0"):
        binding.lin_varlen_forward(p, 0, T=3, N=2, stream=7, **kw)
    assert library.calls == 0


def test_block_operations(library):
    p = pool(binding.Pool)
    here, there = (OnDevice((2,), torch.int32, dev) for dev in (0, 1))
    p.copy_blocks(here, here, stream=7)
    p.clear_blocks(here, stream=7)
    p.compact(here, here, stream=7)
    assert library.calls == 3
    for call in (lambda: p.copy_blocks(here, there, stream=7), lambda: p.copy_blocks(there, here, stream=7),
                 lambda: p.clear_blocks(there, stream=7), lambda: p.compact(there, stream=7),
                 lambda: p.compact(here, there, stream=7)):
        with pytest.raises(ValueError, match="cuda:0"):
            call()
    assert library.calls == 3


def test_keys_without_heads_are_refused(library):
    flat = OnDevice((192,), torch.float32, 0)
    with pytest.raises(ValueError):
        binding.lin_varlen_forward(pool(binding.LinPool, dims=(3, 1, 1, 64), dtype=torch.float32), 0, flat,
                                   flat, flat, flat, flat, flat, flat, flat, 3, 1, stream=7)
    assert library.calls == 0


def test_a_pool_in_host_memory_is_refused(library, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(ValueError):
        binding.LinPool(3, 1, 1, 32, "f32", memory=torch.empty(3 * 4096, dtype=torch.uint8))
    with pytest.raises(ValueError):
        binding.LinPool(3, 1, 1, 32, "f32", memory=OnDevice((3 * 4096,), torch.uint8, 1))
    assert library.calls == 0
