"""Thin ctypes binding of libgdn.so (include/gdn.h).

Argument marshalling only: every step of the forward runs in the library's
CUDA kernels.  Torch tensors are accepted for convenience and passed as raw
device pointers; the current torch stream is used unless one is given.  If
the library is missing the import fails loudly: there is no other path.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

from . import build as _build

GDN_OK = 0
GDN_F32 = 0
GDN_BF16 = 1
FLAG_SEQLENS = 0x1
FLAG_BLOCK_RANGE = 0x2
FLAG_TRASH_WRITE = 0x4
FLAG_DUPLICATE = 0x8
FLAG_TIMEOUT = 0x10
FLAG_HINT = 0x20
FLAG_RANGE = 0x40

EXPORTED = [
    "gdn_state_pool_layout_for",
    "gdn_state_pool_create",
    "gdn_state_pool_destroy",
    "gdn_state_pool_layout",
    "gdn_state_pool_copy_block",
    "gdn_state_pool_reserve",
    "gdn_varlen_forward",
    "gdn_varlen_forward_noalloc",
    "gdn_kda_varlen_forward",
    "gdn_ssd_pool_layout_for",
    "gdn_ssd_pool_create",
    "gdn_ssd_varlen_forward",
    "gdn_get_error",
    "gdn_pool_set_timing_events",
    "gdn_prefill_scratch_bytes", "gdn_pool_last_prefill_path",
    "gdn_in_proj",
    "gdn_out_proj",
    "gdn_state_pool_copy_blocks",
    "gdn_state_pool_clear_blocks",
    "gdn_state_pool_compact",
    "gdn_lin_pool_layout_for",
    "gdn_lin_pool_create",
    "gdn_lin_varlen_forward",
    "gdn_sel_pool_layout_for",
    "gdn_sel_pool_create",
    "gdn_sel_conv_varlen_forward",
    "gdn_sel_scan_varlen_forward",
    "gdn_win_pool_layout_for",
    "gdn_win_pool_create",
    "gdn_win_varlen_forward",
    "gdn_qk_norm_rope",
    "gdn_status_string",
]

PREFILL_NONE, PREFILL_SPLIT, PREFILL_FUSED, PREFILL_SERIAL = 0, 1, 2, 3


class GdnError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


class Weights(ctypes.Structure):
    _fields_ = [("conv_w", ctypes.c_void_p), ("A_log", ctypes.c_void_p),
                ("dt_bias", ctypes.c_void_p)]


class SsdWeights(ctypes.Structure):
    _fields_ = [("conv_w", ctypes.c_void_p), ("A_log", ctypes.c_void_p),
                ("dt_bias", ctypes.c_void_p), ("D", ctypes.c_void_p)]


class SelWeights(ctypes.Structure):
    _fields_ = [("A_log", ctypes.c_void_p), ("D", ctypes.c_void_p), ("dt_bias", ctypes.c_void_p)]


_lib = None


def lib_path() -> str:
    return _build.LIB_PATH


def load() -> ctypes.CDLL:
    """Load libgdn.so (it must have been built by build())."""
    global _lib
    if _lib is not None:
        return _lib
    path = lib_path()
    if not os.path.exists(path):
        raise ImportError(f"libgdn.so not built at {path}: run __graft_entry__.build() first")
    lib = ctypes.CDLL(path)
    P, I, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    PS = ctypes.POINTER(ctypes.c_size_t)
    lib.gdn_state_pool_layout_for.argtypes = [I] * 8 + [S, PS, PS, PS, PS]
    lib.gdn_state_pool_create.argtypes = [ctypes.POINTER(P)] + [I] * 8 + [S, P, S]
    lib.gdn_state_pool_destroy.argtypes = [P]
    lib.gdn_state_pool_layout.argtypes = [P, PS, PS, PS, ctypes.POINTER(P)]
    lib.gdn_state_pool_copy_block.argtypes = [P, I, I, I, P]
    lib.gdn_state_pool_reserve.argtypes = [P, I]
    lib.gdn_varlen_forward.argtypes = [P, I, P, P, P, P, P, P, ctypes.POINTER(Weights), P,
                                       I, I, I, P]
    lib.gdn_kda_varlen_forward.argtypes = lib.gdn_varlen_forward.argtypes
    lib.gdn_ssd_pool_layout_for.argtypes = [I] * 8 + [S, PS, PS, PS, PS]
    lib.gdn_ssd_pool_create.argtypes = [ctypes.POINTER(P)] + [I] * 8 + [S, P, S]
    lib.gdn_ssd_varlen_forward.argtypes = [P, I, P, P, P, P, P, ctypes.POINTER(SsdWeights), P,
                                           I, I, I, P]
    lib.gdn_varlen_forward_noalloc.argtypes = [P, S] + [I] * 8 + [S, I] + [P] * 6 + [
        ctypes.POINTER(Weights), P, I, I, I, P, P]
    lib.gdn_get_error.argtypes = [P, I, ctypes.POINTER(ctypes.c_uint32), I, P]
    lib.gdn_pool_set_timing_events.argtypes = [P, P, P]
    lib.gdn_pool_last_prefill_path.argtypes = [P, ctypes.POINTER(ctypes.c_int)]
    lib.gdn_prefill_scratch_bytes.argtypes = [I] * 6 + [PS]
    lib.gdn_in_proj.argtypes = [P, I, I, P, P, P, P, I, I, I, P, P, P, P, P, P]
    lib.gdn_out_proj.argtypes = [P, P, P, ctypes.c_float, P, I, I, I, I, P, P, P, P]
    L = ctypes.c_int64
    lib.gdn_state_pool_copy_blocks.argtypes = [P, I, P, P, I, P]
    lib.gdn_state_pool_clear_blocks.argtypes = [P, I, P, I, P]
    lib.gdn_state_pool_compact.argtypes = [P, P, P, I, P]
    lib.gdn_lin_pool_layout_for.argtypes = [I] * 5 + [S, PS, PS]
    lib.gdn_lin_pool_create.argtypes = [ctypes.POINTER(P)] + [I] * 5 + [S, P, S]
    lib.gdn_lin_varlen_forward.argtypes = [P, I, P, P, P, L, L, L, I, P, P, P, P,
                                           ctypes.c_float, P, L, I, I, I, P]
    F = ctypes.c_float
    lib.gdn_sel_pool_layout_for.argtypes = [I] * 6 + [S, PS, PS, PS, PS]
    lib.gdn_sel_pool_create.argtypes = [ctypes.POINTER(P)] + [I] * 6 + [S, P, S]
    lib.gdn_sel_conv_varlen_forward.argtypes = [P, I, P, L] + [P] * 6 + [L, I, I, I, P]
    lib.gdn_sel_scan_varlen_forward.argtypes = [P, I] + [P, L] * 5 + [P, P, P] + [
        ctypes.POINTER(SelWeights), P, L, I, I, I, P]
    lib.gdn_win_pool_layout_for.argtypes = [I] * 7 + [S, PS, PS, PS]
    lib.gdn_win_pool_create.argtypes = [ctypes.POINTER(P)] + [I] * 7 + [S, P, S]
    lib.gdn_win_varlen_forward.argtypes = [P, I, P, P, P, L, L, L, I, P, P, P, F, P, L, I, I, I, P]
    lib.gdn_qk_norm_rope.argtypes = [P, P, L, L, P, P, I, I, P, P, F, F] + [I] * 5 + [P, P, L, L, P]
    lib.gdn_diag_umma_gemm.argtypes = [P, P, P, P, I, I, I, P]
    lib.gdn_diag_umma_gemm.restype = I
    lib.gdn_diag_umma_gemm_ex.argtypes = [P, P, P, P, I, I, I, I, I, P]
    lib.gdn_diag_umma_gemm_ex.restype = I
    lib.gdn_diag_wait_timeout.argtypes = [P, P]
    lib.gdn_diag_wait_timeout.restype = I
    lib.gdn_status_string.argtypes = [I]
    lib.gdn_status_string.restype = ctypes.c_char_p
    for name in EXPORTED[:-1]:
        getattr(lib, name).restype = I
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load().gdn_status_string(status).decode()


def _check(status: int, what: str):
    if status != GDN_OK:
        raise GdnError(status, what)


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _index(t, device: Optional[int] = None) -> Optional[int]:
    """The address of a list of block indices, on the pool's device."""
    if t.dtype != torch.int32 or not t.is_cuda or t.dim() != 1 or not t.is_contiguous():
        raise ValueError("block indices are a contiguous int32 CUDA tensor of one dimension")
    if device is not None and t.get_device() != device:
        raise ValueError(f"block indices on {t.device}: the pool is on cuda:{device}")
    return t.data_ptr()


# torch.cuda.current_stream() builds a Stream object, half of a small call's host time
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


# (torch.cuda.current_device() checks that CUDA is initialised first)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _stream(stream, device: Optional[int] = None) -> Optional[int]:
    """A stream's handle; None: the current one, of the current device or the
    one given."""
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device() if device is None else device)
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


_ACT_CODES = {torch.float32: GDN_F32, "f32": GDN_F32, torch.bfloat16: GDN_BF16, "bf16": GDN_BF16}


def act_code(dtype) -> int:
    code = _ACT_CODES.get(dtype)
    if code is None:
        raise ValueError(f"unsupported activation dtype {dtype}")
    return code


def layout_for(num_blocks, num_layers, Hk, Hv, dk, dv, K, act, block_align=0):
    """(block_stride, conv_off, rec_off, total_bytes) without allocating."""
    out = [ctypes.c_size_t() for _ in range(4)]
    _check(load().gdn_state_pool_layout_for(num_blocks, num_layers, Hk, Hv, dk, dv, K,
                                            act_code(act), block_align,
                                            *[ctypes.byref(o) for o in out]),
           "gdn_state_pool_layout_for")
    return tuple(o.value for o in out)


def ssd_layout_for(num_blocks, num_layers, H, P, N, G, K, act, block_align=0):
    """(block_stride, conv_off, ssm_off, total_bytes) of a Mamba2 pool."""
    out = [ctypes.c_size_t() for _ in range(4)]
    _check(load().gdn_ssd_pool_layout_for(num_blocks, num_layers, H, P, N, G, K, act_code(act),
                                          block_align, *[ctypes.byref(o) for o in out]),
           "gdn_ssd_pool_layout_for")
    return tuple(o.value for o in out)


class Pool:
    """A state pool (gdn_state_pool_create).  With ``memory`` (a CUDA uint8
    tensor) the pool lives in that tensor, which then is a byte view of it."""

    def __init__(self, num_blocks, num_layers, Hk, Hv, dk, dv, K, act, block_align=0,
                 memory: Optional[torch.Tensor] = None):
        self.dims = (num_blocks, num_layers, Hk, Hv, dk, dv, K)
        self.act = act_code(act)
        self.num_blocks, self.num_layers = num_blocks, num_layers
        self.memory = memory
        h = ctypes.c_void_p()
        nbytes = memory.numel() * memory.element_size() if memory is not None else 0
        _check(load().gdn_state_pool_create(ctypes.byref(h), num_blocks, num_layers, Hk, Hv, dk,
                                            dv, K, self.act, block_align, _ptr(memory), nbytes),
               "gdn_state_pool_create")
        self.handle, self.device = h, torch.cuda.current_device()
        s, c, r, b = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_void_p()
        _check(load().gdn_state_pool_layout(h, ctypes.byref(s), ctypes.byref(c), ctypes.byref(r),
                                            ctypes.byref(b)), "gdn_state_pool_layout")
        self.stride, self.conv_off, self.rec_off, self.base = s.value, c.value, r.value, b.value

    def close(self):
        if self.handle is not None and self.handle.value:
            load().gdn_state_pool_destroy(self.handle)
        self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def set_timing_events(self, before=None, after=None):
        """Record torch.cuda.Event ``before``/``after`` around the compute
        kernels of every later forward (None, None: off)."""
        hb = before.cuda_event if before is not None else None
        ha = after.cuda_event if after is not None else None
        _check(load().gdn_pool_set_timing_events(self.handle, hb, ha),
               "gdn_pool_set_timing_events")

    def reserve(self, max_tokens: int):
        """gdn_state_pool_reserve: > 0 grow the prefill scratch now, 0 free it
        and use the fused prefill kernel only, < 0 grow on demand."""
        _check(load().gdn_state_pool_reserve(self.handle, max_tokens), "gdn_state_pool_reserve")

    def last_prefill_path(self) -> int:
        """gdn_pool_last_prefill_path: PREFILL_NONE / SPLIT / FUSED / SERIAL."""
        v = ctypes.c_int()
        _check(load().gdn_pool_last_prefill_path(self.handle, ctypes.byref(v)),
               "gdn_pool_last_prefill_path")
        return v.value

    def copy_block(self, layer, src, dst, stream=None):
        _check(load().gdn_state_pool_copy_block(self.handle, layer, src, dst, _stream(stream)),
               "gdn_state_pool_copy_block")

    def copy_blocks(self, src, dst, layer=-1, stream=None):
        """gdn_state_pool_copy_blocks: block dst[i] <- block src[i] for all i
        at once (int32 device tensors), in one layer or (-1) in all."""
        if len(src) != len(dst):
            raise ValueError(f"{len(src)} sources and {len(dst)} destinations")
        dev = self.device
        _check(load().gdn_state_pool_copy_blocks(self.handle, layer, _index(src, dev),
                                                 _index(dst, dev), len(src), _stream(stream)),
               "gdn_state_pool_copy_blocks")

    def clear_blocks(self, idx, layer=-1, stream=None):
        """gdn_state_pool_clear_blocks: blocks idx (int32 device tensor) <- zeros."""
        _check(load().gdn_state_pool_clear_blocks(self.handle, layer, _index(idx, self.device),
                                                  len(idx), _stream(stream)),
               "gdn_state_pool_clear_blocks")

    def compact(self, idx, new_idx=None, stream=None):
        """gdn_state_pool_compact: the live blocks idx (int32 device tensor)
        move to the lowest indices; new_idx (or idx itself) receives where
        each one is afterwards.  Returns new_idx."""
        new_idx = idx if new_idx is None else new_idx
        if len(idx) != len(new_idx):
            raise ValueError(f"{len(idx)} indices and room for {len(new_idx)}")
        dev = self.device
        _check(load().gdn_state_pool_compact(self.handle, _index(idx, dev), _index(new_idx, dev),
                                             len(idx), _stream(stream)), "gdn_state_pool_compact")
        return new_idx

    def error_flags(self, layer=-1, reset=True, stream=None) -> int:
        v = ctypes.c_uint32()
        _check(load().gdn_get_error(self.handle, layer, ctypes.byref(v), 1 if reset else 0,
                                    _stream(stream)), "gdn_get_error")
        return v.value


class SsdPool(Pool):
    """A Mamba2 state pool (gdn_ssd_pool_create); ``rec_off`` is the SSM
    state's offset.  With ``memory`` the pool lives in that CUDA uint8 tensor."""

    def __init__(self, num_blocks, num_layers, H, P, N, G, K, act, block_align=0,
                 memory: Optional[torch.Tensor] = None):
        self.dims = (num_blocks, num_layers, H, P, N, G, K)
        self.act = act_code(act)
        self.num_blocks, self.num_layers = num_blocks, num_layers
        self.memory = memory
        h = ctypes.c_void_p()
        nbytes = memory.numel() * memory.element_size() if memory is not None else 0
        _check(load().gdn_ssd_pool_create(ctypes.byref(h), num_blocks, num_layers, H, P, N, G, K,
                                          self.act, block_align, _ptr(memory), nbytes),
               "gdn_ssd_pool_create")
        self.handle, self.device = h, torch.cuda.current_device()
        s, c, r, b = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_void_p()
        _check(load().gdn_state_pool_layout(h, ctypes.byref(s), ctypes.byref(c), ctypes.byref(r),
                                            ctypes.byref(b)), "gdn_state_pool_layout")
        self.stride, self.conv_off, self.rec_off, self.base = s.value, c.value, r.value, b.value


def ssd_varlen_forward(pool: SsdPool, layer: int, xbc, dt, cu_seqlens, state_block_idx, has_past,
                       conv_w, A_log, dt_bias, D, y, T: int, N: int, max_seqlen_hint: int = 0,
                       stream=None) -> None:
    """gdn_ssd_varlen_forward on device tensors (or raw device pointers)."""
    w = SsdWeights(_ptr(conv_w), _ptr(A_log), _ptr(dt_bias), _ptr(D))
    _check(load().gdn_ssd_varlen_forward(pool.handle, layer, _ptr(xbc), _ptr(dt),
                                         _ptr(cu_seqlens), _ptr(state_block_idx), _ptr(has_past),
                                         ctypes.byref(w), _ptr(y), T, N, max_seqlen_hint,
                                         _stream(stream)), "gdn_ssd_varlen_forward")


def lin_layout_for(num_blocks, num_layers, H, d, act, block_align=0):
    """(block_stride, total_bytes) of a decayed linear attention pool."""
    out = [ctypes.c_size_t() for _ in range(2)]
    _check(load().gdn_lin_pool_layout_for(num_blocks, num_layers, H, d, act_code(act), block_align,
                                          *[ctypes.byref(o) for o in out]),
           "gdn_lin_pool_layout_for")
    return tuple(o.value for o in out)


class LinPool(Pool):
    """A decayed linear attention state pool (gdn_lin_pool_create): blocks of
    [H][d][d] fp32.  With ``memory`` the pool lives in that CUDA uint8 tensor."""

    def __init__(self, num_blocks, num_layers, H, d, act, block_align=0,
                 memory: Optional[torch.Tensor] = None):
        self.dims = (num_blocks, num_layers, H, d)
        self.act = act_code(act)
        self.dtype = torch.float32 if self.act == GDN_F32 else torch.bfloat16
        self.num_blocks, self.num_layers = num_blocks, num_layers
        self.memory = memory
        h = ctypes.c_void_p()
        if memory is not None and not (memory.is_contiguous() and memory.is_cuda and
                                       memory.get_device() == torch.cuda.current_device()):
            raise ValueError("the pool's memory is a contiguous tensor on the current CUDA device")
        nbytes = memory.numel() * memory.element_size() if memory is not None else 0
        _check(load().gdn_lin_pool_create(ctypes.byref(h), num_blocks, num_layers, H, d, self.act,
                                          block_align, _ptr(memory), nbytes),
               "gdn_lin_pool_create")
        self.handle, self.device = h, torch.cuda.current_device()
        s, c, r, b = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_void_p()
        _check(load().gdn_state_pool_layout(h, ctypes.byref(s), ctypes.byref(c), ctypes.byref(r),
                                            ctypes.byref(b)), "gdn_state_pool_layout")
        self.stride, self.conv_off, self.rec_off, self.base = s.value, c.value, r.value, b.value


def _heads(t, name, heads, d, dtype, T, device):
    """(address, row pitch) of at least T rows of heads [T][heads][d]: any row
    pitch, the rows themselves dense."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or shape[1] != heads or shape[2] != d or t.dtype != dtype or shape[0] < T:
        raise ValueError(f"{name} is [>= {T}][{heads}][{d}] of {dtype}: got {tuple(shape)} of "
                         f"{t.dtype}")
    rows = shape[0]
    # (get_device() is -1 for a tensor of the host)
    if rows and (stride[2] != 1 or (heads > 1 and stride[1] != d) or t.get_device() != device):
        raise ValueError(f"the rows of {name} have to be dense, on cuda:{device}")
    return t.data_ptr(), stride[0] if rows > 1 else heads * d


def _list(t, name, dtype, n, device):
    """The address of a dense device list of at least n elements."""
    if (t.dtype != dtype or t.numel() < n or t.get_device() != device or
            not t.is_contiguous()):
        raise ValueError(f"{name} is a contiguous tensor of >= {n} {dtype} on cuda:{device}: got "
                         f"{t.numel()} of {t.dtype} on {t.device}")
    return t.data_ptr()


def lin_varlen_forward(pool: LinPool, layer: int, q, k, v, cu_seqlens, state_block_idx, has_past,
                       log_decay, out, T: int, N: int, scale: float = 1.0,
                       max_seqlen_hint: int = 0, stream=None) -> None:
    """gdn_lin_varlen_forward on device tensors: q and out [T][H][d], k and v
    [T][Hkv][d], each with any row pitch (views of a fused projection's rows)."""
    H, d, dtype, dev = pool.dims[2], pool.dims[3], pool.dtype, pool.device
    if k.dim() != 3:
        raise ValueError(f"k is [>= {T}][heads][{d}]: got {tuple(k.shape)}")
    Hkv = k.shape[1]
    pq, ldq = _heads(q, "q", H, d, dtype, T, dev)
    pk, ldk = _heads(k, "k", Hkv, d, dtype, T, dev)
    pv, ldv = _heads(v, "v", Hkv, d, dtype, T, dev)
    po, ldo = _heads(out, "out", H, d, dtype, T, dev)
    _check(load().gdn_lin_varlen_forward(
        pool.handle, layer, pq, pk, pv, ldq, ldk, ldv, Hkv,
        _list(cu_seqlens, "cu_seqlens", torch.int32, N + 1, dev),
        _list(state_block_idx, "state_block_idx", torch.int32, N, dev),
        _list(has_past, "has_past", torch.uint8, N, dev),
        _list(log_decay, "log_decay", torch.float32, H, dev),
        scale, po, ldo, T, N, max_seqlen_hint, _stream(stream, dev)),
        "gdn_lin_varlen_forward")


def sel_layout_for(num_blocks, num_layers, channels, N, K, act, block_align=0):
    """(block_stride, conv_off, ssm_off, total_bytes) of a selective scan pool."""
    out = [ctypes.c_size_t() for _ in range(4)]
    _check(load().gdn_sel_pool_layout_for(num_blocks, num_layers, channels, N, K, act_code(act),
                                          block_align, *[ctypes.byref(o) for o in out]),
           "gdn_sel_pool_layout_for")
    return tuple(o.value for o in out)


def win_layout_for(num_blocks, num_layers, Hkv, d, window, sinks, act, block_align=0):
    """(block_stride, v_off, total_bytes) of a windowed attention pool."""
    out = [ctypes.c_size_t() for _ in range(3)]
    _check(load().gdn_win_pool_layout_for(num_blocks, num_layers, Hkv, d, window, sinks,
                                          act_code(act), block_align,
                                          *[ctypes.byref(o) for o in out]),
           "gdn_win_pool_layout_for")
    return tuple(o.value for o in out)


class _TypedPool(Pool):
    """What the pools of the selective scan and of windowed attention share."""

    def _create(self, create, dims, act, block_align, memory):
        self.dims = tuple(dims)
        self.act = act_code(act)
        self.dtype = torch.float32 if self.act == GDN_F32 else torch.bfloat16
        self.num_blocks, self.num_layers = dims[0], dims[1]
        self.memory = memory
        h = ctypes.c_void_p()
        if memory is not None and not (memory.is_contiguous() and memory.is_cuda and
                                       memory.get_device() == torch.cuda.current_device()):
            raise ValueError("the pool's memory is a contiguous tensor on the current CUDA device")
        nbytes = memory.numel() * memory.element_size() if memory is not None else 0
        _check(getattr(load(), create)(ctypes.byref(h), *dims, self.act, block_align, _ptr(memory),
                                       nbytes), create)
        self.handle, self.device = h, torch.cuda.current_device()
        s, c, r, b = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_void_p()
        _check(load().gdn_state_pool_layout(h, ctypes.byref(s), ctypes.byref(c), ctypes.byref(r),
                                            ctypes.byref(b)), "gdn_state_pool_layout")
        self.stride, self.conv_off, self.rec_off, self.base = s.value, c.value, r.value, b.value


class SelPool(_TypedPool):
    """A selective scan pool (gdn_sel_pool_create): blocks of a conv state
    [K-1][channels] and, at ``rec_off``, a state [channels][N] fp32.  With
    ``memory`` the pool lives in that CUDA uint8 tensor."""

    handle = None

    def __init__(self, num_blocks, num_layers, channels, N, K, act, block_align=0,
                 memory: Optional[torch.Tensor] = None):
        self._create("gdn_sel_pool_create", (num_blocks, num_layers, channels, N, K), act,
                     block_align, memory)


class WinPool(_TypedPool):
    """A windowed attention pool (gdn_win_pool_create): blocks of the keys
    and, at ``rec_off``, the values [Hkv][sinks + window][d].  With ``memory``
    the pool lives in that CUDA uint8 tensor."""

    handle = None

    def __init__(self, num_blocks, num_layers, Hkv, d, window, sinks, act, block_align=0,
                 memory: Optional[torch.Tensor] = None):
        self._create("gdn_win_pool_create", (num_blocks, num_layers, Hkv, d, window, sinks), act,
                     block_align, memory)


def _rows(t, name, cols, dtype, T, device):
    """(address, row pitch) of at least T dense rows [T][cols], any row pitch."""
    shape = t.shape
    if len(shape) != 2 or shape[1] != cols or t.dtype != dtype or shape[0] < T:
        raise ValueError(f"{name} is [>= {T}][{cols}] of {dtype}: got {tuple(shape)} of {t.dtype}")
    rows, stride = shape[0], t.stride()
    if rows and (stride[1] != 1 or t.get_device() != device):
        raise ValueError(f"the rows of {name} have to be dense, on cuda:{device}")
    return t.data_ptr(), stride[0] if rows > 1 else cols


def _maybe(t, name, dtype, n, device):
    return None if t is None else _list(t, name, dtype, n, device)


def sel_conv_varlen_forward(pool: SelPool, layer: int, x, cu_seqlens, state_block_idx, has_past,
                            conv_w, conv_b, out, T: int, N: int, max_seqlen_hint: int = 0,
                            stream=None) -> None:
    """gdn_sel_conv_varlen_forward on device tensors: x and out [T][channels],
    each with any row pitch; conv_w [channels][K], conv_b [channels] or None."""
    C, K, dtype, dev = pool.dims[2], pool.dims[4], pool.dtype, pool.device
    px, ldx = _rows(x, "x", C, dtype, T, dev)
    po, ldo = _rows(out, "out", C, dtype, T, dev)
    _check((_lib or load()).gdn_sel_conv_varlen_forward(
        pool.handle, layer, px, ldx,
        _list(cu_seqlens, "cu_seqlens", torch.int32, N + 1, dev),
        _list(state_block_idx, "state_block_idx", torch.int32, N, dev),
        _list(has_past, "has_past", torch.uint8, N, dev),
        _list(conv_w, "conv_w", dtype, C * K, dev), _maybe(conv_b, "conv_b", dtype, C, dev),
        po, ldo, T, N, max_seqlen_hint, _stream(stream, dev)), "gdn_sel_conv_varlen_forward")


def sel_scan_varlen_forward(pool: SelPool, layer: int, u, dt, B, C, z, cu_seqlens, state_block_idx,
                            has_past, A_log, D, dt_bias, y, T: int, N: int,
                            max_seqlen_hint: int = 0, stream=None) -> None:
    """gdn_sel_scan_varlen_forward on device tensors: u, dt, z (or None) and y
    [T][channels], B and C [T][d_state], each with any row pitch; A_log
    [channels][d_state], D and dt_bias [channels] or None, fp32."""
    chan, n, dtype, dev = pool.dims[2], pool.dims[3], pool.dtype, pool.device
    rows = []
    for t, name, cols in ((u, "u", chan), (dt, "dt", chan), (B, "B", n), (C, "C", n), (z, "z", chan)):
        rows += (None, 0) if t is None and name == "z" else _rows(t, name, cols, dtype, T, dev)
    py, ldy = _rows(y, "y", chan, dtype, T, dev)
    w = SelWeights(_list(A_log, "A_log", torch.float32, chan * n, dev),
                   _maybe(D, "D", torch.float32, chan, dev),
                   _maybe(dt_bias, "dt_bias", torch.float32, chan, dev))
    _check((_lib or load()).gdn_sel_scan_varlen_forward(
        pool.handle, layer, *rows,
        _list(cu_seqlens, "cu_seqlens", torch.int32, N + 1, dev),
        _list(state_block_idx, "state_block_idx", torch.int32, N, dev),
        _list(has_past, "has_past", torch.uint8, N, dev), ctypes.byref(w), py, ldy, T, N,
        max_seqlen_hint, _stream(stream, dev)), "gdn_sel_scan_varlen_forward")


def win_varlen_forward(pool: WinPool, layer: int, q, k, v, cu_seqlens, state_block_idx, past_lens,
                       out, T: int, N: int, scale: float = 1.0, max_seqlen_hint: int = 0,
                       stream=None) -> None:
    """gdn_win_varlen_forward on device tensors: q and out [T][H][d], k and v
    [T][Hkv][d], each with any row pitch (views of a fused projection's rows);
    past_lens [N] int32, the requests' tokens before this call."""
    Hkv, d, dtype, dev = pool.dims[2], pool.dims[3], pool.dtype, pool.device
    if q.dim() != 3:
        raise ValueError(f"q is [>= {T}][heads][{d}]: got {tuple(q.shape)}")
    H = q.shape[1]
    pq, ldq = _heads(q, "q", H, d, dtype, T, dev)
    pk, ldk = _heads(k, "k", Hkv, d, dtype, T, dev)
    pv, ldv = _heads(v, "v", Hkv, d, dtype, T, dev)
    po, ldo = _heads(out, "out", H, d, dtype, T, dev)
    _check((_lib or load()).gdn_win_varlen_forward(
        pool.handle, layer, pq, pk, pv, ldq, ldk, ldv, H,
        _list(cu_seqlens, "cu_seqlens", torch.int32, N + 1, dev),
        _list(state_block_idx, "state_block_idx", torch.int32, N, dev),
        _list(past_lens, "past_lens", torch.int32, N, dev),
        scale, po, ldo, T, N, max_seqlen_hint, _stream(stream, dev)),
        "gdn_win_varlen_forward")


def qk_norm_rope(q, k, positions, inv_freq, q_weight=None, k_weight=None, q_out=None, k_out=None,
                 eps: float = 1e-6, weight_offset: float = 0.0, interleaved: bool = False,
                 stream=None):
    """gdn_qk_norm_rope on device tensors: q [T][H][d] and k [T][Hkv][d] (k may
    be None), each with any row pitch; positions [T] int32; inv_freq [rot/2]
    fp32 (None: no rotation).  Without q_out and k_out in place.  Returns
    (q_out, k_out)."""
    shape = q.shape
    if len(shape) != 3 or (k is not None and k.dim() != 3):
        raise ValueError("q and k are [T][heads][d]")
    T, H, d = shape
    dtype, dev = q.dtype, q.get_device()
    if dev < 0 or dev != _current_device():
        raise ValueError(f"q is on {q.device}, not on the current CUDA device")
    pq, ldq = _heads(q, "q", H, d, dtype, T, dev)
    if q_out is None or q_out is q:
        q_out, pqo, ldqo = q, pq, ldq
    else:
        pqo, ldqo = _heads(q_out, "q_out", H, d, dtype, T, dev)
    if k is None:
        if k_out is not None:
            raise ValueError("k_out without k")
        Hkv, pk, ldk, pko, ldko = 0, None, 0, None, 0
    else:
        rows, Hkv, _ = k.shape
        if rows != T:
            raise ValueError(f"{T} rows of q and {rows} of k")
        pk, ldk = _heads(k, "k", Hkv, d, dtype, T, dev)
        if k_out is None or k_out is k:
            k_out, pko, ldko = k, pk, ldk
        else:
            pko, ldko = _heads(k_out, "k_out", Hkv, d, dtype, T, dev)
    half = 0 if inv_freq is None else inv_freq.numel()
    f32 = torch.float32
    _check((_lib or load()).gdn_qk_norm_rope(
        pq, pk, ldq, ldk, _list(positions, "positions", torch.int32, T, dev),
        _maybe(inv_freq, "inv_freq", f32, half, dev), 2 * half, 1 if interleaved else 0,
        _maybe(q_weight, "q_weight", f32, d, dev), _maybe(k_weight, "k_weight", f32, d, dev),
        weight_offset, eps, T, H, Hkv, d, act_code(dtype), pqo, pko, ldqo, ldko,
        _stream(stream, dev)), "gdn_qk_norm_rope")
    return q_out, k_out


def varlen_forward(pool: Pool, layer: int, x_qkv, a, b, cu_seqlens, state_block_idx, has_past,
                   conv_w, A_log, dt_bias, out, T: int, N: int, max_seqlen_hint: int = 0,
                   stream=None) -> None:
    """gdn_varlen_forward on device tensors (or raw device pointers)."""
    w = Weights(_ptr(conv_w), _ptr(A_log), _ptr(dt_bias))
    _check(load().gdn_varlen_forward(pool.handle, layer, _ptr(x_qkv), _ptr(a), _ptr(b),
                                     _ptr(cu_seqlens), _ptr(state_block_idx), _ptr(has_past),
                                     ctypes.byref(w), _ptr(out), T, N, max_seqlen_hint,
                                     _stream(stream)), "gdn_varlen_forward")


def kda_varlen_forward(pool: Pool, layer: int, x_qkv, a, b, cu_seqlens, state_block_idx,
                       has_past, conv_w, A_log, dt_bias, out, T: int, N: int,
                       max_seqlen_hint: int = 0, stream=None) -> None:
    """gdn_kda_varlen_forward: the per-channel-decay rule (a [T][Hv][d_k],
    dt_bias [Hv][d_k]) on device tensors (or raw device pointers)."""
    w = Weights(_ptr(conv_w), _ptr(A_log), _ptr(dt_bias))
    _check(load().gdn_kda_varlen_forward(pool.handle, layer, _ptr(x_qkv), _ptr(a), _ptr(b),
                                         _ptr(cu_seqlens), _ptr(state_block_idx), _ptr(has_past),
                                         ctypes.byref(w), _ptr(out), T, N, max_seqlen_hint,
                                         _stream(stream)), "gdn_kda_varlen_forward")


def diag_umma_gemm(A, B, C, D, operand_f16=False, stream=None) -> None:
    """gdn_diag_umma_gemm: D = (C or 0) + A @ B^T on the tensor cores
    (A [128][K], B [N][K] bf16; C, D [128][N] fp32; device tensors)."""
    N, K = B.shape
    _check(load().gdn_diag_umma_gemm(_ptr(A), _ptr(B), _ptr(C), _ptr(D), N, K,
                                     1 if operand_f16 else 0, _stream(stream)),
           "gdn_diag_umma_gemm")


def diag_umma_gemm_ex(A, B, C, D, operand_f16=False, a_mn=False, b_mn=False,
                      stream=None) -> None:
    """gdn_diag_umma_gemm_ex: the same GEMM with A and/or B staged MN-major
    (a_mn=2: A in tensor memory instead)."""
    N, K = B.shape
    _check(load().gdn_diag_umma_gemm_ex(_ptr(A), _ptr(B), _ptr(C), _ptr(D), N, K,
                                        1 if operand_f16 else 0, int(a_mn),
                                        1 if b_mn else 0, _stream(stream)),
           "gdn_diag_umma_gemm_ex")


def diag_wait_timeout(flags, stream=None) -> None:
    """gdn_diag_wait_timeout: a bounded wait that runs out and ORs
    GDN_FLAG_TIMEOUT into ``flags`` (a 1-element int32/uint32 CUDA tensor)."""
    _check(load().gdn_diag_wait_timeout(_ptr(flags), _stream(stream)), "gdn_diag_wait_timeout")


def in_proj(hidden, w_qkv, w_z, w_b, w_a, x_qkv, z, b, a, C, Hv, dv, flags=None,
            stream=None) -> None:
    """gdn_in_proj: x_qkv | z | b | a = hidden W^T (device tensors)."""
    T, d_model = hidden.shape
    _check(load().gdn_in_proj(_ptr(hidden), T, d_model, _ptr(w_qkv), _ptr(w_z), _ptr(w_b),
                              _ptr(w_a), C, Hv, dv, _ptr(x_qkv), _ptr(z), _ptr(b), _ptr(a),
                              _ptr(flags), _stream(stream)), "gdn_in_proj")


def out_proj(o, z, norm_w, eps, w_out, o_norm, y, flags=None, stream=None) -> None:
    """gdn_out_proj: o_norm = gated RMS norm of o, y = o_norm W_out^T."""
    T, Hv, dv = o.shape
    d_model = w_out.shape[0]
    _check(load().gdn_out_proj(_ptr(o), _ptr(z), _ptr(norm_w), float(eps), _ptr(w_out), T, Hv,
                               dv, d_model, _ptr(o_norm), _ptr(y), _ptr(flags), _stream(stream)),
           "gdn_out_proj")


def prefill_scratch_bytes(num_blocks, Hk, Hv, dk, dv, max_tokens) -> int:
    """gdn_prefill_scratch_bytes: bytes of prefill scratch the split prefill
    needs for calls of at most max_tokens tokens."""
    out = ctypes.c_size_t(0)
    _check(load().gdn_prefill_scratch_bytes(num_blocks, Hk, Hv, dk, dv, max_tokens,
                                            ctypes.byref(out)), "gdn_prefill_scratch_bytes")
    return int(out.value)


def varlen_forward_noalloc(pool_mem, num_blocks, num_layers, Hk, Hv, dk, dv, K, act, block_align,
                           layer, x_qkv, a, b, cu_seqlens, state_block_idx, has_past, conv_w,
                           A_log, dt_bias, out, T, N, max_seqlen_hint=0, flags_out=None,
                           stream=None) -> None:
    """gdn_varlen_forward_noalloc: the forward on caller-owned pool memory
    (a CUDA uint8 tensor or a raw device pointer), allocating nothing."""
    nbytes = pool_mem.numel() * pool_mem.element_size() if hasattr(pool_mem, "numel") else 0
    w = Weights(_ptr(conv_w), _ptr(A_log), _ptr(dt_bias))
    _check(load().gdn_varlen_forward_noalloc(
        _ptr(pool_mem), nbytes, num_blocks, num_layers, Hk, Hv, dk, dv, K, act_code(act),
        block_align, layer, _ptr(x_qkv), _ptr(a), _ptr(b), _ptr(cu_seqlens),
        _ptr(state_block_idx), _ptr(has_past), ctypes.byref(w), _ptr(out), T, N,
        max_seqlen_hint, _ptr(flags_out), _stream(stream)), "gdn_varlen_forward_noalloc")
