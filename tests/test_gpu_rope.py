"""GPU parity of gdn_qk_norm_rope with its fp64 definition."""
import numpy as np
import pytest
import torch

from continuous_linear_attention_gb300 import binding
from hybrid_check import EPS, SENTINEL, ULP, bits, close, dtype_of, f64
from oracle import hybrid as ref

pytestmark = pytest.mark.gpu


def rope_check(T, H, Hkv, d, rot, act="bf16", norm=True, offset=0.0, inter=False, seed=0, positions=None,
               in_place=False, eps=1e-6, values=None, base=10000.0):
    g = torch.Generator().manual_seed(seed)
    dt = dtype_of(act)
    x = torch.randn(T, H + 2 * Hkv, d, generator=g) * 2
    if values is not None:
        values(x)
    x = x.to(dt)
    dev = x.cuda()
    q, k = dev[:, :H], dev[:, H:H + Hkv]
    pos = torch.randint(0, 100_000, (T,), generator=g) if positions is None else torch.tensor(positions)
    pos = pos.to(torch.int32)
    f = torch.tensor(base ** (-np.arange(0, rot, 2) / max(rot, 1)), dtype=torch.float32) if rot else None
    wq, wk = ((1 - offset + 0.2 * torch.randn(d, generator=g)) if norm else None for _ in range(2))
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    if in_place:
        qo, ko = q, k
    else:
        qo = torch.full((T, H + 1, d), SENTINEL, dtype=dt, device="cuda")[:, :H]
        ko = torch.full((T, Hkv, d), SENTINEL, dtype=dt, device="cuda")
    binding.qk_norm_rope(q, k if Hkv else None, pos.cuda(), cu(f), cu(wq), cu(wk), None if in_place else qo,
                         None if in_place or not Hkv else ko, eps=eps, weight_offset=offset, interleaved=inter)
    torch.cuda.synchronize()
    live = (pos >= 0).numpy()
    for got, src, w in ((qo, x[:, :H], wq), (ko, x[:, H:H + Hkv], wk)):
        if src.shape[1] == 0:
            continue
        with np.errstate(all="ignore"):
            want, mag = ref.norm_rope(f64(src), pos.numpy(), None if f is None else f.numpy(),
                                      None if w is None else f64(w), offset, eps, inter)
        # the norm: 21 roundings in the sum (half of them after the root), the root to 2^-22,
        # three products; sine and cosine to 2^-22, the angle to 2 pi (2^-25 + 2^-54 position)
        turn = 2 * np.pi * (2.0 ** -25 + np.abs(pos.numpy().astype(float)) * 2.0 ** -54)[:, None, None]
        tol = (24 * EPS * (w is not None) + 8 * EPS + turn) * mag + ULP[act] * np.abs(want) + 2.0 ** -126
        close(f64(got)[live], want[live], tol[live], "rows")
        if not live.all():
            was = src if in_place else torch.full_like(src, SENTINEL)
            assert torch.equal(bits(got.cpu()[~live]), bits(was[~live]))
    if in_place:  # what lies beside the heads (the values) is as it was
        assert torch.equal(bits(dev[:, H + Hkv:].cpu()), bits(x[:, H + Hkv:]))
    else:
        assert (torch.as_strided(qo, (T, d), (qo.stride(0), 1), H * d) == SENTINEL).all()


@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("part", [1, 2, 4])
def test_sizes_types_and_orders(d, act, inter, part):
    rope_check(7, 6, 2, d, d // part, act, inter=inter, offset=1.0 if part == 2 else 0.0)


@pytest.mark.parametrize("rot", [0, 2, 6, 20, 30, 62, 64])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_rotated_part(rot, inter, norm):
    rope_check(5, 3, 1, 64, rot, "f32", inter=inter, norm=norm)


@pytest.mark.parametrize("T", [1, 2, 33, 1500])
@pytest.mark.parametrize("H,Hkv", [(1, 1), (32, 8), (5, 0), (40, 1)])
def test_tokens_and_heads(T, H, Hkv):
    rope_check(T, H, Hkv, 128, 128, seed=T)


def test_keys_alone_through_the_c_entry():
    x = torch.randn(5, 3, 64, device="cuda")
    out, pos = torch.zeros_like(x), torch.arange(5, dtype=torch.int32, device="cuda")
    f = torch.tensor([1.0, 0.1], device="cuda")
    st = binding.load().gdn_qk_norm_rope(None, x.data_ptr(), 0, 192, pos.data_ptr(), f.data_ptr(), 4, 0, None, None,
                                         0.0, 1e-6, 5, 0, 3, 64, 0, None, out.data_ptr(), 0, 192, None)
    torch.cuda.synchronize()
    assert st == 0
    want, mag = ref.norm_rope(f64(x), np.arange(5), f.cpu().numpy())
    close(f64(out), want, 16 * EPS * mag, "keys")


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rot", [64, 20])
def test_in_place(act, inter, rot):
    rope_check(300, 4, 2, 64, rot, act, inter=inter, in_place=True)


def test_far_positions():
    rope_check(8, 2, 1, 128, 128, "f32", norm=False,
               positions=[0, 1, 4095, 1_000_000, 16_777_217, 123_456_789, 2 ** 31 - 2, 2 ** 31 - 1])
    rope_check(4, 2, 1, 64, 64, "f32", norm=False, base=0.001, positions=[0, 3, 1000, 77_777])  # frequencies above 1


@pytest.mark.parametrize("in_place", [False, True])
def test_negative_positions_are_left_out(in_place):
    rope_check(70, 3, 1, 64, 64, positions=[-1 if i % 3 == 0 else i for i in range(70)], in_place=in_place)
    rope_check(4, 3, 1, 32, 6, positions=[-1, 5, -2 ** 31, 7], in_place=in_place)


def test_zero_rows_and_values_that_are_not_finite():
    def put(x):
        x[0] = 0.0
        x[1, 0, 3] = float("nan")
        x[2, 1, 5] = float("inf")
        x[3, 0] = 1e-20

    rope_check(5, 3, 1, 64, 64, "f32", norm=True, eps=1e-6, values=lambda x: (x[0].zero_(), x[3].mul_(1e-20)))
    g = torch.Generator().manual_seed(0)
    x = torch.randn(5, 3, 64, generator=g)
    y = x.clone()
    put(y)
    pos, f = torch.arange(5, dtype=torch.int32, device="cuda"), torch.full((32,), 0.1, device="cuda")
    w = torch.ones(64, device="cuda")
    a, _ = binding.qk_norm_rope(x.cuda(), None, pos, f, w)
    b, _ = binding.qk_norm_rope(y.cuda(), None, pos, f, w)
    same = torch.ones(5, 3, dtype=torch.bool)
    same[0] = same[1, 0] = same[2, 1] = same[3, 0] = False
    assert torch.equal(bits(a.cpu()[same]), bits(b.cpu()[same]))  # other heads and tokens
    assert torch.isnan(b[1, 0]).all() and torch.isnan(b[2, 1]).any()


def test_no_rows():
    q = torch.zeros(0, 4, 64, device="cuda")
    binding.qk_norm_rope(q, None, torch.zeros(0, dtype=torch.int32, device="cuda"), None)


def test_captured_on_another_stream():
    x = torch.randn(9, 4, 128, device="cuda").bfloat16()
    pos, f = torch.arange(9, dtype=torch.int32, device="cuda"), torch.rand(64, device="cuda")
    want, _ = binding.qk_norm_rope(x, None, pos, f, q_out=torch.empty_like(x))
    out = torch.zeros_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.qk_norm_rope(x, None, pos, f, q_out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_binding_refusals():
    q, k = torch.zeros(3, 4, 64, device="cuda"), torch.zeros(3, 2, 64, device="cuda")
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    f = torch.zeros(32, device="cuda")
    for bad in (lambda: binding.qk_norm_rope(q, k[:2], pos, f), lambda: binding.qk_norm_rope(q, k, pos[:2], f),
                lambda: binding.qk_norm_rope(q, k, pos.long(), f), lambda: binding.qk_norm_rope(q, k.bfloat16(), pos, f),
                lambda: binding.qk_norm_rope(q.transpose(0, 1), None, pos, f),
                lambda: binding.qk_norm_rope(q, None, pos, f, k_out=k),
                lambda: binding.qk_norm_rope(q, k, pos, f, q_weight=torch.ones(32, device="cuda")),
                lambda: binding.qk_norm_rope(q.half(), k.half(), pos, f)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(binding.GdnError):
        binding.qk_norm_rope(q, k, pos, torch.zeros(33, device="cuda"))


@pytest.mark.parametrize("act,d,rot", [("bf16", 128, 128), ("f32", 32, 6), ("f32", 256, 20), ("bf16", 64, 32)])
@pytest.mark.parametrize("in_place", [False, True])
def test_a_warps_share_goes_over_many_tokens(act, d, rot, in_place):
    """Few heads of many tokens, some without a position between the others."""
    for H, Hkv, T in ((1, 0, 50_011), (2, 1, 20_003)):
        pos = [-1 if i % 7 == 3 or 900 < i < 950 else 3 * i for i in range(T)]
        rope_check(T, H, Hkv, d, rot, act, positions=pos, in_place=in_place, seed=H)
