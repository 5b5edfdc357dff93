"""Calls on one pool right behind each other on the GPU, with nothing between
them that waits (all lists are on the device beforehand), give the bits of the
same calls with the host waiting after each: a call's kernels start beside the
last one's, and share its work area, marks and segment states."""
import numpy as np
import pytest
import torch

from continuous_linear_attention_gb300 import binding, harness, synth

pytestmark = pytest.mark.gpu

I32 = dict(dtype=torch.int32, device="cuda")


def twice(play):
    """play(wait) -> tensors; with and without waiting, the same bits."""
    want = play(torch.cuda.synchronize)
    got = play(lambda: None)
    torch.cuda.synchronize()
    for i, (a, b) in enumerate(zip(got, want)):
        assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8)), i


def batches(H, Hkv, d, act, blocks, seed):
    """Forwards of every form, some with sequences that are computed again for
    a value that is not finite, some left out."""
    lists = [
        [200, 1, 90, 300], [1] * 12, [1500, 3], [7, 1, 16, 2], [70, 2000], [128, 129, 40, 1, 1],
        [1] * 300, [1100, 1, 5, 0, 260], [65] * 6,
    ]
    rng = np.random.default_rng(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    dtype = torch.float32 if act == "f32" else torch.bfloat16
    out = []
    for i, lens in enumerate(lists):
        T = sum(lens)
        x = torch.randn(T, (H + 2 * Hkv) * d, device="cuda", generator=g).to(dtype)
        if i in (0, 2, 5):
            x[T // 3, -5] = float("nan")
        b = rng.permutation(blocks - 1)[:len(lens)] + 1
        if i in (1, 5, 7):
            b[1] = b[0] if i == 5 else -1
        out.append(dict(
            T=T, N=len(lens), hint=max(lens) if i % 2 else 0,
            qkv=[t.unflatten(1, (-1, d)) for t in x.split([H * d, Hkv * d, Hkv * d], 1)],
            cu=torch.tensor(np.cumsum([0] + lens), **I32), blk=torch.tensor(b, **I32),
            past=torch.tensor(rng.integers(0, 2, len(lens)), dtype=torch.uint8, device="cuda")))
    return out


@pytest.mark.parametrize("act,d,H,Hkv", [("bf16", 128, 4, 2), ("f32", 64, 3, 3), ("bf16", 32, 8, 1)])
def test_forwards(act, d, H, Hkv):
    nb, rounds, layers = 320, 4, 2
    calls = batches(H, Hkv, d, act, nb, seed=d)
    decay = torch.tensor([-0.01, -0.3, 0.0, -2.0] * 2, device="cuda")[:H].contiguous()
    start = torch.randn(layers, nb, H, d, d, device="cuda")
    start[:, 0] = 0
    dtype = calls[0]["qkv"][0].dtype

    def play(wait):
        mem = start.clone()
        pool = binding.LinPool(nb, layers, H, d, act, memory=mem.view(-1).view(torch.uint8))
        mem.copy_(start)
        outs = [[torch.zeros(c["T"], H, d, dtype=dtype, device="cuda") for c in calls] for _ in range(rounds)]
        torch.cuda.synchronize()
        for r in range(rounds):
            for i, c in enumerate(calls):
                binding.lin_varlen_forward(pool, (r + i) % layers, *c["qkv"], c["cu"], c["blk"], c["past"], decay,
                                           outs[r][i], c["T"], c["N"], scale=0.1, max_seqlen_hint=c["hint"])
                wait()
        torch.cuda.synchronize()
        assert pool.error_flags() == 0x8  # one batch names a block twice
        return [mem] + [o for r in outs for o in r]

    twice(play)


@pytest.mark.parametrize("make,nb", [
    (lambda nb, mem: binding.LinPool(nb, 5, 1, 32, "f32", memory=mem), 64),
    (lambda nb, mem: binding.LinPool(nb, 1, 1, 32, "f32", memory=mem), 9000),   # plans in device memory
    (lambda nb, mem: binding.Pool(nb, 2, 16, 32, 128, 128, 4, "bf16", memory=mem), 40),
])
def test_block_operations(make, nb):
    probe = make(2, None)
    words, layers = probe.stride // 4, probe.num_layers
    probe.close()
    start = torch.randint(-2 ** 31, 2 ** 31, (layers, nb, words), device="cuda").int()
    start[:, 0] = 0
    rng = np.random.default_rng(nb)
    ops = []
    for i in range(40):
        n = int(rng.integers(1, nb - 1))
        dst = torch.tensor(rng.permutation(np.arange(1, nb))[:n], **I32)
        if i % 4 == 2:
            ops.append(("compact", dst))
        elif i % 4 == 3:
            ops.append(("clear", dst[:n // 2 + 1]))
        else:
            src = rng.permutation(dst.cpu().numpy()) if i % 8 == 1 else rng.integers(0, nb, n)
            ops.append(("copy", torch.tensor(src, **I32), dst))

    def play(wait):
        mem = torch.empty_like(start)
        pool = make(nb, mem.view(-1).view(torch.uint8))
        mem.copy_(start)
        mine = [(o[0], *(t.clone() for t in o[1:])) for o in ops]
        torch.cuda.synchronize()
        for o in mine:
            if o[0] == "compact":
                pool.compact(o[1])
            elif o[0] == "clear":
                pool.clear_blocks(o[1])
            else:
                pool.copy_blocks(o[1], o[2])
            wait()
        torch.cuda.synchronize()
        assert pool.error_flags() == 0
        return [mem] + [o[1] for o in mine]

    twice(play)


def workloads():
    full = synth.Dims(Hk=16, Hv=32, dk=128, dv=128, K=4, act="bf16")
    small = synth.Dims(Hk=2, Hv=4, dk=32, dv=32, K=4, act="f32")
    ssd = synth.SsdDims(H=16, P=64, N=128, G=2, K=4, act="bf16")
    yield "gdn", lambda: harness.DeviceRun(synth.make_workload("order", full, [1] * 24, [1] * 24, 64, 1))
    yield "gdn_prompts", lambda: harness.DeviceRun(
        synth.make_workload("order", full, [1] * 5 + [70, 130], [1] * 7, 40, 2))
    yield "gdn_small", lambda: harness.DeviceRun(synth.make_workload("order", small, [1, 5, 1, 9], [1] * 4, 500, 3))
    yield "kda", lambda: harness.DeviceRun(
        synth.make_workload("order", full, [1] * 24, [1] * 24, 64, 4, channel_gate=True))
    yield "ssd", lambda: harness.SsdDeviceRun(synth.make_ssd_workload("order", ssd, [1] * 24, [1] * 24, 64, 5))


@pytest.mark.parametrize("name,make", list(workloads()), ids=[n for n, _ in workloads()])
def test_a_forward_reads_the_table_that_a_compaction_rewrites(name, make):
    """The schedulers of these forwards read their lists before they wait for
    the kernel before them: the moving kernel, which lets them start only when
    the plan, and so the table, is there."""
    rounds = 6
    probe = make()
    n, nb = probe.wl.N, probe.wl.num_blocks
    rng = np.random.default_rng(7)
    scattered = [rng.permutation(np.arange(n + 1, nb))[:n] for _ in range(rounds)]

    def play(wait):
        run = make()
        first = torch.arange(1, n + 1, **I32)
        # (from the workload's blocks to 1 .. n, then scattered before each compaction)
        run.pool.copy_blocks(run.idx, first)
        tables = [torch.tensor(t, **I32) for t in scattered]
        wants = [t.clone() for t in tables]
        torch.cuda.synchronize()
        where, outs = first, []
        for table, want in zip(tables, wants):
            run.pool.copy_blocks(where, want)
            wait()
            run.pool.compact(table)
            wait()
            run.idx = table
            run.run()
            wait()
            where = table
        torch.cuda.synchronize()
        assert run.pool.error_flags() == 0
        out = run.out if hasattr(run, "out") else run.y
        # what blocks behind the live ones hold is nobody's
        mem = run.mem.view(-1, run.stride)[:n + 1]
        return [mem, out, *tables]

    twice(play)
