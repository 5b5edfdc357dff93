"""The operators of decayed linear attention on the state pool, as measured.

Two operators, each in a plain form (elementary torch operations, fp32) and,
with ``own`` true, through the calls a user makes of the library:

``lin``   linear attention with one decay per head over a packed batch,
          continued from each request's fp32 state in a paged pool:
            S_t = e^{g_h} S_{t-1} + k_t v_t^T,   o_t = scale * q_t S_t
          chunked for prompts, recurrent for single tokens.
``pool``  the pool's block operations over all layers: fork or reorder (copy
          lists with every source read before any block is overwritten),
          compaction (the live blocks move to the lowest indices) and free
          (blocks are zeroed).

Lengths are texts such as "1*64,300,512": 64 single tokens, then two prompts.
"""
import math
import random

import torch

own = False

CHUNK = 64  # tokens per chunk of the plain form

# Which parent each of four beams of a request continues from, by request.
BEAMS = ((1, 0, 2, 2), (0, 0, 1, 3), (2, 3, 0, 1), (3, 3, 3, 3), (0, 1, 2, 2), (1, 2, 3, 0),
         (0, 1, 1, 0))


def lengths(text):
    out = []
    for part in text.split(","):
        n, _, times = part.partition("*")
        out += [int(n)] * int(times or 1)
    return out


def _spread(rng, lo, hi):
    """An integer of [lo, hi], uniform in its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _lin(name, lens, heads, kv_heads, d, act, past):
    c = {"op": "lin", "lens": lens, "heads": heads, "kv_heads": kv_heads, "d": d, "act": act,
         "past": past}
    return {"name": name, **c} if name else c


def _pool(name, what, n, layers, hk, hv, d, act, blocks, fan):
    c = {"op": "pool", "what": what, "n": n, "layers": layers, "hk": hk, "hv": hv, "d": d,
         "act": act, "blocks": blocks, "fan": fan}
    return {"name": name, **c} if name else c


def listed():
    return [
        # one request generating alone: the latency of a token
        _lin("decode_1", "1", 16, 16, 128, "bf16", 1),
        # a full generation batch: every state streams in and out
        _lin("decode_256", "1*256", 32, 32, 128, "bf16", 1),
        # drafted tokens checked four at a time, keys and values shared by four heads
        _lin("verify_4x64", "4*64", 32, 8, 128, "bf16", 1),
        # a prompt batch of ragged lengths, no past
        _lin("prefill_16k", "1077,3211,1519,793,2618,3999,547,2079", 64, 64, 128, "bf16", 0),
        # one long prompt of few heads: not enough chains to fill the GPU by themselves
        _lin("long_32k", "32768", 16, 16, 128, "bf16", 0),
        # continuous batching: generation with prompts and continued prompts among it
        _lin("mixed_8k", "1*64,511,2048,1283,700,1790,1796", 32, 32, 128, "bf16", 1),
        # fp32 activations and a smaller head
        _lin("ragged_f32", "5,1,130,64,1021,333", 12, 4, 64, "f32", 1),
        # one request forked into four samples after its prompt, in every layer
        _pool("fork_1_to_4", "fork", 1, 24, 16, 32, 128, "bf16", 64, 4),
        # beams of 64 requests continue from their parents, in place
        _pool("reorder_256", "reorder", 64, 3, 16, 32, 128, "bf16", 257, 4),
        # the same for small states: latency and many short blocks
        _pool("reorder_small", "reorder", 100, 8, 2, 4, 32, "f32", 512, 4),
        # finished requests have left holes: the live blocks move down
        _pool("compact_512", "compact", 300, 2, 16, 32, 128, "bf16", 513, 100),
        # finished requests' blocks are zeroed
        _pool("free_37", "free", 37, 6, 16, 32, 128, "bf16", 129, 1),
    ]


def draw(rng):
    what = rng.choice(["decode", "short", "prefill", "mixed", "f32", "d64", "fork", "reorder",
                       "compact", "free"])
    if what in ("decode", "short", "prefill", "mixed"):
        kv = rng.choice([1, 2, 4, 8, 16])
        heads = kv * rng.choice([r for r in (1, 2, 4) if kv * r <= 48])
        past = rng.randrange(2)
        most = 500_000  # tokens times heads
        if what == "decode":
            return _lin(None, "1*%d" % _spread(rng, 1, min(300, 8000 // heads)), heads, kv, 128,
                        "bf16", past)
        if what == "short":
            n = _spread(rng, 1, min(96, 3000 // heads))
            return _lin(None, ",".join(str(rng.randint(1, 24)) for _ in range(n)), heads, kv, 128,
                        "bf16", past)
        lens = []
        for _ in range(_spread(rng, 1, 12)):
            left = most // heads - sum(lens)
            if left < 17:
                break
            lens.append(_spread(rng, 17, min(left, 32768)))
        if what == "mixed":
            lens += [1] * _spread(rng, 1, 64)
            rng.shuffle(lens)
        return _lin(None, ",".join(map(str, lens)), heads, kv, 128, "bf16", past)
    if what in ("f32", "d64"):
        act, d = ("f32", rng.choice([32, 64, 128])) if what == "f32" else ("bf16", rng.choice([32, 64]))
        kv = rng.choice([1, 3, 5, 8])
        lens = [_spread(rng, 1, 1200) for _ in range(_spread(rng, 1, 8))]
        return _lin(None, ",".join(map(str, lens)), kv * rng.choice([1, 2]), kv, d, act, rng.randrange(2))
    hk, ratio, d, act = rng.choice([(16, 2, 128, "bf16"), (8, 2, 128, "bf16"), (2, 2, 32, "f32"),
                                    (3, 1, 64, "f32"), (4, 2, 64, "bf16")])
    layers = rng.randint(1, 4)
    if what == "fork":
        n, fan = _spread(rng, 1, 30), rng.randint(1, 4)
        return _pool(None, what, n, layers, hk, hk * ratio, d, act, n * (fan + 1) + rng.randint(1, 60), fan)
    if what == "reorder":
        n = _spread(rng, 1, 48)
        return _pool(None, what, n, layers, hk, hk * ratio, d, act, 4 * n + rng.randint(1, 60), 4)
    n = _spread(rng, 2, 100)
    return _pool(None, what, n, layers, hk, hk * ratio, d, act, 2 * n + rng.randint(1, 60),
                 rng.randint(1, n) if what == "compact" else 1)


def _block_bytes(case):
    """A pool block of a gated delta net layer: conv state, then fp32 state, on 128 bytes."""
    size = 4 if case["act"] == "f32" else 2
    conv = 3 * (2 * case["hk"] + case["hv"]) * case["d"] * size
    return -(-conv // 128) * 128 + case["hv"] * case["d"] ** 2 * 4


def work(case):
    if case["op"] == "pool":
        n, fan = case["n"], case["fan"]
        if case["what"] == "fork":
            blocks = n + n * fan
        elif case["what"] == "compact":
            blocks = 2 * fan
        elif case["what"] == "free":
            blocks = n
        else:
            blocks = 0
            for i in range(n):
                moved = [(b, p) for b, p in enumerate(BEAMS[i % len(BEAMS)]) if b != p]
                blocks += len(moved) + len({p for _, p in moved})
        return {"bytes": blocks * _block_bytes(case) * case["layers"], "flops": 0}
    lens = lengths(case["lens"])
    tokens, d, h = sum(lens), case["d"], case["heads"]
    size = 4 if case["act"] == "f32" else 2
    states = len(lens) * h * d * d * 4 * (2 if case["past"] else 1)
    rows = tokens * (2 * h + 2 * case["kv_heads"]) * d * size
    return {"bytes": states + rows, "flops": 4 * tokens * h * d * d}


# -- linear attention with a decay for each head -----------------------------


def _chunks(lens):
    """Per chunk: (sequence, first row, tokens, tokens of its sequence before it)."""
    out, row = [], 0
    for s, n in enumerate(lens):
        for at in range(0, n, CHUNK):
            out.append((s, row + at, min(CHUNK, n - at), at))
        row += n
    return out


def _prepare_lin(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    lens = lengths(case["lens"])
    h, hkv, d, n, t = case["heads"], case["kv_heads"], case["d"], len(lens), sum(lens)
    dtype = torch.float32 if case["act"] == "f32" else torch.bfloat16
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    # the rows of one fused projection: q, k and v are views of it
    qkv = rand(t, (h + 2 * hkv) * d).to(dtype)
    q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split([h * d, hkv * d, hkv * d], dim=1))
    # decays from fast to slow heads, geometric, with a layer's own factor
    speed = 0.2 + 0.8 * torch.rand(1, device="cuda", generator=g)
    log_decay = -(2.0 ** (-8.0 * torch.arange(1, h + 1, device="cuda") / h)) * speed
    blocks = n + 3
    states = torch.empty(blocks, h, d, d, device="cuda")
    pool = None
    if own:
        from continuous_linear_attention_gb300 import binding
        pool = binding.LinPool(blocks, 1, h, d, case["act"],
                               memory=states.view(-1).view(torch.uint8))
    states.normal_(0.0, 0.5, generator=g)
    states[0] = 0  # the block that stands for "no past"
    order = torch.randperm(blocks - 1, device="cuda", generator=g)[:n] + 1
    ch = _chunks(lens)
    col = lambda i: torch.tensor([c[i] for c in ch], device="cuda")  # noqa: E731
    return {
        "pool": pool, "q": q, "k": k, "v": v, "log_decay": log_decay.float(), "scale": d ** -0.5,
        "states": states, "idx": order.to(torch.int32),
        "has_past": torch.full((n,), case["past"], dtype=torch.uint8, device="cuda"),
        "cu": torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32),
        "out": torch.zeros(t, h, d, dtype=dtype, device="cuda"), "n": n, "t": t,
        "hint": max(lens), "case": case,
        # where the plain form's chunks lie, from the host's own lengths
        "chunk_seq": col(0), "chunk_row": col(1), "chunk_len": col(2), "chunk_at": col(3),
        "chunk_end": col(3) + col(2), "lens": torch.tensor(lens, device="cuda"),
        "width": min(CHUNK, max(lens)),
    }


def _decay(log_decay, steps):
    """e^{g steps} in fp64 for far positions, rounded to fp32."""
    return torch.exp(log_decay.double().view(-1, *[1] * steps.dim()) * steps.double()).float()


def _run_lin(st):
    if own:
        from continuous_linear_attention_gb300 import binding
        binding.lin_varlen_forward(st["pool"], 0, st["q"], st["k"], st["v"], st["cu"], st["idx"],
                                   st["has_past"], st["log_decay"], st["out"], st["t"], st["n"],
                                   scale=st["scale"], max_seqlen_hint=st["hint"])
        return st["out"], st["states"]
    q, k, v, w = st["q"].float(), st["k"].float(), st["v"].float(), st["width"]
    h, d, g = q.shape[1], q.shape[2], st["log_decay"]
    group = h // k.shape[1]
    past = torch.where(st["has_past"].bool()[:, None, None, None], st["states"][st["idx"].long()], 0.0)
    if w == 1:  # one token each: the recurrence itself
        k, v = k.repeat_interleave(group, 1), v.repeat_interleave(group, 1)
        s = past * torch.exp(g)[:, None, None] + k[..., :, None] * v[..., None, :]
        st["out"].copy_((q[..., None, :] @ s).squeeze(-2) * st["scale"])
        st["states"][st["idx"].long()] = s
        return st["out"], st["states"]
    seq, row, num, at, end = (st["chunk_" + x] for x in ("seq", "row", "len", "at", "end"))
    pos = torch.arange(w, device=q.device)
    valid = pos < num[:, None]
    rows = torch.where(valid, row[:, None] + pos, 0)
    # [chunk, head, token, channel], rows past a chunk's end zero
    pick = lambda x: torch.where(valid[..., None, None], x[rows], 0.0).transpose(1, 2)  # noqa: E731
    qc, kc, vc = pick(q), pick(k), pick(v)
    kc, vc = kc.repeat_interleave(group, 1), vc.repeat_interleave(group, 1)
    gap = pos[:, None] - pos
    inside = _decay(g, gap.clamp(min=0)) * (gap >= 0)
    o = ((qc @ kc.transpose(-1, -2)) * inside) @ vc
    # what each chunk adds to the state at its own end
    to_end = _decay(g, (num[:, None] - 1 - pos).clamp(min=0)) * valid
    add = (kc * to_end.transpose(0, 1)[..., None]).transpose(-1, -2) @ vc
    add = add.transpose(0, 1).flatten(2)  # [head, chunk, d * d]
    # the state before every chunk, and behind every sequence
    between = at[:, None] - end
    before = (seq[:, None] == seq) & (between >= 0)
    s = (_decay(g, between.clamp(min=0)) * before) @ add
    s = s.unflatten(-1, (d, d)).transpose(0, 1) + past[seq] * _decay(g, at).transpose(0, 1)[..., None, None]
    o = o + (qc @ s) * _decay(g, pos + 1)[..., None]
    left = st["lens"][:, None] - end
    mine = torch.arange(st["n"], device=q.device)[:, None] == seq
    last = (_decay(g, left.clamp(min=0)) * mine) @ add
    last = last.unflatten(-1, (d, d)).transpose(0, 1)
    last = last + past * _decay(g, st["lens"]).transpose(0, 1)[..., None, None]
    st["out"][rows[valid]] = (o.transpose(1, 2)[valid] * st["scale"]).to(st["out"].dtype)
    st["states"][st["idx"].long()] = last
    return st["out"], st["states"]


def _exact_lin(case, seed):
    st = _prepare_lin(case, seed)
    lens = lengths(case["lens"])
    if max(lens) > 20000 and case["heads"] * len(lens) > 64:
        return None  # too many steps over too many states
    alpha = torch.exp(st["log_decay"].double())[:, None, None]
    q, k, v = st["q"].double(), st["k"].double(), st["v"].double()
    group = q.shape[1] // k.shape[1]
    idx = st["idx"].long()
    s = st["states"][idx].double() * case["past"]
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    first = st["cu"][:-1].long()
    # token by token; the sequences that have one, longest first, are a prefix
    order = sorted(range(len(lens)), key=lambda i: -lens[i])
    s, first = s[order], first[order]
    live = len(lens)
    for t in range(max(lens)):
        while lens[order[live - 1]] <= t:
            live -= 1
        r = first[:live] + t
        kt, vt = (x[r].repeat_interleave(group, 1) for x in (k, v))
        s[:live] = s[:live] * alpha + kt[..., :, None] * vt[..., None, :]
        out[r] = torch.einsum("nhk,nhkv->nhv", q[r], s[:live]) * st["scale"]
    states = st["states"].double()
    states[idx[order]] = s
    return out, states


# -- the pool's blocks --------------------------------------------------------


def _prepare_pool(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    blocks, layers, n, fan = case["blocks"], case["layers"], case["n"], case["fan"]
    words = _block_bytes(case) // 4
    mem = torch.empty(layers, blocks, words, dtype=torch.int32, device="cuda")
    pool = None
    if own:
        from continuous_linear_attention_gb300 import binding
        pool = binding.Pool(blocks, layers, case["hk"], case["hv"], case["d"], case["d"], 4,
                            case["act"], memory=mem.view(-1).view(torch.uint8))
    mem.random_(generator=g)
    mem[:, 0] = 0  # the block that stands for "no past"
    perm = torch.randperm(blocks - 1, device="cuda", generator=g).to(torch.int32) + 1
    st = {"pool": pool, "mem": mem, "what": case["what"]}
    if case["what"] == "fork":
        st["src"] = perm[:n].repeat_interleave(fan)
        st["dst"] = perm[n:n + n * fan].clone()
    elif case["what"] == "reorder":
        parent = torch.tensor([4 * i + p for i in range(n) for p in BEAMS[i % len(BEAMS)]], device="cuda")
        st["dst"] = perm[:4 * n].clone()
        st["src"] = st["dst"][parent]
    elif case["what"] == "free":
        st["dst"] = perm[:n].clone()
    else:
        # `fan` live blocks lie above the n lowest, as many of those are free
        low, high = perm[perm <= n], perm[perm > n]
        idx = torch.cat([low[:n - fan], high[:fan]])
        st["idx"] = idx[torch.randperm(n, device="cuda", generator=g)].contiguous()
        st["new"] = torch.zeros_like(st["idx"])
    return st


def _run_pool(st):
    mem, what = st["mem"], st["what"]
    if own:
        if what == "free":
            st["pool"].clear_blocks(st["dst"])
        elif what == "compact":
            st["pool"].compact(st["idx"], st["new"])
        else:
            st["pool"].copy_blocks(st["src"], st["dst"])
        return (mem, st["new"]) if what == "compact" else mem
    if what == "free":
        mem[:, st["dst"].long()] = 0
        return mem
    if what != "compact":
        mem[:, st["dst"].long()] = mem[:, st["src"].long()]
        return mem
    idx = st["idx"].long()
    number = torch.arange(mem.shape[1], device=mem.device)
    live = torch.zeros_like(number).scatter_(0, idx, 1)
    top = live.sum()
    is_high = (live == 1) & (number > top)
    is_hole = (live == 0) & (number > 0) & (number <= top)
    high, hole = number[is_high], number[is_hole]
    mem[:, hole] = mem[:, high]
    moved = number.clone()
    moved[high] = hole
    st["new"].copy_(moved[idx])
    return mem, st["new"]


def prepare(case, seed):
    return _prepare_lin(case, seed) if case["op"] == "lin" else _prepare_pool(case, seed)


def run(state):
    return _run_lin(state) if "q" in state else _run_pool(state)


def exact(case, seed):
    return _exact_lin(case, seed) if case["op"] == "lin" else None  # blocks are only moved
