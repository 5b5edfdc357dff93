"""The operators of the layers beside the gated delta net ones in hybrid models, as measured.

Four operators, each in a plain form (elementary torch operations, fp32) and,
with ``own`` true, through the calls a user makes of the library:

``rope``  norms of queries and keys for each head with the position rotation
          in the same pass: RMS norm over a head's channels times a weight,
          then channel pairs turned by position * inv_freq.
``win``   causal attention with a sliding window and a few first tokens that
          stay visible, over a packed batch, continued from each request's
          keys and values in its pool block (the first tokens, then a ring):
          position p sees j <= p with j > p - window or j < sinks.
``conv``  the short causal convolution and SiLU before a selective scan,
          continued from each request's last inputs in its pool block.
``scan``  the selective state space scan with its skip and gate, continued
          from each request's fp32 state in its pool block:
            h_t = e^{dt_t A} h_{t-1} + dt_t u_t B_t,  dt = softplus(dt_raw + bias)
            y_t = (h_t C_t + D u_t) silu(z_t)

Lengths are texts such as "1*64,300,512": 64 single tokens, then two prompts.
"""
import math
import random

import torch

own = False

PROMPTS = "1077,3211,1519,793,2618,3999,547,2079"  # a prompt batch of ragged lengths
CHUNK = 64     # tokens per chunk of the plain scan
QUERIES = 128  # queries per chunk of the plain attention


def lengths(text):
    out = []
    for part in text.split(","):
        n, _, times = part.partition("*")
        out += [int(n)] * int(times or 1)
    return out


def _spread(rng, lo, hi):
    """An integer of [lo, hi], uniform in its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _rope(name, tokens, heads, kv_heads, d, rot, act, norm=1, offset=0, pairs=0, far=100_000):
    c = {"op": "rope", "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "d": d, "rot": rot,
         "act": act, "norm": norm, "offset": offset, "pairs": pairs, "far": far}
    return {"name": name, **c} if name else c


def _win(name, lens, heads, kv_heads, d, window, sinks, act, past):
    c = {"op": "win", "lens": lens, "heads": heads, "kv_heads": kv_heads, "d": d, "window": window,
         "sinks": sinks, "act": act, "past": past}
    return {"name": name, **c} if name else c


def _conv(name, lens, channels, taps, act, past, bias=1):
    c = {"op": "conv", "lens": lens, "channels": channels, "taps": taps, "act": act, "past": past,
         "bias": bias}
    return {"name": name, **c} if name else c


def _scan(name, lens, channels, n, act, past, gate=1):
    c = {"op": "scan", "lens": lens, "channels": channels, "n": n, "act": act, "past": past,
         "gate": gate}
    return {"name": name, **c} if name else c


def listed():
    return [
        # one request generating alone: the latency of a token's norms and rotation
        _rope("rope_1", 1, 32, 8, 128, 128, "bf16"),
        # the rows of a prompt batch: every query and key head streams in and out
        _rope("rope_16k", 15843, 32, 8, 128, 128, "bf16"),
        # one request generating alone over a long window
        _win("win_1", "1", 32, 8, 128, 4096, 4, "bf16", 100_000),
        # a full generation batch: every window streams in
        _win("win_256", "1*256", 32, 8, 128, 1024, 4, "bf16", 8192),
        # a prompt batch of ragged lengths, no past
        _win("win_16k", PROMPTS, 32, 8, 128, 1024, 4, "bf16", 0),
        # continuous batching: generation with drafted tokens, prompts and continued prompts among it
        _win("win_mixed", "1*48,4*16,511,2048,1283,700,1790,1732", 32, 8, 128, 1024, 4, "bf16", 3000),
        # fp32 activations, a smaller head, an odd window, few heads
        _win("win_f32", "5,1,130,64,1021,333", 12, 4, 64, 200, 3, "f32", 77),
        # a full generation batch's convolution: latency and short rows
        _conv("conv_256", "1*256", 4096, 4, "bf16", 1),
        # the convolution of a prompt batch
        _conv("conv_16k", PROMPTS, 4096, 4, "bf16", 0),
        # a full generation batch: every state streams in and out
        _scan("scan_256", "1*256", 4096, 16, "bf16", 1),
        # a prompt batch of ragged lengths, no past
        _scan("scan_16k", PROMPTS, 4096, 16, "bf16", 0),
        # one long prompt of few channels: not enough chains to fill the GPU by themselves
        _scan("scan_32k", "32768", 2048, 16, "bf16", 0),
    ]


def _ragged(rng, tokens, most, longest):
    """Lengths of up to `most` sequences of 2 .. longest tokens, `tokens` in all at most."""
    lens = []
    for _ in range(_spread(rng, 1, most)):
        left = tokens - sum(lens)
        if left < 2:
            break
        lens.append(_spread(rng, 2, min(left, longest)))
    return lens


def _text(lens):
    return ",".join(map(str, lens))


def draw(rng):
    what = rng.choice(["rope", "rope", "decode", "verify", "prompts", "mixed", "other", "conv", "conv",
                       "scan_decode", "scan", "scan", "scan_other"])
    if what == "rope":
        d = rng.choice([32, 64, 128, 128, 256])
        kv = rng.choice([1, 2, 3, 4, 8])
        heads = kv * rng.choice([1, 2, 4, 5, 8])
        tokens = _spread(rng, 1, min(16000, 80_000_000 // ((heads + kv) * d)))
        return _rope(None, tokens, heads, kv, d, rng.choice([d, d, d // 2, d // 4]),
                     rng.choice(["bf16", "bf16", "f32"]), rng.choice([1, 1, 0]), rng.randrange(2),
                     rng.randrange(2), rng.choice([100, 100_000, 4_000_000]))
    if what in ("decode", "verify", "prompts", "mixed"):
        kv = rng.choice([1, 2, 4, 8])
        heads = kv * rng.choice([1, 2, 4, 4, 7, 8])
        d = rng.choice([64, 128, 128])
        window, sinks = _spread(rng, 64, 4096), rng.choice([0, 1, 4, 4, 16, 64])
        past = rng.choice([0, 5, window // 2, 3 * window, 2_000_000])
        if what in ("decode", "verify"):
            n = _spread(rng, 1, min(300, 2_000_000 // (kv * window)))
            lens = [1] * n if what == "decode" else [rng.randint(1, 12) for _ in range(n)]
            return _win(None, _text(lens), heads, kv, d, window, sinks, "bf16", past)
        lens = _ragged(rng, 360_000_000 // (heads * window), 10, 16000)
        if what == "mixed":
            lens += [1] * _spread(rng, 1, 64)
            rng.shuffle(lens)
        return _win(None, _text(lens), heads, kv, d, window, sinks, "bf16", past)
    if what == "other":
        d, act = rng.choice([(32, "bf16"), (32, "f32"), (64, "f32"), (128, "f32")])
        kv = rng.choice([1, 2, 3])
        window = _spread(rng, 1, 600)
        return _win(None, _text([_spread(rng, 1, 900) for _ in range(_spread(rng, 1, 8))]),
                    kv * rng.choice([1, 2, 3]), kv, d, window, rng.choice([0, 2, 9]), act,
                    rng.choice([0, 40, 1000]))
    channels = rng.choice([8 * rng.randint(8, 200), 1024, 2048, 4096])
    if what == "conv":
        lens = [1] * _spread(rng, 1, 256) if rng.randrange(2) else _ragged(rng, 30_000_000 // channels, 12, 16000)
        return _conv(None, _text(lens), channels, rng.choice([2, 3, 4, 4]),
                     rng.choice(["bf16", "bf16", "f32"]), rng.randrange(2), rng.randrange(2))
    if what == "scan_decode":
        return _scan(None, "1*%d" % _spread(rng, 1, 300), channels, rng.choice([16, 16, 32]),
                     rng.choice(["bf16", "bf16", "f32"]), rng.randrange(2), rng.randrange(2))
    if what == "scan":
        lens = _ragged(rng, 30_000_000 // channels, 10, 16000) + [1] * rng.choice([0, 0, 3, 20])
        rng.shuffle(lens)
        return _scan(None, _text(lens), channels, 16, "bf16", rng.randrange(2), rng.randrange(2))
    lens = _ragged(rng, 6_000_000 // channels, 6, 4000)
    return _scan(None, _text(lens), channels, rng.choice([16, 32, 64]), rng.choice(["bf16", "f32"]),
                 rng.randrange(2), rng.randrange(2))


def _size(case):
    return 4 if case["act"] == "f32" else 2


def _dtype(case):
    return torch.float32 if case["act"] == "f32" else torch.bfloat16


def work(case):
    size = _size(case)
    if case["op"] == "rope":
        values = case["tokens"] * (case["heads"] + case["kv_heads"]) * case["d"]
        return {"bytes": 2 * values * size + 4 * case["tokens"], "flops": 8 * values}
    lens = lengths(case["lens"])
    tokens = sum(lens)
    if case["op"] == "win":
        h, kv, d, w, s, past = (case[x] for x in ("heads", "kv_heads", "d", "window", "sinks", "past"))
        rows, pairs = 2 * tokens * (h + kv), 0
        for n in lens:
            rows += 2 * kv * (min(past, s + w - 1) + min(n, s + w))
            for p in range(past, past + n):
                pairs += min(p + 1, w) + min(s, max(0, p + 1 - w))
        return {"bytes": rows * d * size, "flops": 4 * pairs * h * d}
    c = case["channels"]
    states = len(lens) * (2 if case["past"] else 1)
    if case["op"] == "conv":
        return {"bytes": (2 * tokens + states * (case["taps"] - 1) + case["taps"]) * c * size,
                "flops": 2 * tokens * c * case["taps"]}
    n = case["n"]
    return {"bytes": states * c * n * 4 + tokens * ((3 + case["gate"]) * c + 2 * n) * size + 4 * c * n,
            "flops": tokens * c * (7 * n + 4)}


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


# -- norms of queries and keys with the rotation -------------------------------


def _prepare_rope(case, seed):
    g = _generator(seed)
    t, h, kv, d, dtype = case["tokens"], case["heads"], case["kv_heads"], case["d"], _dtype(case)
    # the rows of one fused projection: q and k are views of it
    qkv = (torch.randn(t, (h + 2 * kv) * d, device="cuda", generator=g) * 2).to(dtype)
    q, k, _ = (x.unflatten(1, (-1, d)) for x in qkv.split([h * d, kv * d, kv * d], dim=1))
    first = int(torch.randint(case["far"], (1,), device="cuda", generator=g))
    # two requests' positions, one behind the other
    positions = torch.cat([first + torch.arange(t - t // 3), torch.arange(t // 3)]).to(torch.int32).cuda()
    weight = lambda: 1 - case["offset"] + 0.2 * torch.randn(d, device="cuda", generator=g)  # noqa: E731
    return {
        "case": case, "q": q, "k": k, "positions": positions,
        "q_weight": weight() if case["norm"] else None, "k_weight": weight() if case["norm"] else None,
        "inv_freq": (10000.0 ** (-torch.arange(0, case["rot"], 2).double() / case["rot"])).float().cuda(),
        "q_out": torch.zeros(t, h, d, dtype=dtype, device="cuda"),
        "k_out": torch.zeros(t, kv, d, dtype=dtype, device="cuda"),
    }


def _turned(x, weight, offset, cos, sin, pairs, eps):
    """x [T, heads, d] (fp32 or fp64) with its norm and rotation."""
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * (weight + offset)
    half = cos.shape[-1]
    cos, sin = cos[:, None], sin[:, None]
    if pairs:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([y, x[..., 2 * half:]], dim=-1)


def _run_rope(st):
    case = st["case"]
    if own:
        from continuous_linear_attention_gb300 import binding
        binding.qk_norm_rope(st["q"], st["k"], st["positions"], st["inv_freq"], q_weight=st["q_weight"],
                             k_weight=st["k_weight"], q_out=st["q_out"], k_out=st["k_out"], eps=1e-6,
                             weight_offset=case["offset"], interleaved=bool(case["pairs"]))
        return st["q_out"], st["k_out"]
    angle = st["positions"].double()[:, None] * st["inv_freq"].double()
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    for x in "qk":
        st[x + "_out"].copy_(_turned(st[x].float(), st[x + "_weight"], float(case["offset"]), cos, sin,
                                     case["pairs"], 1e-6))
    return st["q_out"], st["k_out"]


def _exact_rope(case, seed):
    st = _prepare_rope(case, seed)
    turns = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                        st["positions"].double()[:, None] * st["inv_freq"].double())[:, None]
    half, out = case["rot"] // 2, []
    for x in "qk":
        y, w = st[x].double(), st[x + "_weight"]
        if w is not None:
            y = y / (y.square().mean(-1, keepdim=True) + 1e-6).sqrt() * (w.double() + case["offset"])
        r = y[..., :2 * half]
        r = r.unflatten(-1, (half, 2)) if case["pairs"] else r.unflatten(-1, (2, half)).transpose(-1, -2)
        r = torch.view_as_real(torch.view_as_complex(r.contiguous()) * turns)
        y[..., :2 * half] = (r if case["pairs"] else r.transpose(-1, -2)).flatten(-2)
        out.append(y)
    return tuple(out)


# -- attention with a sliding window and sinks -----------------------------------


def _prepare_win(case, seed):
    g = _generator(seed)
    lens = lengths(case["lens"])
    h, kv, d, w, s = (case[x] for x in ("heads", "kv_heads", "d", "window", "sinks"))
    n, t, dtype = len(lens), sum(lens), _dtype(case)
    qkv = torch.randn(t, (h + 2 * kv) * d, device="cuda", generator=g).to(dtype)
    q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split([h * d, kv * d, kv * d], dim=1))
    blocks = n + 2
    # a block: keys, then values, of the first `sinks` positions and of a ring of `window`
    words = -(-2 * kv * (s + w) * d * _size(case) // 128) * 128 // _size(case)
    mem = torch.empty(blocks, words, dtype=dtype, device="cuda")
    pool = None
    if own:
        from continuous_linear_attention_gb300 import binding
        pool = binding.WinPool(blocks, 1, kv, d, w, s, case["act"], memory=mem.view(-1).view(torch.uint8))
    mem.normal_(generator=g)
    mem[0] = 0  # the block that stands for "no past"
    order = torch.randperm(blocks - 1, device="cuda", generator=g)[:n] + 1
    past = torch.randint(64, (n,), device="cuda", generator=g) + case["past"] if case["past"] else \
        torch.zeros(n, dtype=torch.int64, device="cuda")
    st = {
        "case": case, "pool": pool, "q": q, "k": k, "v": v, "scale": d ** -0.5, "mem": mem,
        "kv": mem[:, :2 * kv * (s + w) * d].unflatten(1, (2, kv, s + w, d)),
        "idx": order.to(torch.int32), "past": past.to(torch.int32),
        "cu": torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32),
        "out": torch.zeros(t, h, d, dtype=dtype, device="cuda"), "n": n, "t": t, "hint": max(lens),
        "lens": lens,
    }
    # where the plain form's chunks of queries lie, single tokens apart from longer sequences
    st["chunks"], row = [], 0
    one, more = [], []
    for i, m in enumerate(lens):
        if m == 1:
            one.append((i, row, 1, 0))
        else:
            more += [(i, row + a, min(QUERIES, m - a), a) for a in range(0, m, QUERIES)]
        row += m
    for width, group in ((1, one), (QUERIES, more)):
        per = max(1, (1 << 27) // (h * width * (width + w + s)))
        for a in range(0, len(group), per):
            st["chunks"].append((width, torch.tensor(group[a:a + per], device="cuda").T))
    return st


def _run_win(st):
    if own:
        from continuous_linear_attention_gb300 import binding
        binding.win_varlen_forward(st["pool"], 0, st["q"], st["k"], st["v"], st["cu"], st["idx"], st["past"],
                                   st["out"], st["t"], st["n"], scale=st["scale"],
                                   max_seqlen_hint=st["hint"])
        return st["out"], st["kv"]
    case, dev = st["case"], st["q"].device
    w, s = case["window"], case["sinks"]
    cu, past, idx = st["cu"].long(), st["past"].long(), st["idx"].long()
    group = case["heads"] // case["kv_heads"]
    for width, (seq, row, num, at) in st["chunks"]:
        i = torch.arange(width, device=dev)
        rows = (row[:, None] + i).clamp(max=st["t"] - 1)
        first = past[seq] + at  # the chunk's first position
        pos = first[:, None] + i
        # the keys: the sinks, then the window of the first query up to the last one
        j = torch.cat([torch.arange(s, device=dev).expand(len(seq), s),
                       first[:, None] - w + 1 + torch.arange(w + width - 1, device=dev)], dim=1)
        there = (j >= 0) & (j < (first + num)[:, None])
        there[:, s:] &= j[:, s:] >= s
        new = j >= past[seq][:, None]
        new_row = torch.where(there & new, cu[seq][:, None] + j - past[seq][:, None], 0)
        slot = torch.where(j < s, j, s + (j - s) % w)
        slot = torch.where(there & ~new, slot, 0)
        blk = idx[seq][:, None]

        def pick(fresh, part):
            x = torch.where(new[..., None, None], fresh[new_row], st["kv"][blk, part, :, slot]).float()
            return torch.where(there[..., None, None], x, 0.0).transpose(1, 2)  # [chunk, kv, key, d]

        kk, vv = pick(st["k"], 0), pick(st["v"], 1)
        qq = st["q"][rows].float().transpose(1, 2).unflatten(1, (-1, group))  # [chunk, kv, group, width, d]
        see = there[:, None] & (j[:, None] <= pos[..., None]) & \
            ((j[:, None] > pos[..., None] - w) | (j[:, None] < s))
        see = see[:, None, None]
        score = qq.flatten(2, 3) @ kk.transpose(-1, -2) * st["scale"]
        score = score.unflatten(2, (group, width)).masked_fill(~see, -math.inf)
        top = score.amax(-1, keepdim=True).clamp(min=-3e38)
        p = torch.exp(score - top)
        o = (p.flatten(2, 3) @ vv).unflatten(2, (group, width)) / p.sum(-1, keepdim=True)
        o = o.flatten(1, 2).transpose(1, 2)
        real = i < num[:, None]
        st["out"][rows[real]] = o[real].to(st["out"].dtype)
    # the last tokens go into the ring, the first ones to their places
    seq = torch.repeat_interleave(torch.arange(st["n"], device=dev), cu[1:] - cu[:-1], output_size=st["t"])
    j = past[seq] + torch.arange(st["t"], device=dev) - cu[seq]
    total = past + cu[1:] - cu[:-1]
    keep = (j < s) | (j >= total[seq] - w)
    slot = torch.where(j < s, j, s + (j - s) % w)
    b, at = idx[seq][keep], slot[keep]
    st["kv"][b, 0, :, at] = st["k"][keep]
    st["kv"][b, 1, :, at] = st["v"][keep]
    return st["out"], st["kv"]


def _exact_win(case, seed):
    st = _prepare_win(case, seed)
    w, s, kv, h, d = (case[x] for x in ("window", "sinks", "kv_heads", "heads", "d"))
    pairs = work(case)["flops"]
    if pairs > 1.5e12:
        return None  # too many products in 64 bits
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    kv_after = st["kv"].double()
    row = 0
    for i, n in enumerate(st["lens"]):
        past, blk = int(st["past"][i]), int(st["idx"][i])
        # every position that any of these queries can see, in order
        lo = max(s, past - w + 1)
        old = list(range(min(s, past))) + list(range(lo, past))
        slots = torch.tensor([p if p < s else s + (p - s) % w for p in old], dtype=torch.long, device="cuda")
        pos = torch.cat([torch.tensor(old, dtype=torch.long, device="cuda"),
                         torch.arange(past, past + n, device="cuda")])
        keys, values = (torch.cat([st["kv"][blk, part][:, slots].double(),
                                   st["kv"[part]][row:row + n].transpose(0, 1).double()], dim=1)
                        for part in (0, 1))
        for a in range(0, n, 512):
            m = min(512, n - a)
            p = torch.arange(past + a, past + a + m, device="cuda")
            near = ((pos < s) | (pos > past + a - w)) & (pos < past + a + m)
            kk, vv, pp = keys[:, near], values[:, near], pos[near]
            qq = st["q"][row + a:row + a + m].double().reshape(m, kv, h // kv, d).permute(1, 2, 0, 3)
            score = torch.einsum("ngmd,nkd->ngmk", qq, kk) * st["scale"]
            hidden = (pp > p[:, None]) | ((pp <= p[:, None] - w) & (pp >= s))
            o = torch.softmax(score.masked_fill(hidden, -math.inf), -1)
            out[row + a:row + a + m] = torch.einsum("ngmk,nkd->mngd", o, vv).reshape(m, h, d)
        last = [p for p in range(past, past + n) if p < s or p >= past + n - w]
        to = torch.tensor([p if p < s else s + (p - s) % w for p in last], dtype=torch.long, device="cuda")
        at = torch.tensor(last, dtype=torch.long, device="cuda") - past + row
        for part in (0, 1):
            kv_after[blk, part][:, to] = st["kv"[part]][at].transpose(0, 1).double()
        row += n
    return out, kv_after


# -- the selective scan's pool, convolution and scan --------------------------------


def _prepare_sel(case, seed):
    g = _generator(seed)
    lens = lengths(case["lens"])
    c, n, t, dtype = case["channels"], len(lens), sum(lens), _dtype(case)
    taps, states = case.get("taps", 4), case.get("n", 16)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    blocks = n + 2
    up = lambda b: -(-b // 128) * 128  # noqa: E731
    conv_bytes = (taps - 1) * c * _size(case)
    stride = up(up(conv_bytes) + c * states * 4)
    mem = torch.empty(blocks, stride, dtype=torch.uint8, device="cuda")
    pool = None
    if own:
        from continuous_linear_attention_gb300 import binding
        pool = binding.SelPool(blocks, 1, c, states, taps, case["act"], memory=mem.view(-1))
    mem.zero_()
    conv = mem[:, :conv_bytes].view(dtype).unflatten(1, (taps - 1, c))
    ssm = mem[:, up(conv_bytes):up(conv_bytes) + c * states * 4].view(torch.float32).unflatten(1, (c, states))
    conv.copy_(rand(blocks, taps - 1, c))
    ssm.copy_(rand(blocks, c, states) * 0.1)
    mem[0] = 0  # the block that stands for "no past"
    order = torch.randperm(blocks - 1, device="cuda", generator=g)[:n] + 1
    # x and z are the two halves of one projection's rows
    xz = rand(t, 2 * c).to(dtype)
    st = {
        "case": case, "pool": pool, "x": xz[:, :c], "conv": conv, "ssm": ssm, "idx": order.to(torch.int32),
        "has_past": torch.full((n,), case["past"], dtype=torch.uint8, device="cuda"),
        "cu": torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32),
        "out": torch.zeros(t, c, dtype=dtype, device="cuda"), "n": n, "t": t, "hint": max(lens), "lens": lens,
    }
    if case["op"] == "conv":
        st["weight"] = (rand(c, taps) * 0.5).to(dtype)
        st["bias"] = (rand(c) * 0.1).to(dtype) if case["bias"] else None
        return st
    rank = -(-c // 128) * 8
    low = rand(t, rank + 2 * states).to(dtype)  # time step, B and C of one projection's rows
    st["z"] = xz[:, c:] if case["gate"] else None
    st["u"] = torch.nn.functional.silu(rand(t, c)).to(dtype)
    st["dt"] = (rand(t, c) * 0.5).to(dtype)
    st["B"], st["C"] = low[:, rank:rank + states], low[:, rank + states:]
    st["A_log"] = torch.log(torch.arange(1, states + 1, device="cuda").float()) + 0.1 * rand(c, states)
    step = torch.exp(torch.rand(c, device="cuda", generator=g) * math.log(100.0) + math.log(1e-3))
    st["dt_bias"] = step + torch.log(-torch.expm1(-step))
    st["D"] = 1 + 0.1 * rand(c)
    # where the plain form's chunks lie
    ch, row = [], 0
    for i, m in enumerate(lens):
        ch += [(i, row + a, min(CHUNK, m - a), a) for a in range(0, m, CHUNK)]
        row += m
    st["chunks"] = torch.tensor(ch, device="cuda").T
    st["width"] = min(CHUNK, max(lens))
    # the chunks that are k-th of their sequence, for every k
    order = {}
    for i, (_, _, _, a) in enumerate(ch):
        order.setdefault(a // CHUNK, []).append(i)
    st["kth"] = [torch.tensor(order[k], device="cuda") for k in sorted(order)]
    last = {q: i for i, (q, _, _, _) in enumerate(ch)}
    st["last"] = torch.tensor([last[i] for i in range(n)], device="cuda")
    return st


def _run_conv(st):
    case, taps = st["case"], st["case"]["taps"]
    if own:
        from continuous_linear_attention_gb300 import binding
        binding.sel_conv_varlen_forward(st["pool"], 0, st["x"], st["cu"], st["idx"], st["has_past"],
                                        st["weight"], st["bias"], st["out"], st["t"], st["n"],
                                        max_seqlen_hint=st["hint"])
        return st["out"], st["conv"]
    dev, cu, idx = st["x"].device, st["cu"].long(), st["idx"].long()
    seq = torch.repeat_interleave(torch.arange(st["n"], device=dev), cu[1:] - cu[:-1], output_size=st["t"])
    at = torch.arange(st["t"], device=dev) - cu[seq]
    past = torch.where(st["has_past"].bool()[:, None, None], st["conv"][idx], 0.0)
    acc = torch.zeros(st["t"], case["channels"], device=dev)
    if st["bias"] is not None:
        acc += st["bias"].float()
    for k in range(taps):
        back = taps - 1 - k  # tokens before this one
        row = torch.arange(st["t"], device=dev) - back
        x = st["x"][row.clamp(min=0)].float()
        before = at < back
        rows = before.nonzero().squeeze(1)
        x[rows] = past[seq[rows], at[rows] - back + taps - 1].float()
        acc += x * st["weight"][:, k].float()
    st["out"].copy_(acc / (1 + torch.exp(-acc)))
    # the last inputs, the former ones among them where a sequence is short
    lens = cu[1:] - cu[:-1]
    for k in range(taps - 1):
        row = lens - (taps - 1) + k
        fresh = st["x"][(cu[:-1] + row).clamp(min=0)]
        old = past[torch.arange(st["n"], device=dev), (row + taps - 1).clamp(max=taps - 2)]
        st["conv"][idx, k] = torch.where((row >= 0)[:, None], fresh, old)
    return st["out"], st["conv"]


def _exact_conv(case, seed):
    st = _prepare_sel(case, seed)
    taps, row = case["taps"], 0
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    conv = st["conv"].double()
    for i, n in enumerate(st["lens"]):
        blk = int(st["idx"][i])
        line = torch.cat([st["conv"][blk].double() * case["past"], st["x"][row:row + n].double()])
        y = (line.unfold(0, taps, 1) * st["weight"].double()).sum(-1)
        if st["bias"] is not None:
            y = y + st["bias"].double()
        out[row:row + n] = y * torch.sigmoid(y)
        conv[blk] = line[n:]
        row += n
    return out, conv


def _run_scan(st):
    case = st["case"]
    if own:
        from continuous_linear_attention_gb300 import binding
        binding.sel_scan_varlen_forward(st["pool"], 0, st["u"], st["dt"], st["B"], st["C"], st["z"], st["cu"],
                                        st["idx"], st["has_past"], st["A_log"], st["D"], st["dt_bias"],
                                        st["out"], st["t"], st["n"], max_seqlen_hint=st["hint"])
        return st["out"], st["ssm"]
    idx = st["idx"].long()
    a = -torch.exp(st["A_log"])
    u = st["u"].float()
    raw = st["dt"].float() + st["dt_bias"]
    dt = raw.clamp(min=0) + torch.log1p(torch.exp(-raw.abs()))
    b, c = st["B"].float(), st["C"].float()
    past = torch.where(st["has_past"].bool()[:, None, None], st["ssm"][idx], 0.0)
    y = torch.zeros(st["t"] + 1, u.shape[1], device=u.device)  # the last row takes what is behind a chunk's end
    if st["width"] == 1:  # one token each: the recurrence itself
        h = past * torch.exp(dt[..., None] * a) + (dt * u)[..., None] * b[:, None]
        y = (h * c[:, None]).sum(-1)
        st["ssm"][idx] = h
    else:
        seq, row, num, _ = st["chunks"]

        def advance(h, out):
            """All chunks side by side, a token at a time; rows behind a chunk's end change nothing."""
            for i in range(st["width"]):
                r = (row + i).clamp(max=st["t"] - 1)
                real = (i < num).float()[:, None]
                step = dt[r] * real
                h = h * torch.exp(step[..., None] * a) + (step * u[r])[..., None] * b[r][:, None]
                if out is not None:
                    out[torch.where(i < num, row + i, st["t"])] = (h * c[r][:, None]).sum(-1)
            return h

        start = torch.zeros(len(seq), *a.shape, device=u.device)
        if len(st["kth"]) > 1:  # the states at the chunks' starts, from the chunks' own
            mine = advance(start, None)
            total = torch.zeros(st["t"] + 1, u.shape[1], dtype=torch.float64, device=u.device)
            torch.cumsum(dt.double(), 0, out=total[1:])
            span = (total[row + num] - total[row]).float()
            h = past
            for of in st["kth"]:
                start[of] = h[seq[of]]
                h = h.clone()
                h[seq[of]] = h[seq[of]] * torch.exp(span[of][..., None] * a) + mine[of]
        else:
            start = past[seq]
        end = advance(start, y)
        st["ssm"][idx] = end[st["last"]]
    y = y[:st["t"]] + st["D"] * u
    if st["z"] is not None:
        z = st["z"].float()
        y = y * z / (1 + torch.exp(-z))
    st["out"].copy_(y)
    return st["out"], st["ssm"]


def _exact_scan(case, seed):
    st = _prepare_sel(case, seed)
    lens = st["lens"]
    idx = st["idx"].long()
    a = -torch.exp(st["A_log"].double())
    h = st["ssm"][idx].double() * case["past"]
    # token by token; the sequences that have one, longest first, are a prefix
    order = sorted(range(len(lens)), key=lambda i: -lens[i])
    h, first = h[order], st["cu"][:-1].long()[order]
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    live = len(lens)
    for t in range(max(lens)):
        while lens[order[live - 1]] <= t:
            live -= 1
        r = first[:live] + t
        u = st["u"][r].double()
        dt = torch.nn.functional.softplus(st["dt"][r].double() + st["dt_bias"].double(), threshold=700)
        h[:live] = h[:live] * torch.exp(dt[..., None] * a) + (dt * u)[..., None] * st["B"][r].double()[:, None]
        out[r] = torch.einsum("scn,sn->sc", h[:live], st["C"][r].double()) + u * st["D"].double()
    if st["z"] is not None:
        z = st["z"].double()
        out = out * z * torch.sigmoid(z)
    states = st["ssm"].double()
    states[idx[order]] = h
    return out, states


def prepare(case, seed):
    op = case["op"]
    return _prepare_rope(case, seed) if op == "rope" else _prepare_win(case, seed) if op == "win" else \
        _prepare_sel(case, seed)


def run(state):
    return {"rope": _run_rope, "win": _run_win, "conv": _run_conv, "scan": _run_scan}[state["case"]["op"]](state)


def exact(case, seed):
    return {"rope": _exact_rope, "win": _exact_win, "conv": _exact_conv, "scan": _exact_scan}[case["op"]](case, seed)
