"""Timed cases of the operators around an 8-bit KV cache and the scoring of tokens.

Three groups, as a serving program uses them next to the decode step:

- "store": keys and values of new tokens quantised into the cache as they are written (one scale for each
  block of tokens, KV head and tensor; keys rotated on the way), and read back;
- "attend": attention of one or more query tokens of each sequence over that cache;
- "score": the log probability of a given token for each row of logits, the row's entropy and its most
  likely alternatives.

`run` computes them in their plain form (elementary torch operations, fp32, fp64 for angles and long
sums), or, where `own` is true, through this package's entry points. `exact` is the definition in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
QMAX = {"e4m3": 448.0, "int8": 127.0}
DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SMALLEST_SCALE = 2.0 ** -126

# (query heads, KV heads, head_dim, RoPE base, vocabulary) of the decode workloads of this repository
HEADS = {
    "tiny": (4, 2, 64, 10000.0, 2048),
    "llama1b": (32, 8, 64, 500000.0, 128256),
    "tinyllama": (32, 4, 64, 10000.0, 32000),
    "qwen1.5b": (12, 2, 128, 1000000.0, 151936),
    "3b": (40, 8, 64, 10000.0, 49152),
}


def _store(name, heads, seqs, tokens, pos_lo, pos_hi, fmt, block, dtype, back, ragged=False):
    return {"name": name, "op": "store", "heads": heads, "seqs": seqs, "tokens": tokens, "pos_lo": pos_lo,
            "pos_hi": pos_hi, "fmt": fmt, "block": block, "dtype": dtype, "back": back, "ragged": ragged}


def _attend(name, heads, seqs, tokens, pos_lo, pos_hi, fmt, block, dtype, ragged=False):
    return {"name": name, "op": "attend", "heads": heads, "seqs": seqs, "tokens": tokens, "pos_lo": pos_lo,
            "pos_hi": pos_hi, "fmt": fmt, "block": block, "dtype": dtype, "ragged": ragged}


def _score(name, rows, vocab, dtype, top, pad=0, masked=0):
    return {"name": name, "op": "score", "rows": rows, "vocab": vocab, "dtype": dtype, "top": top, "pad": pad,
            "masked": masked}


def listed():
    return [
        # one decode step's key and value of one sequence, into a started block (the smallest call)
        _store("store_token", "llama1b", 1, 1, 1051, 1051, "e4m3", 64, "f32", False),
        # a prompt of one sequence, stored and read back
        _store("store_prompt", "qwen1.5b", 1, 4095, 0, 0, "int8", 64, "bf16", True),
        # prompts of a batch, of different lengths and from odd positions on, stored and read back
        _store("store_batch", "llama1b", 32, 2048, 0, 777, "e4m3", 32, "bf16", True, True),
        # one decode step of one sequence at the benchmark's context
        _attend("attend_token", "llama1b", 1, 1, 1151, 1151, "e4m3", 64, "f32"),
        # one decode step over a long context, two KV heads only: the context has to be split
        _attend("attend_long", "qwen1.5b", 1, 1, 131000, 131000, "e4m3", 128, "bf16"),
        # one decode step of a batch with contexts from short to long
        _attend("attend_batch", "3b", 64, 1, 15, 8191, "int8", 64, "bf16"),
        # drafted tokens verified, eight of each sequence (fewer in some)
        _attend("attend_verify", "tinyllama", 8, 8, 500, 4096, "e4m3", 16, "bf16", True),
        # a chunk of a long prompt over what is cached of it
        _attend("attend_chunk", "llama1b", 1, 512, 7680, 7680, "e4m3", 64, "bf16"),
        # a whole prompt
        _attend("attend_prompt", "qwen1.5b", 1, 4096, 0, 0, "int8", 64, "bf16"),
        # one sampled token's log probability and five alternatives
        _score("score_token", 1, 128256, "f32", 5),
        # drafted tokens scored, rows apart by an odd pad, a part of the vocabulary masked
        _score("score_verify", 64, 151936, "bf16", 20, 8, 1000),
        # every token of a prompt scored
        _score("score_prompt", 2047, 128256, "f32", 1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["store", "attend", "attend", "score"])
    if op == "score":
        vocab = rng.choice([2048, 32000, 49152, 128256, 151936, _log(rng, 50, 200000)])
        rows = _log(rng, 1, max(1, min(4096, 2047 * 128256 // vocab // 2)))
        top = rng.choice([0, 1, 5, 20, rng.randint(1, 32)])
        return {k: v for k, v in _score("", rows, vocab, rng.choice(["f32", "bf16", "f16"]), min(top, vocab),
                                        rng.choice([0, rng.randint(0, 64)]),
                                        rng.choice([0, rng.randint(0, vocab // 2)])).items() if k != "name"}
    heads = rng.choice(sorted(HEADS))
    hq, hk, d = HEADS[heads][:3]
    fmt, block = rng.choice(["e4m3", "int8"]), rng.choice([16, 32, 64, 128])
    dtype, ragged = rng.choice(["bf16", "f32"]), rng.random() < 0.5
    seqs = _log(rng, 1, 64)
    if op == "store":
        tokens = _log(rng, 1, min(4096, 65536 // seqs))
        pos_lo = rng.choice([0, _log(rng, 1, 2000)])
        pos_hi = pos_lo + rng.choice([0, _log(rng, 1, 1000)])
        back = dtype == "bf16"
        if not back:
            fmt = "e4m3"
        c = _store("", heads, seqs, tokens, pos_lo, pos_hi, fmt, block, dtype, back, ragged)
    else:
        many = rng.random() < 0.3
        if many:
            seqs = rng.randint(1, 3)
        tokens = _log(rng, 9, 1500) if many else rng.choice([1, 1, rng.randint(2, 8)])
        pos_hi = _log(rng, 1, min(100000, 400000 // seqs) if not many else 4000)
        pos_lo = rng.choice([pos_hi, rng.randint(0, pos_hi)])
        c = _attend("", heads, seqs, tokens, pos_lo, pos_hi, fmt, block, dtype, ragged)
        while work(c)["flops"] > 5e10:
            c["tokens"] = c["tokens"] * 2 // 3
    return {k: v for k, v in c.items() if k != "name"}


# ------------------------------------------------------------------ the cases' shapes

def _positions(case):
    """First new position and number of new tokens of each sequence: spread evenly over the case's range, in a
    fixed shuffled order."""
    s, lo, hi, t = case["seqs"], case["pos_lo"], case["pos_hi"], case["tokens"]
    pos = [lo + (hi - lo) * ((i * 37) % s) // max(1, s - 1) if s > 1 else hi for i in range(s)]
    pos = [min(hi, p) for p in pos]
    counts = [max(1, t - (i * 5) % max(1, t)) if case["ragged"] else t for i in range(s)]
    return pos, counts


def _max_ctx(case):
    pos, _ = _positions(case)
    return max(pos) + case["tokens"] + 5


def work(case):
    size = {"f32": 4, "bf16": 2, "f16": 2}[case["dtype"]]
    if case["op"] == "score":
        r, v, k = case["rows"], case["vocab"], case["top"]
        return {"bytes": r * v * size + 4 * r + 8 * r + 8 * r * k, "flops": 5 * r * v}
    hq, hk, d = HEADS[case["heads"]][:3]
    pos, counts = _positions(case)
    if case["op"] == "store":
        n = sum(counts) * hk * d * 2
        scales = sum((p % case["block"] + c + case["block"] - 1) // case["block"] for p, c in zip(pos, counts)) * hk * 8
        return {"bytes": n * (size + 1) + scales + (n * (2 + 1) + scales if case["back"] else 0), "flops": 4 * n}
    cached = sum(p + c for p, c in zip(pos, counts)) * hk
    pairs = sum(c * p + c * (c + 1) // 2 for p, c in zip(pos, counts)) * hq
    return {"bytes": int(cached * (2 * d + 8 / case["block"])) + 2 * sum(counts) * hq * d * size, "flops": 4 * d * pairs}


# ------------------------------------------------------------------ inputs

def _to_codes(x, fmt):
    """Values in units of their scale, rounded to the 8-bit format, as bytes."""
    if fmt == "e4m3":
        return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    return x.round().clamp(-127.0, 127.0).to(torch.int8).view(torch.uint8)


def _from_codes(c, fmt):
    return c.view(torch.float8_e4m3fn).float() if fmt == "e4m3" else c.view(torch.int8).float()


def _cached(g, shape, n_blocks, block, fmt, spread):
    """Codes and scales of a cache that earlier calls have filled."""
    s, h, ctx, d = shape
    size = torch.exp(spread * torch.randn((s, h, n_blocks), generator=g, device=DEV))
    x = torch.randn(shape, generator=g, device=DEV)
    if fmt == "e4m3":
        codes = _to_codes(x * 110.0, fmt)
    else:
        codes = _to_codes(x * 31.0, fmt)
    return codes, size * (1.0 / 110.0 if fmt == "e4m3" else 1.0 / 31.0)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 2654435761 % (1 << 62) + 17)
    if case["op"] == "score":
        rows, vocab, pad = case["rows"], case["vocab"], case["pad"]
        logits = torch.empty((rows, vocab + pad), dtype=DTYPE[case["dtype"]], device=DEV)
        step = max(1, (1 << 28) // (vocab + pad))
        for r in range(0, rows, step):
            logits[r:r + step] = torch.randn((min(step, rows - r), vocab + pad), generator=g, device=DEV) * 2.5
        if case["masked"]:
            hidden = torch.randperm(vocab, generator=g, device=DEV)[:case["masked"]]
            logits[:, hidden] = -math.inf
        targets = torch.randint(0, vocab, (rows,), generator=g, device=DEV, dtype=torch.int32)
        return {"case": case, "logits": logits[:, :vocab], "targets": targets}
    hq, hk, d, theta, _ = HEADS[case["heads"]]
    pos, counts = _positions(case)
    s, t, ctx, block = case["seqs"], case["tokens"], _max_ctx(case), case["block"]
    n_blocks = (ctx + block - 1) // block
    dt = DTYPE[case["dtype"]]
    state = {"case": case, "theta": theta, "longest": max(p + c for p, c in zip(pos, counts)),
             "pos": torch.tensor(pos, dtype=torch.int32, device=DEV),
             "counts": torch.tensor(counts, dtype=torch.int32, device=DEV)}
    state["k_codes"], state["k_scales"] = _cached(g, (s, hk, ctx, d), n_blocks, block, case["fmt"], 0.3)
    state["v_codes"], state["v_scales"] = _cached(g, (s, hk, ctx, d), n_blocks, block, case["fmt"], 0.5)
    if case["op"] == "store":
        state["k"] = (1.3 * torch.randn((s, t, hk, d), generator=g, device=DEV)).to(dt)
        state["v"] = (0.7 * torch.randn((s, t, hk, d), generator=g, device=DEV)).to(dt)
        if case["back"]:
            state["k_back"] = torch.zeros((s, t, hk, d), dtype=dt, device=DEV)
            state["v_back"] = torch.zeros((s, t, hk, d), dtype=dt, device=DEV)
    else:
        state["q"] = (1.5 * torch.randn((s, t, hq, d), generator=g, device=DEV)).to(dt)
        state["out"] = torch.zeros((s, t, hq, d), dtype=dt, device=DEV)
    if own:  # the handle over these buffers that a serving program keeps
        import decode_persistent_megakernel_gb300 as T
        state["cache"] = T.Kv8Cache(hk, d, ctx, n_seqs=s, fmt=T.TINFER_KV8_E4M3 if case["fmt"] == "e4m3" else T.TINFER_KV8_INT8,
                                    block=block, buffers=(state["k_codes"], state["v_codes"], state["k_scales"], state["v_scales"]))
    return state


# ------------------------------------------------------------------ plain forms

def _rotate(x, pos, theta):
    """Rotary positions (half-split pairs) of x [s][t][h][d] at pos[s] + t, angles in 64 bits."""
    s, t, h, d = x.shape
    i = torch.arange(d // 2, dtype=torch.float64, device=x.device)
    at = pos.to(torch.float64)[:, None] + torch.arange(t, dtype=torch.float64, device=x.device)
    angle = at[:, :, None] * torch.pow(torch.tensor(theta, dtype=torch.float64, device=x.device), -2.0 * i / d)
    c, n = torch.cos(angle).to(x.dtype)[:, :, None, :], torch.sin(angle).to(x.dtype)[:, :, None, :]
    a, b = x[..., :d // 2], x[..., d // 2:]
    return torch.cat([a * c - b * n, b * c + a * n], dim=-1)


def _plain_store_one(x, codes, scales, pos, counts, fmt, block):
    """Writes the rows x [s][t][h][d] (fp32) into one tensor of the cache."""
    s, t, h, d = x.shape
    dev = x.device
    n = (t + block - 2) // block + 1 if block > 1 else t
    first = torch.div(pos, block, rounding_mode="floor").long()
    into = (pos.long() - first * block)[:, None] + torch.arange(t, device=dev)
    valid = torch.arange(t, device=dev) < counts[:, None]
    which = torch.arange(s, device=dev)[:, None].expand(s, t)
    n = n + 1
    grid = torch.zeros((s, n * block, h, d), dtype=torch.float32, device=dev)
    grid[which[valid], into[valid]] = x[valid]
    new = torch.zeros((s, n * block), dtype=torch.bool, device=dev)
    new[which[valid], into[valid]] = True
    grid = grid.view(s, n, block, h, d)
    new = new.view(s, n, block)
    amax = grid.abs().amax(dim=(2, 4))                                   # [s][n][h]
    ids = first[:, None] + torch.arange(n, device=dev)                   # [s][n]
    here = new.any(dim=2)
    ids = torch.minimum(ids, torch.tensor(scales.shape[2] - 1, device=dev))
    seq = torch.arange(s, device=dev)[:, None].expand(s, n)
    old = scales[seq, :, ids]                                            # [s][n][h]
    started = torch.zeros((s, n), dtype=torch.bool, device=dev)
    started[:, 0] = pos % block > 0
    qmax = QMAX[fmt]
    fresh = torch.where(amax > 0, (amax / qmax).clamp_min(SMALLEST_SCALE), torch.zeros_like(amax))
    ratio = (amax.double() / qmax) / torch.where(old > 0, old, torch.ones_like(old)).double()
    grown = old * torch.exp2(torch.ceil(torch.log2(ratio.clamp_min(1.0)))).float()
    scale = torch.where(started[:, :, None] & (old > 0), grown, fresh)
    safe = torch.where(scale > 0, scale, torch.ones_like(scale))
    fresh_codes = _to_codes(grid / safe[:, :, None, :, None], fmt)        # [s][n][block][h][d]
    # codes of a started block's earlier tokens, in units of the grown scale
    row = ids[:, 0, None] * block + torch.arange(block, device=dev)
    earlier = (torch.arange(block, device=dev) < (pos.long() % block)[:, None])
    row = torch.minimum(row, torch.tensor(codes.shape[2] - 1, device=dev))
    seq_row = torch.arange(s, device=dev)[:, None].expand(s, block)
    held = codes[seq_row, :, row]                                         # [s][block][h][d]
    again = _to_codes(_from_codes(held, fmt) * (old[:, 0] / safe[:, 0])[:, None, :, None], fmt)
    grew = (old[:, 0] > 0) & (scale[:, 0] != old[:, 0])                   # [s][h]
    again = torch.where(grew[:, None, :, None], again, held)
    codes[seq_row[earlier], :, row[earlier]] = again[earlier]
    flat = fresh_codes.view(s, n * block, h, d)
    at = pos.long()[:, None] + torch.arange(t, device=dev)
    codes[which[valid], :, at[valid]] = flat[which[valid], into[valid]]
    scales[seq[here], :, ids[here]] = scale[here]


def _plain_read_one(codes, scales, pos, counts, fmt, block, out):
    s, t, h, d = out.shape
    dev = out.device
    at = pos.long()[:, None] + torch.arange(t, device=dev)
    valid = torch.arange(t, device=dev) < counts[:, None]
    seq = torch.arange(s, device=dev)[:, None].expand(s, t)
    x = _from_codes(codes[seq[valid], :, at[valid]], fmt)
    scale = scales[seq[valid], :, torch.div(at[valid], block, rounding_mode="floor")]
    out[valid] = (x * scale[:, :, None]).to(out.dtype)


def _plain_attend(st):
    c = st["case"]
    q, out, pos, counts = st["q"], st["out"], st["pos"], st["counts"]
    s, t, hq, d = q.shape
    hk, n, block = st["k_codes"].shape[1], st["longest"], c["block"]
    rows = torch.arange(n, device=q.device)
    blocks = torch.div(rows, block, rounding_mode="floor")
    k = _from_codes(st["k_codes"][:, :, :n], c["fmt"]) * st["k_scales"][:, :, blocks][..., None]
    v = _from_codes(st["v_codes"][:, :, :n], c["fmt"]) * st["v_scales"][:, :, blocks][..., None]
    x = _rotate(q.float(), pos, st["theta"]).view(s, t, hk, hq // hk, d).permute(0, 2, 3, 1, 4).reshape(s, hk, hq // hk * t, d)
    score = torch.matmul(x, k.transpose(-1, -2)) * (1.0 / math.sqrt(d))
    last = pos.long()[:, None] + torch.arange(t, device=q.device)
    seen = rows[None, None, :] <= last[:, :, None]                        # [s][t][n]
    score = score.view(s, hk, hq // hk, t, n).masked_fill(~seen[:, None, None], -math.inf)
    e = torch.exp(score - score.amax(dim=-1, keepdim=True))
    p = e / e.sum(dim=-1, keepdim=True)
    y = torch.matmul(p.view(s, hk, hq // hk * t, n), v).view(s, hk, hq // hk, t, d)
    y = y.permute(0, 3, 1, 2, 4).reshape(s, t, hq, d).to(out.dtype)
    valid = torch.arange(t, device=q.device) < counts[:, None]
    out.copy_(torch.where(valid[:, :, None, None], y, out))
    return out


def _plain_score(st):
    x = st["logits"].float()
    k = st["case"]["top"]
    m = x.amax(dim=1, keepdim=True)
    z = x - m
    e = torch.exp(z)
    total = e.sum(dim=1, dtype=torch.float64)
    mean = torch.where(e > 0, e * z, torch.zeros_like(e)).sum(dim=1, dtype=torch.float64) / total
    norm = torch.log(total)
    got = {"logp": (z.gather(1, st["targets"].long()[:, None])[:, 0].double() - norm).float(),
           "entropy": (norm - mean).float()}
    if k:
        value, index = torch.sort(z, dim=1, descending=True, stable=True)
        got["top_ids"] = index[:, :k].to(torch.int32).contiguous()
        got["top_logp"] = (value[:, :k].double() - norm[:, None]).float()
    return got


def _stored(st):
    """What a store pass returns: the values read back and the scales, or the cache as it is held."""
    if st["case"]["back"]:
        return {"k": st["k_back"], "v": st["v_back"], "k_scales": st["k_scales"], "v_scales": st["v_scales"]}
    return {"k": st["k_codes"].view(torch.float8_e4m3fn), "v": st["v_codes"].view(torch.float8_e4m3fn),
            "k_scales": st["k_scales"], "v_scales": st["v_scales"]}


def run(st):
    c = st["case"]
    if own:
        return _run_own(st)
    if c["op"] == "score":
        return _plain_score(st)
    if c["op"] == "attend":
        return {"out": _plain_attend(st)}
    a = (st["pos"], st["counts"], c["fmt"], c["block"])
    _plain_store_one(_rotate(st["k"].float(), st["pos"], st["theta"]), st["k_codes"], st["k_scales"], *a)
    _plain_store_one(st["v"].float(), st["v_codes"], st["v_scales"], *a)
    if c["back"]:
        _plain_read_one(st["k_codes"], st["k_scales"], *a, st["k_back"])
        _plain_read_one(st["v_codes"], st["v_scales"], *a, st["v_back"])
    return _stored(st)


def _run_own(st):
    c = st["case"]
    if c["op"] == "score":
        import decode_persistent_megakernel_gb300 as T
        logp, entropy, ids, top = T.logprobs(st["logits"], st["targets"], top_k=c["top"])
        got = {"logp": logp, "entropy": entropy}
        return {**got, "top_ids": ids, "top_logp": top} if c["top"] else got
    cache = st["cache"]
    if c["op"] == "attend":
        return {"out": cache.attention(st["q"], st["pos"], counts=st["counts"], rope_theta=st["theta"], out=st["out"])}
    cache.append(st["k"], st["v"], st["pos"], counts=st["counts"], rope_theta=st["theta"])
    if c["back"]:
        cache.read(c["tokens"], st["pos"], counts=st["counts"], out=(st["k_back"], st["v_back"]))
    return _stored(st)


# ------------------------------------------------------------------ the definitions in 64 bits

def _nearest(x, fmt):
    """x rounded to the nearest value of the format, ties to even, saturating (fp64 arithmetic)."""
    if fmt == "int8":
        return torch.round(x).clamp(-127, 127)
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 1).clamp_min(-6) - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _turned(x, first, theta):
    """Rotary positions of x [t][h][d] in fp64, as products of complex numbers."""
    t, h, d = x.shape
    f = torch.tensor([theta ** (-2.0 * i / d) for i in range(d // 2)], dtype=torch.float64, device=x.device)
    a = torch.outer(torch.arange(first, first + t, dtype=torch.float64, device=x.device), f)
    z = torch.complex(x[..., :d // 2], x[..., d // 2:]) * torch.polar(torch.ones_like(a), a)[:, None, :]
    return torch.cat([z.real, z.imag], dim=-1)


def _exact_store_one(x, codes, scales, pos, count, fmt, block):
    """x [t][h][d] fp64 into codes [h][ctx][d] and scales [h][blocks], both fp64, block by block."""
    qmax, at = QMAX[fmt], pos
    while at < pos + count:
        b = at // block
        end = min(pos + count, (b + 1) * block)
        rows = x[at - pos:end - pos].transpose(0, 1)                      # [h][rows][d]
        amax = rows.abs().amax(dim=(1, 2))
        scale = torch.where(amax > 0, (amax / qmax).clamp_min(SMALLEST_SCALE), torch.zeros_like(amax))
        if at > b * block:
            held = scales[:, b].clone()
            k = torch.ceil(torch.log2((amax / qmax / torch.where(held > 0, held, torch.ones_like(held))).clamp_min(1.0)))
            kept = held * torch.exp2(k)
            scale = torch.where(held > 0, kept, scale)
            part = codes[:, b * block:at]
            again = _nearest(part * torch.exp2(-k)[:, None, None], fmt)
            codes[:, b * block:at] = torch.where(((held > 0) & (k > 0))[:, None, None], again, part)
        safe = torch.where(scale > 0, scale, torch.ones_like(scale))
        codes[:, at:end] = _nearest(rows / safe[:, None, None], fmt)
        scales[:, b] = scale
        at = end


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "score":
        logp, entropy, top = [], [], []
        step = max(1, (1 << 27) // case["vocab"])
        for r in range(0, case["rows"], step):
            x = st["logits"][r:r + step].double()
            norm = torch.logsumexp(x, dim=1)
            p = torch.exp(x - norm[:, None])
            logp.append(x.gather(1, st["targets"][r:r + step].long()[:, None])[:, 0] - norm)
            entropy.append(norm - torch.nan_to_num(p * x, nan=0.0).sum(dim=1))
            if case["top"]:
                top.append(torch.topk(x, case["top"], dim=1).values - norm[:, None])
        got = {"logp": torch.cat(logp), "entropy": torch.cat(entropy)}
        return {**got, "top_ids": None, "top_logp": torch.cat(top)} if case["top"] else got
    hq, hk, d, theta, _ = HEADS[case["heads"]]
    pos, counts = _positions(case)
    fmt, block, t = case["fmt"], case["block"], case["tokens"]
    kc, vc = (_from_codes(st[n], fmt) for n in ("k_codes", "v_codes"))
    ks, vs = st["k_scales"].double(), st["v_scales"].double()
    if case["op"] == "store":
        kd, vd = kc.double(), vc.double()
        back = [torch.zeros((case["seqs"], t, hk, d), dtype=torch.float64, device=DEV) for _ in range(2)]
        for s, (p, c) in enumerate(zip(pos, counts)):
            _exact_store_one(_turned(st["k"][s].double(), p, theta), kd[s], ks[s], p, c, fmt, block)
            _exact_store_one(st["v"][s].double(), vd[s], vs[s], p, c, fmt, block)
            b = torch.arange(p, p + c, device=DEV) // block
            back[0][s, :c] = (kd[s, :, p:p + c] * ks[s][:, b, None]).transpose(0, 1)
            back[1][s, :c] = (vd[s, :, p:p + c] * vs[s][:, b, None]).transpose(0, 1)
        k, v = back if case["back"] else (kd, vd)
        return {"k": k, "v": v, "k_scales": ks, "v_scales": vs}
    out = torch.zeros((case["seqs"], t, hq, d), dtype=torch.float64, device=DEV)
    for s, (p, c) in enumerate(zip(pos, counts)):
        n = p + c
        b = torch.arange(n, device=DEV) // block
        late = torch.arange(n, device=DEV)[None, :] > torch.arange(p, n, device=DEV)[:, None]
        q = _turned(st["q"][s, :c].double(), p, theta)
        for h in range(hk):
            k = kc[s, h, :n].double() * ks[s, h, b][:, None]
            v = vc[s, h, :n].double() * vs[s, h, b][:, None]
            for g in range(h * (hq // hk), (h + 1) * (hq // hk)):
                w = torch.softmax((q[:, g] @ k.T / math.sqrt(d)).masked_fill(late, -math.inf), dim=1)
                out[s, :c, g] = w @ v
    return {"out": out}
