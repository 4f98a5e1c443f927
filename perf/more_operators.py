"""Timed cases of the operators that take a decoding step of several sequences through a mixture-of-experts
model, beside the products, the cache and the attention that are there already.

Three groups, in the order in which a step meets them:

- "norm": each head's query and key divided by its root mean square, scaled by the gains and rotated to its
  position, in one pass;
- "moe": a whole mixture-of-experts layer for a few tokens: the router's logits, the chosen experts and their
  weights, the experts' SwiGLU products and their weighted sum;
- "sample": the next token of each sequence drawn from its logits with temperature, top-k, top-p and min-p, from
  one given uniform number.

`run` computes them in their plain form (elementary torch operations, fp32; fp64 for angles, for the router's logits
and for the sampler's sums, where neighbouring values decide a whole number), or, where `own` is true, through this
package's entry points. `exact` is the definition in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}

# (query heads, KV heads, head_dim, RoPE base) of the decode workloads of this repository
HEADS = {
    "tiny": (4, 2, 64, 10000.0),
    "llama1b": (32, 8, 64, 500000.0),
    "tinyllama": (32, 4, 64, 10000.0),
    "qwen1.5b": (12, 2, 128, 1000000.0),
    "3b": (40, 8, 64, 10000.0),
}


def _norm(name, heads, seqs, tokens, pos_lo, pos_hi, dtype, rotary, ragged=False):
    """rotary: rotated dimensions of a head."""
    return {"name": name, "op": "norm", "heads": heads, "seqs": seqs, "tokens": tokens, "pos_lo": pos_lo,
            "pos_hi": pos_hi, "dtype": dtype, "rotary": rotary, "ragged": ragged}


def _moe(name, tokens, experts, top_k, hidden, ffn, weights, group, dtype, renormalise=True):
    """weights: "bf16", "int4 f16" or "int4 bf16" (4-bit weights with scales of that type for each `group` inputs)."""
    return {"name": name, "op": "moe", "tokens": tokens, "experts": experts, "top_k": top_k, "hidden": hidden,
            "ffn": ffn, "weights": weights, "group": group, "dtype": dtype, "renormalise": renormalise}


def _sample(name, rows, vocab, dtype, temperature, top_k, top_p, min_p, spread=2.5, masked=0, mixed=False):
    """mixed: parameters differ from row to row (each around the given one)."""
    return {"name": name, "op": "sample", "rows": rows, "vocab": vocab, "dtype": dtype, "temperature": temperature,
            "top_k": top_k, "top_p": top_p, "min_p": min_p, "spread": spread, "masked": masked, "mixed": mixed}


def listed():
    return [
        # one decode step of one sequence (the smallest call)
        _norm("norm_token", "llama1b", 1, 1, 1051, 1051, "f32", 64),
        # one decode step of a batch with contexts from short to long
        _norm("norm_batch", "3b", 64, 1, 15, 8191, "bf16", 64),
        # prompts of different lengths, half of each head rotated
        _norm("norm_ragged", "tinyllama", 16, 511, 0, 777, "f16", 32, True),
        # long prompts of a batch
        _norm("norm_prompt", "qwen1.5b", 8, 4095, 0, 0, "bf16", 128),
        # one decode step of one sequence, 4-bit experts
        _moe("moe_token", 1, 64, 8, 2048, 1024, "int4 f16", 64, "f32"),
        # eight drafted tokens verified
        _moe("moe_verify", 8, 64, 8, 2048, 1024, "bf16", 0, "f32"),
        # a few sequences, few and small experts, weights as the softmax leaves them
        _moe("moe_small", 5, 16, 2, 512, 256, "int4 bf16", 128, "f16", False),
        # one decode step of a batch: nearly every expert is used
        _moe("moe_batch", 64, 64, 8, 2048, 1024, "bf16", 0, "bf16"),
        # one token of one sequence with everything switched on
        _sample("sample_token", 1, 128256, "f32", 0.7, 50, 0.9, 0.02),
        # one token of each sequence of a batch from the nucleus of the whole vocabulary, requests of their own
        _sample("sample_nucleus", 64, 151936, "bf16", 1.0, 0, 0.95, 0.0, masked=1000, mixed=True),
        # drawn from the softmax as it is
        _sample("sample_whole", 37, 32000, "f32", 1.0, 0, 1.0, 0.0),
        # many sequences, likeliest tokens only
        _sample("sample_many", 512, 128256, "bf16", 0.8, 40, 1.0, 0.05),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "moe", "moe", "sample", "sample"])
    if op == "norm":
        heads = rng.choice(sorted(HEADS))
        d = HEADS[heads][2]
        seqs = _log(rng, 1, 64)
        tokens = _log(rng, 1, max(1, 32000 // seqs)) if rng.random() < 0.6 else 1
        pos_lo = rng.choice([0, _log(rng, 1, 2000)])
        pos_hi = pos_lo + rng.choice([0, _log(rng, 1, 100000)])
        c = _norm("", heads, seqs, min(tokens, 5000), pos_lo, pos_hi, rng.choice(["f32", "bf16", "f16"]),
                  rng.choice([d, d, d // 2]), rng.random() < 0.5)
        while work(c)["bytes"] > 2.3e8:
            c["tokens"] = c["tokens"] * 2 // 3
    elif op == "moe":
        weights = rng.choice(["bf16", "int4 f16", "int4 bf16"])
        group = rng.choice([32, 64, 128]) if weights != "bf16" else 0
        step = max(group, 32)
        experts = _log(rng, 4, 64)
        hidden = step * (_log(rng, 256, 2560) // step)
        ffn = step * (_log(rng, 128, 1536) // step)
        c = _moe("", _log(rng, 1, 64), experts, rng.randint(1, min(8, experts)), hidden, ffn, weights, group,
                 rng.choice(["f32", "bf16", "f16"]), rng.random() < 0.7)
        while work(c)["bytes"] > 7.5e8:
            c["experts"] -= 4
    else:
        vocab = rng.choice([2048, 32000, 49152, 128256, 151936, _log(rng, 50, 200000)])
        rows = _log(rng, 1, max(1, min(1000, 512 * 128256 // vocab // 2)))
        c = _sample("", rows, vocab, rng.choice(["f32", "bf16", "f16"]), rng.choice([1.0, round(rng.uniform(0.3, 1.8), 3)]),
                    rng.choice([0, 0, _log(rng, 1, 1000)]), rng.choice([1.0, round(rng.uniform(0.3, 0.99), 3)]),
                    rng.choice([0.0, 0.0, round(rng.uniform(0.001, 0.3), 4)]), round(rng.uniform(1.0, 4.0), 2),
                    rng.choice([0, rng.randint(0, vocab // 2)]), rng.random() < 0.3)
    return {k: v for k, v in c.items() if k != "name"}


# ------------------------------------------------------------------ the cases' shapes

def _positions(case):
    """First position and number of tokens of each sequence: spread evenly over the case's range, in a fixed shuffled
    order."""
    s, lo, hi, t = case["seqs"], case["pos_lo"], case["pos_hi"], case["tokens"]
    pos = [min(hi, lo + (hi - lo) * ((i * 37) % s) // max(1, s - 1)) if s > 1 else hi for i in range(s)]
    counts = [max(1, t - (i * 5) % max(1, t)) if case["ragged"] else t for i in range(s)]
    return pos, counts


def work(case):
    size = SIZE[case["dtype"]]
    if case["op"] == "norm":
        hq, hk, d, _ = HEADS[case["heads"]]
        n = sum(_positions(case)[1]) * (hq + hk) * d
        return {"bytes": 2 * n * size + 8 * d, "flops": 6 * n}
    if case["op"] == "sample":
        r, v = case["rows"], case["vocab"]
        return {"bytes": r * v * size + 12 * r, "flops": 5 * r * v}
    m, e, k, h, f = (case[n] for n in ("tokens", "experts", "top_k", "hidden", "ffn"))
    used = e * (1.0 - (1.0 - k / e) ** m)  # experts that some token chooses, where tokens choose by chance
    per = 2.0 if case["weights"] == "bf16" else 0.5 + 2.0 / case["group"]
    return {"bytes": int(used * 3 * h * f * per) + 2 * e * h + 2 * m * h * size + 8 * m * k,
            "flops": 6 * m * k * h * f + 2 * m * e * h}


# ------------------------------------------------------------------ inputs

def _weight(g, case, rows, cols):
    """A stack of matrices [experts][rows][cols] and its scales (None: bf16)."""
    e = case["experts"]
    if case["weights"] == "bf16":
        w = torch.empty((e, rows, cols), dtype=torch.bfloat16, device=DEV)
        for i in range(e):
            w[i] = torch.randn((rows, cols), generator=g, device=DEV) * cols ** -0.5
        return w, None
    w = torch.randint(0, 256, (e, rows, cols // 2), generator=g, device=DEV, dtype=torch.uint8)
    s = torch.randn((e, rows, cols // case["group"]), generator=g, device=DEV).abs() * (0.2 * cols ** -0.5)
    return w, s.to(torch.float16 if case["weights"] == "int4 f16" else torch.bfloat16)


def _own():
    import decode_persistent_megakernel_gb300 as T
    return T


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 2654435761 % (1 << 62) + 29)
    dt = DTYPE[case["dtype"]]
    if case["op"] == "norm":
        hq, hk, d, theta = HEADS[case["heads"]]
        pos, counts = _positions(case)
        s, t = case["seqs"], case["tokens"]
        # queries, keys and values of a token lie side by side, as the fused projection leaves them
        qkv = torch.empty((s, t, hq + 2 * hk, d), dtype=dt, device=DEV)
        for i in range(s):
            qkv[i] = torch.randn((t, hq + 2 * hk, d), generator=g, device=DEV) * 2.0
        return {"case": case, "theta": theta, "eps": 1e-6, "q": qkv[:, :, :hq], "k": qkv[:, :, hq:hq + hk],
                "q_gain": 1.0 + 0.2 * torch.randn(d, generator=g, device=DEV),
                "k_gain": 1.0 + 0.2 * torch.randn(d, generator=g, device=DEV),
                "pos": torch.tensor(pos, dtype=torch.int32, device=DEV),
                "counts": torch.tensor(counts, dtype=torch.int32, device=DEV),
                "q_out": torch.zeros((s, t, hq, d), dtype=dt, device=DEV),
                "k_out": torch.zeros((s, t, hk, d), dtype=dt, device=DEV)}
    if case["op"] == "moe":
        m, e, h, f = (case[n] for n in ("tokens", "experts", "hidden", "ffn"))
        state = {"case": case, "x": torch.randn((m, h), generator=g, device=DEV).to(dt)}
        favour = torch.exp(0.3 * torch.randn((e, 1), generator=g, device=DEV))  # some experts are chosen more often
        state["router"] = (torch.randn((e, h), generator=g, device=DEV) * favour * h ** -0.5).to(torch.bfloat16)
        for name, rows, cols in (("g", f, h), ("u", f, h), ("d", h, f)):
            state["w" + name], state["s" + name] = _weight(g, case, rows, cols)
        state["y"] = torch.zeros((m, h), dtype=dt, device=DEV)
        if own:  # the layer that a serving program keeps, its experts packed once
            T = _own()
            state["layer"] = T.MoeLayer(state["router"], state["wg"], state["wu"], state["wd"], top_k=case["top_k"],
                                        scales=(state["sg"], state["su"], state["sd"]) if state["sg"] is not None else None,
                                        group=case["group"], renormalise=case["renormalise"], max_tokens=m)
        return state
    rows, vocab = case["rows"], case["vocab"]
    logits = torch.empty((rows, vocab), dtype=dt, device=DEV)
    step = max(1, (1 << 27) // vocab)
    for r in range(0, rows, step):
        logits[r:r + step] = torch.randn((min(step, rows - r), vocab), generator=g, device=DEV) * case["spread"]
    if case["masked"]:
        hidden = torch.randperm(vocab, generator=g, device=DEV)[:min(case["masked"], vocab - 1)]
        logits[:, hidden] = -math.inf
    state = {"case": case, "logits": logits, "u": torch.rand(rows, generator=g, device=DEV)}
    for name in ("temperature", "top_k", "top_p", "min_p"):
        state[name] = case[name]
    if case["mixed"]:  # each sequence has a request of its own
        v = torch.rand((4, rows), generator=g, device=DEV)
        state["temperature"] = case["temperature"] * (0.5 + v[0])
        state["top_k"] = (case["top_k"] * (0.5 + v[1])).to(torch.int32)
        state["top_p"] = 1.0 - (1.0 - case["top_p"]) * 2.0 * v[2]
        state["min_p"] = case["min_p"] * 2.0 * v[3]
    return state


# ------------------------------------------------------------------ plain forms

def _plain_norm_one(x, gain, pos, counts, eps, theta, rotary, out):
    s, t, h, d = x.shape
    x = x.float()
    y = x / torch.sqrt((x * x).mean(dim=-1, keepdim=True) + eps) * gain
    i = torch.arange(rotary // 2, dtype=torch.float64, device=x.device)
    at = pos.to(torch.float64)[:, None] + torch.arange(t, dtype=torch.float64, device=x.device)
    angle = at[:, :, None] * torch.pow(torch.tensor(theta, dtype=torch.float64, device=x.device), -2.0 * i / rotary)
    c, n = torch.cos(angle).float()[:, :, None, :], torch.sin(angle).float()[:, :, None, :]
    a, b, rest = y[..., :rotary // 2], y[..., rotary // 2:rotary], y[..., rotary:]
    y = torch.cat([a * c - b * n, b * c + a * n, rest], dim=-1).to(out.dtype)
    valid = torch.arange(t, device=x.device) < counts[:, None]
    out.copy_(torch.where(valid[:, :, None, None], y, out))


def _dense(w, s, group):
    """Matrices [...][rows][cols] in fp32."""
    if s is None:
        return w.float()
    q = torch.stack([w & 15, w >> 4], dim=-1).flatten(-2).float() - 8.0
    return (q.unflatten(-1, (-1, group)) * s.float()[..., None]).flatten(-2)


def _plain_moe(st):
    c = st["case"]
    x = st["x"].float()
    logits = torch.matmul(x.double(), st["router"].double().t())
    value, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    value, ids = value[:, :c["top_k"]], ids[:, :c["top_k"]]
    e = torch.exp(value - value[:, :1])
    total = e.sum(dim=1, keepdim=True) if c["renormalise"] else torch.exp(logits - value[:, :1]).sum(dim=1, keepdim=True)
    weights = (e / total).float()
    if ids.numel() <= c["experts"]:  # the chosen experts' matrices, token by token
        chosen = ids.flatten()
        wg, wu, wd = (_dense(st["w" + n][chosen], None if st["s" + n] is None else st["s" + n][chosen], c["group"])
                      for n in "gud")
        each = x.repeat_interleave(c["top_k"], dim=0)[:, :, None]
        a = torch.matmul(wg, each)
        h = a / (1.0 + torch.exp(-a)) * torch.matmul(wu, each)
        st["y"].copy_((torch.matmul(wd, h)[:, :, 0].view(x.shape[0], c["top_k"], -1) * weights[:, :, None]).sum(dim=1))
        return {"y": st["y"], "ids": ids.to(torch.int32), "weights": weights}
    share = torch.zeros((x.shape[0], c["experts"]), device=x.device).scatter_(1, ids, weights)
    y = torch.zeros_like(x)
    for i in range(c["experts"]):  # every expert over all tokens, those that did not choose it with weight 0
        wg, wu, wd = (_dense(st["w" + n][i], None if st["s" + n] is None else st["s" + n][i], c["group"]) for n in "gud")
        a = torch.matmul(x, wg.t())
        h = a / (1.0 + torch.exp(-a)) * torch.matmul(x, wu.t())
        y += share[:, i:i + 1] * torch.matmul(h, wd.t())
    st["y"].copy_(y)
    return {"y": st["y"], "ids": ids.to(torch.int32), "weights": weights}


def _column(v, like):
    """A parameter as a column of fp64, one value for each row."""
    if not torch.is_tensor(v):
        v = torch.full((like.shape[0],), float(torch.tensor(v, dtype=torch.float32)), dtype=torch.float64, device=like.device)
    return v.double()[:, None]


def _plain_sample(st):
    x = st["logits"].float()
    t, k, p, low = (_column(st[n], x) for n in ("temperature", "top_k", "top_p", "min_p"))
    value, index = torch.sort(x, dim=1, descending=True, stable=True)
    w = torch.exp((value.double() - value[:, :1].double()) / t)
    place = torch.arange(x.shape[1], device=x.device)
    w = torch.where((k > 0) & (place >= k), 0.0, w)
    before = torch.cumsum(w, dim=1) - w
    w = torch.where((p < 1) & (place > 0) & (before >= p * w.sum(dim=1, keepdim=True)), 0.0, w)
    w = torch.where(w < low, 0.0, w)
    w = torch.zeros_like(w).scatter_(1, index, w)  # in the vocabulary's order
    end = torch.cumsum(w, dim=1)
    total = end[:, -1:].clone()
    ids = (end <= st["u"].double()[:, None] * total).sum(dim=1)
    return {"ids": ids.to(torch.int32), "logp": torch.log(w.gather(1, ids[:, None]) / total)[:, 0].float()}


def run(st):
    c = st["case"]
    if c["op"] == "norm":
        a = (st["pos"], st["counts"], st["eps"], st["theta"], c["rotary"])
        if own:
            _own().qk_norm_rope(st["q"], st["k"], st["q_gain"], st["k_gain"], st["pos"], counts=st["counts"], eps=st["eps"],
                                rope_theta=st["theta"], rotary_dim=c["rotary"], out=(st["q_out"], st["k_out"]))
        else:
            _plain_norm_one(st["q"], st["q_gain"], *a, st["q_out"])
            _plain_norm_one(st["k"], st["k_gain"], *a, st["k_out"])
        return {"q": st["q_out"], "k": st["k_out"]}
    if c["op"] == "moe":
        if not own:
            return _plain_moe(st)
        y, ids, weights = st["layer"](st["x"], out=st["y"])
        return {"y": y, "ids": ids, "weights": weights}
    if not own:
        return _plain_sample(st)
    ids, logp = _own().sample(st["logits"], st["u"], temperature=st["temperature"], top_k=st["top_k"], top_p=st["top_p"],
                              min_p=st["min_p"])
    return {"ids": ids, "logp": logp}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_norm(x, gain, pos, counts, eps, theta, rotary):
    s, t, h, d = x.shape
    out = torch.zeros((s, t, h, d), dtype=torch.float64, device=x.device)
    f = torch.tensor([theta ** (-2.0 * i / rotary) for i in range(rotary // 2)], dtype=torch.float64, device=x.device)
    for i, (first, n) in enumerate(zip(pos, counts)):
        y = x[i, :n].double()
        y = y * torch.rsqrt(torch.linalg.vector_norm(y, dim=-1, keepdim=True) ** 2 / d + eps) * gain.double()
        a = torch.outer(torch.arange(first, first + n, dtype=torch.float64, device=x.device), f)
        z = torch.complex(y[..., :rotary // 2], y[..., rotary // 2:rotary]) * torch.polar(torch.ones_like(a), a)[:, None, :]
        out[i, :n] = torch.cat([z.real, z.imag, y[..., rotary:]], dim=-1)
    return out


def _exact_matrix(w, s, group):
    if s is None:
        return w.double()
    q = torch.empty((w.shape[0], 2 * w.shape[1]), dtype=torch.float64, device=w.device)
    q[:, 0::2] = torch.remainder(w, 16).double() - 8.0
    q[:, 1::2] = torch.div(w, 16, rounding_mode="floor").double() - 8.0
    return q * s.double().repeat_interleave(group, dim=1)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm":
        pos, counts = _positions(case)
        a = (pos, counts, st["eps"], st["theta"], case["rotary"])
        return {"q": _exact_norm(st["q"], st["q_gain"], *a), "k": _exact_norm(st["k"], st["k_gain"], *a)}
    if case["op"] == "moe":
        x = st["x"].double()
        logits = torch.stack([(x * r).sum(dim=1) for r in st["router"].double()], dim=1)
        top, ids = torch.topk(logits, case["top_k"], dim=1)
        weights = torch.softmax(top, dim=1) if case["renormalise"] else torch.softmax(logits, dim=1).gather(1, ids)
        y = torch.zeros_like(x)
        for e in sorted(set(ids.flatten().tolist())):
            who, slot = (ids == e).nonzero(as_tuple=True)
            wg, wu, wd = (_exact_matrix(st["w" + n][e], None if st["s" + n] is None else st["s" + n][e], case["group"])
                          for n in "gud")
            h = torch.nn.functional.silu(x[who] @ wg.T) * (x[who] @ wu.T)
            y.index_add_(0, who, (h @ wd.T) * weights[who, slot][:, None])
        return {"y": y, "ids": ids.to(torch.int32), "weights": weights}
    ids, logp = [], []
    each = [_column(st[n], st["logits"])[:, 0].tolist() for n in ("temperature", "top_k", "top_p", "min_p")]
    for r, (t, k, p, low) in enumerate(zip(*each)):
        z = st["logits"][r].double() / t
        order = torch.argsort(z, descending=True, stable=True)
        n = int(k) if k > 0 else z.numel()
        share = torch.softmax(z[order][:n], dim=0)
        if p < 1:
            n = max(1, int((torch.cumsum(share, dim=0) - share < p).sum()))
        n = min(n, int((share >= low * share[0]).sum()))
        kept, _ = torch.sort(order[:n])
        q = torch.softmax(z[kept], dim=0)
        i = int(torch.searchsorted(torch.cumsum(q, dim=0), st["u"][r].double(), right=True))
        i = min(i, n - 1)
        ids.append(int(kept[i]))
        logp.append(torch.log(q[i]))
    return {"ids": torch.tensor(ids, dtype=torch.int32, device=DEV), "logp": torch.stack(logp)}
