"""The operators around the FP8 linears, as cases to measure.

A rollout step of a decoder runs, besides its FP8 linears: the norm that ends
a residual branch and quantises the next linear's input (``rmsnorm_quant``),
causal attention over packed prompts (``attn_prefill``), attention of one new
token per sequence over the paged E4M3 cache that ``kv_append`` writes
(``attn_decode``), and the log probabilities of the sampled tokens with
entropy and top alternatives (``logprobs``), whose gradient the trainer takes
(``logprobs_backward``) and which ``tis_weights`` consumes.

``run`` computes each in its plain form (elementary torch operations in fp32,
one rounding at the end), or, with ``own`` set, through the package.  Head
counts and widths are those the benchmark and the tests use: hidden 4096 with
32 query and 8 KV heads of 128, hidden 2048 with 32 query and 4 KV heads.
"""
import math
import random

import torch

own = False

E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


# ------------------------------------------------------------------ the cases

def _norm(m, k, fmt, residual=True, **more):
    return {"op": "norm", "m": m, "k": k, "fmt": fmt, "residual": residual, **more}


def _prefill(lens, most, seed, hq, hkv, d, **more):
    # `lens` sequences, the longest of `most` tokens, the others drawn from `seed`
    return {"op": "prefill", "batch": lens, "most": most, "lens_seed": seed, "hq": hq, "hkv": hkv, "d": d, **more}


def _decode(batch, least, most, seed, hq, hkv, d, page, **more):
    return {"op": "decode", "batch": batch, "least": least, "most": most, "lens_seed": seed, "hq": hq, "hkv": hkv,
            "d": d, "page": page, **more}


def _logprob(op, rows, vocab, dtype, topk, temperature, **more):
    return {"op": op, "rows": rows, "vocab": vocab, "dtype": dtype, "topk": topk, "temperature": temperature, **more}


def listed():
    return [
        # one decode step's tokens: the call is launch latency
        _norm(16, 4096, "fp32", name="norm 16 tokens"),
        # a prefill batch in the power-of-two scale format
        _norm(8192, 4096, "ue8m0", name="norm 8192 tokens"),
        # one short prompt: a few tiles, latency
        _prefill(1, 509, 1, 32, 8, 128, name="prompt of 509"),
        # one long prompt
        _prefill(1, 8192, 1, 32, 8, 128, name="prompt of 8192"),
        # a rollout batch's prompts, packed, of different lengths; 8 query heads to a KV head
        _prefill(24, 2048, 7, 32, 4, 128, name="24 packed prompts"),
        # one sequence early in its answer: latency
        _decode(1, 1000, 1000, 1, 32, 8, 128, 16, name="cache of 1000"),
        # a rollout batch in flight, every length
        _decode(256, 0, 4096, 3, 32, 8, 128, 16, name="256 caches to 4096"),
        # few long answers: the work is along the cache; 8 query heads to a KV head
        _decode(4, 100000, 131071, 5, 32, 4, 128, 64, name="4 long caches"),
        # the sampled tokens of one decode step, with the top 20 for the log
        _logprob("logprob", 16, 151936, "bf16", 20, 0.7, name="logprob 16 rows top 20"),
        # the trainer's scoring of a packed batch
        _logprob("logprob", 4096, 151936, "bf16", 0, 1.0, name="logprob 4096 rows"),
        # gradient of a small batch in fp32, odd vocabulary
        _logprob("logprob_grad", 61, 32001, "fp32", 0, 1.0, name="logprob grad 61 rows"),
        # gradient of the packed batch
        _logprob("logprob_grad", 4096, 151936, "bf16", 0, 1.0, name="logprob grad 4096 rows"),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "prefill", "decode", "logprob", "logprob_grad"])
    if op == "norm":
        k = rng.choice([rng.choice([1024, 2048, 4096, 5120, 8192]), rng.randrange(200, 9000)])
        m = _log_uniform(rng, 1, 33e6 / k)
        return _norm(m, k, rng.choice(["fp32", "ue8m0"]), rng.random() < 0.75)
    if op == "prefill":
        hq, hkv = rng.choice([(32, 8), (32, 4), (16, 16), (12, 2), (24, 8)])
        d = rng.choice([128, 128, 64])
        batch = _log_uniform(rng, 1, 24)
        most = _log_uniform(rng, 1, 6000 / math.sqrt(batch))
        return _prefill(batch, most, rng.randrange(1 << 20), hq, hkv, d)
    if op == "decode":
        hq, hkv = rng.choice([(32, 8), (32, 4), (16, 16), (12, 2), (40, 4)])
        batch = _log_uniform(rng, 1, 256)
        most = _log_uniform(rng, 1, 400000 / batch if batch > 4 else 100000)
        return _decode(batch, rng.randrange(0, most + 1), most, rng.randrange(1 << 20), hq, hkv, rng.choice([128, 128, 64]),
                       rng.choice([1, 16, 32, 64, 48]))
    vocab = rng.choice([rng.choice([32000, 50257, 128256, 151936]), _log_uniform(rng, 100, 150000)])
    rows = _log_uniform(rng, 1, 3e8 / vocab)
    dtype = rng.choice(["bf16", "fp32"])
    top = rng.choice([0, 1, 5, 20, 32]) if op == "logprob" else 0
    return _logprob(op, min(rows, 8192), vocab, dtype, top, rng.choice([1.0, 0.6, 1.3]))


def _lens(case):
    r = random.Random(case["lens_seed"] * 1000003 + case["batch"])
    if case["op"] == "prefill":  # prompts: mostly short, some long
        lens = [max(1, int(case["most"] * r.random() ** 2)) for _ in range(case["batch"])]
    else:
        lens = [r.randrange(case["least"], case["most"] + 1) for _ in range(case["batch"])]
    lens[r.randrange(case["batch"])] = case["most"]
    return lens


def work(case):
    op = case["op"]
    if op == "norm":
        m, k = case["m"], case["k"]
        scale = 1 if case["fmt"] == "ue8m0" else 4
        # x and the residual in, their sum, the codes and the scales out, the weight
        return {"bytes": m * k * (7 if case["residual"] else 3) + scale * m * -(-k // 128) + 2 * k, "flops": 6 * m * k}
    if op in ("logprob", "logprob_grad"):
        n, size = case["rows"] * case["vocab"], 2 if case["dtype"] == "bf16" else 4
        if op == "logprob":
            return {"bytes": n * size + case["rows"] * (20 + 8 * case["topk"]), "flops": 5 * n}
        return {"bytes": 2 * n * size + case["rows"] * 24, "flops": 8 * n}
    lens = _lens(case)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if op == "prefill":
        return {"bytes": sum(lens) * d * 2 * (2 * hq + 2 * hkv) + sum(lens) * hq * 4, "flops": sum(2 * n * (n + 1) for n in lens) * hq * d}
    pages = sum(-(-n // case["page"]) for n in lens)
    return {"bytes": sum(lens) * hkv * d * 2 + case["batch"] * hq * (d * 4 + 4) + 4 * pages + 4 * case["batch"],
            "flops": sum(lens) * hq * d * 4}


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(dev)
    g.manual_seed(seed)
    op = case["op"]
    s = {"case": case}

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32)

    if op == "norm":
        m, k = case["m"], case["k"]
        # a few channels far larger than the others, as hidden states have them
        channel = torch.exp(normal(k))
        s["x"] = (normal(m, k) * channel).bfloat16()
        s["residual"] = (normal(m, k) * 3 * channel).bfloat16() if case["residual"] else None
        s["weight"] = (1 + 0.2 * normal(k)).bfloat16()
        s["eps"] = 1e-6
    elif op == "prefill":
        lens = _lens(case)
        hq, hkv, d, total = case["hq"], case["hkv"], case["d"], sum(lens)
        # q, k and v are column ranges of one projection's output
        qkv = normal(total, (hq + 2 * hkv) * d).bfloat16()
        qkv[:, :hq * d] *= 1.5
        s["q"] = qkv[:, :hq * d].view(total, hq, d)
        s["k"] = qkv[:, hq * d:(hq + hkv) * d].view(total, hkv, d)
        s["v"] = qkv[:, (hq + hkv) * d:].view(total, hkv, d)
        ends = [0]
        for n in lens:
            ends.append(ends[-1] + n)
        s["cu_seqlens"] = torch.tensor(ends, dtype=torch.int32, device=dev)
        s["plan"] = None
    elif op == "decode":
        lens = _lens(case)
        hq, hkv, d, page, batch = case["hq"], case["hkv"], case["d"], case["page"], case["batch"]
        need = [-(-n // page) for n in lens]
        width = max(1, max(need))
        pages = sum(need) + 7
        at = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
        starts = torch.tensor([sum(need[:i]) for i in range(batch)], device=dev)
        cols = torch.arange(width, device=dev)
        held = cols[None] < torch.tensor(need, device=dev)[:, None]
        s["block_table"] = torch.where(held, at[(starts[:, None] + cols[None]).clamp(max=pages - 1)], -1).to(torch.int32)
        s["page"] = page
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        # the per-tensor scales a calibration gives N(0, 1) rows; codes as the append writes them
        s["scales"] = torch.tensor([5.3 / 448, 5.1 / 448], device=dev)
        for i, name in enumerate(("k_cache", "v_cache")):
            cache = torch.empty(pages * page, hkv * d, dtype=torch.uint8, device=dev)
            step = max(1, (1 << 28) // (hkv * d))
            for r in range(0, pages * page, step):
                part = cache[r:r + step]
                part.copy_((normal(*part.shape) / s["scales"][i]).clamp_(-448, 448).to(E4M3).view(torch.uint8))
            s[name] = cache
        s["q"] = (normal(batch, hq, d) * 1.5).bfloat16()
    else:
        rows, vocab = case["rows"], case["vocab"]
        x = normal(rows, vocab).mul_(2.5)
        # most rows have a clear favourite, as a model's do
        best = torch.randint(0, vocab, (rows,), generator=g, device=dev)
        x[torch.arange(rows, device=dev), best] += 14 * torch.rand(rows, generator=g, device=dev)
        x[:, vocab - vocab // 100:] = -math.inf  # rows of the embedding that no token has
        s["logits"] = x.to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)
        other = torch.randint(0, vocab - vocab // 100, (rows,), generator=g, device=dev)
        tokens = torch.where(torch.rand(rows, generator=g, device=dev) < 0.6, best.clamp(max=vocab - vocab // 100 - 1), other)
        # one position in 32 is a prompt's or padding: it has no token
        tokens = torch.where(torch.rand(rows, generator=g, device=dev) < 1 / 32, -1, tokens)
        s["tokens"] = tokens.to(torch.int32)
        s["temperature"] = case["temperature"]
        if op == "logprob":
            s["topk"] = case["topk"]
        else:
            s["grad_lp"] = normal(rows)
            s["grad_entropy"] = 0.01 * normal(rows)
            # what the forward pass left for the backward one
            y = s["logits"].float()
            top = y.amax(1)
            y = (y - top[:, None]) / s["temperature"]
            e = torch.exp(y)
            total = e.sum(1)
            on = s["tokens"] >= 0
            ent = torch.log(total) - torch.where(e > 0, e * y, 0).sum(1) / total
            s["entropy"] = torch.where(on, ent, 0)
            s["stats"] = torch.where(on[:, None], torch.stack([top, torch.log(total)], 1), 0).contiguous()
    return s


# ------------------------------------------------------------------ the calls

def run(s):
    return {"norm": _run_norm, "prefill": _run_prefill, "decode": _run_decode, "logprob": _run_logprob,
            "logprob_grad": _run_logprob_grad}[s["case"]["op"]](s)


def _run_norm(s):
    ue8m0 = s["case"]["fmt"] == "ue8m0"
    if own:
        import fp8_w8a8_rollout_gb300 as fp8rl
        q, scale, h = fp8rl.rmsnorm_quant(s["x"], s["weight"], s["residual"], eps=s["eps"],
                                          fmt=fp8rl.SCALE_UE8M0 if ue8m0 else fp8rl.SCALE_FP32)
        return {"q": q.view(E4M3), "scale": scale.view(E8M0) if ue8m0 else scale, "h": h}
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + s["eps"]) * s["weight"].float()
    m, k = y.shape
    groups = -(-k // 128)
    y = torch.cat([y, y.new_zeros(m, groups * 128 - k)], 1).view(m, groups, 128)
    amax = y.abs().amax(2, keepdim=True)
    if ue8m0:
        # the smallest e with 448 * 2^e >= amax; 448 = 0.875 * 2^9
        f, e = torch.frexp(amax)
        e = torch.where(amax == 0, 0, (e - 9 + (f > 0.875)).clamp(-127, 127))
        q = torch.ldexp(y, -e)
        scale = (e + 127).to(torch.uint8).view(E8M0)
    else:
        scale = torch.where(amax == 0, 1, amax / 448)
        q = y / scale
    q = q.clamp(-448, 448).to(E4M3).view(m, groups * 128)[:, :k].contiguous()
    return {"q": q, "scale": scale.view(m, groups).t().contiguous(),
            "h": h.bfloat16() if s["residual"] is not None else None}


def _run_prefill(s):
    case = s["case"]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if own:
        import fp8_w8a8_rollout_gb300 as fp8rl
        if s["plan"] is None:  # one plan serves every layer of a step
            s["plan"] = fp8rl.attn_prefill_plan(s["cu_seqlens"], s["q"].shape[0], hq, hkv)
        out, lse = fp8rl.attn_prefill(s["q"], s["k"], s["v"], s["plan"])
        return {"out": out, "lse": lse}
    cu = s["cu_seqlens"].long()
    total, batch, most = s["q"].shape[0], case["batch"], case["most"]
    pos = torch.arange(most, device=cu.device)
    at = (cu[:-1, None] + pos).clamp(max=total - 1)
    q = s["q"].float()[at].view(batch, most, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(batch, hkv, -1, d)
    k = s["k"].float()[at].permute(0, 2, 3, 1)
    v = s["v"].float()[at].permute(0, 2, 1, 3)
    score = torch.matmul(q, k).view(batch, hkv, hq // hkv, most, most) * d ** -0.5
    score.masked_fill_(pos[None] > pos[:, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - top)
    denom = p.sum(-1, keepdim=True)
    out = torch.matmul(p.view(batch, hkv, -1, most), v).view(batch, hkv, hq // hkv, most, d) / denom
    lse = (top + torch.log(denom))[..., 0]
    valid = pos < (cu[1:] - cu[:-1])[:, None]
    out = out.permute(0, 3, 1, 2, 4).reshape(batch, most, hq, d)[valid]
    lse = lse.permute(0, 3, 1, 2).reshape(batch, most, hq)[valid]
    return {"out": out.bfloat16(), "lse": lse}


def _run_decode(s):
    case = s["case"]
    hq, hkv, d, batch, most, page = (case[n] for n in ("hq", "hkv", "d", "batch", "most", "page"))
    if own:
        import fp8_w8a8_rollout_gb300 as fp8rl
        if "workspace" not in s:
            s["workspace"] = fp8rl.attn_decode_workspace(hq, hkv, d)
        out, lse = fp8rl.attn_decode(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["lens"], s["scales"], page,
                                     workspace=s["workspace"])
        return {"out": out, "lse": lse}
    pos = torch.arange(most, device=s["q"].device)
    slots = (s["block_table"].long()[:, pos // page] * page + pos % page).clamp(min=0)
    valid = pos < s["lens"][:, None]
    k = s["k_cache"][slots].view(E4M3).float().view(batch, most, hkv, d) * s["scales"][0]
    v = s["v_cache"][slots].view(E4M3).float().view(batch, most, hkv, d) * s["scales"][1]
    v = v * valid[:, :, None, None]
    q = s["q"].float().view(batch, hkv, hq // hkv, d)
    score = torch.matmul(q, k.permute(0, 2, 3, 1)) * d ** -0.5
    score = score.masked_fill(~valid[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0, top)
    p = torch.exp(score - top)
    denom = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v.permute(0, 2, 1, 3)) / torch.where(denom == 0, 1, denom)
    return {"out": out.view(batch, hq, d).bfloat16(), "lse": (top + torch.log(denom)).view(batch, hq)}


def _run_logprob(s):
    logits, tokens, top = s["logits"], s["tokens"], s["topk"]
    if own:
        import fp8_w8a8_rollout_gb300 as fp8rl
        lp, entropy, stats, ids, top_lp = fp8rl.logprobs(logits, tokens, temperature=s["temperature"], topk=top)
        return {"lp": lp, "entropy": entropy, "stats": stats, "ids": ids, "top_lp": top_lp}
    x = logits.float()
    best = x.amax(1, keepdim=True)
    y = (x - best) / s["temperature"]
    e = torch.exp(y)
    total = e.sum(1, keepdim=True)
    on = tokens >= 0
    lp = torch.where(on, (y.gather(1, tokens.long().clamp(min=0)[:, None]) - torch.log(total))[:, 0], 0)
    entropy = torch.where(on, (torch.log(total) - torch.where(e > 0, e * y, 0).sum(1, keepdim=True) / total)[:, 0], 0)
    stats = torch.where(on[:, None], torch.cat([best, torch.log(total)], 1), 0)
    if not top:
        return {"lp": lp, "entropy": entropy, "stats": stats, "ids": None, "top_lp": None}
    # whole-number keys in the values' order, the lower index first among equals
    bits = x.view(torch.int32).long()
    key = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits) * (1 << 32) - torch.arange(x.shape[1], device=x.device)
    ids = torch.topk(key, top, dim=1).indices
    top_lp = y.gather(1, ids) - torch.log(total)
    return {"lp": lp, "entropy": entropy, "stats": stats, "ids": torch.where(on[:, None], ids, -1).to(torch.int32),
            "top_lp": torch.where(on[:, None], top_lp, 0)}


def _run_logprob_grad(s):
    logits, tokens, temperature = s["logits"], s["tokens"], s["temperature"]
    if own:
        import fp8_w8a8_rollout_gb300 as fp8rl
        return fp8rl.logprobs_backward(logits, tokens, s["stats"], s["entropy"], s["grad_lp"], s["grad_entropy"],
                                       temperature=temperature)
    # log p_j = (x_j - max) / T - log total
    lp = (logits.float() - s["stats"][:, :1]) / temperature - s["stats"][:, 1:]
    p = torch.exp(lp)
    lp = torch.where(p > 0, lp, 0)
    # d lp_t = [j = t] - p_j;  d H = -p_j (log p_j + H)
    grad = -p * (s["grad_lp"][:, None] + s["grad_entropy"][:, None] * (lp + s["entropy"][:, None]))
    grad.scatter_add_(1, tokens.long().clamp(min=0)[:, None], s["grad_lp"][:, None])
    return torch.where((tokens >= 0)[:, None], grad / temperature, 0).to(logits.dtype)


# ------------------------------------------------------------------ from the definition, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        h = s["x"].double() + (0 if s["residual"] is None else s["residual"].double())
        y = h / torch.sqrt(h.pow(2).sum(1, keepdim=True) / case["k"] + s["eps"]) * s["weight"].double()
        q, scales = torch.empty_like(y), []
        for c in range(0, case["k"], 128):
            a = y[:, c:c + 128].abs().max(1).values
            if case["fmt"] == "ue8m0":
                sc = torch.pow(2.0, torch.ceil(torch.log2(a / 448)).clamp(-127, 127))
            else:
                sc = a / 448
            sc = torch.where(a == 0, torch.ones_like(sc), sc)
            q[:, c:c + 128] = y[:, c:c + 128] / sc[:, None]
            scales.append(sc)
        return {"q": q, "scale": torch.stack(scales), "h": h if s["residual"] is not None else None}
    if op == "prefill":
        hq, hkv, d = case["hq"], case["hkv"], case["d"]
        out, lse = torch.empty(*s["q"].shape, dtype=torch.float64, device="cuda"), []
        start = 0
        for n in _lens(case):
            later = torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1)
            cols = []
            for h in range(hq):
                a = s["q"][start:start + n, h].double() @ s["k"][start:start + n, h // (hq // hkv)].double().T / math.sqrt(d)
                a[later] = -math.inf
                z = torch.logsumexp(a, 1)
                out[start:start + n, h] = torch.exp_(a - z[:, None]) @ s["v"][start:start + n, h // (hq // hkv)].double()
                cols.append(z)
            lse.append(torch.stack(cols, 1))
            start += n
        return {"out": out, "lse": torch.cat(lse)}
    if op == "decode":
        hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
        out = torch.zeros(case["batch"], hq, d, dtype=torch.float64, device="cuda")
        lse = torch.full((case["batch"], hq), -math.inf, dtype=torch.float64, device="cuda")
        for b, n in enumerate(_lens(case)):
            if n == 0:
                continue
            pages = s["block_table"][b, :-(-n // page)].long()
            rows = (pages[:, None] * page + torch.arange(page, device="cuda")).reshape(-1)[:n]
            k = s["k_cache"][rows].view(E4M3).double().view(n, hkv, d) * s["scales"][0].double()
            v = s["v_cache"][rows].view(E4M3).double().view(n, hkv, d) * s["scales"][1].double()
            q = s["q"][b].double().view(hkv, hq // hkv, d)
            a = torch.einsum("hgd,nhd->hgn", q, k) / math.sqrt(d)
            z = torch.logsumexp(a, 2)
            out[b] = torch.einsum("hgn,nhd->hgd", torch.exp(a - z[:, :, None]), v).reshape(hq, d)
            lse[b] = z.reshape(hq)
        return {"out": out, "lse": lse}
    rows = case["rows"]
    temperature = s["temperature"]
    got = {"lp": [], "entropy": [], "stats": [], "top_lp": []} if op == "logprob" else []
    step = max(1, (1 << 28) // case["vocab"])
    for r in range(0, rows, step):
        x = s["logits"][r:r + step].double() / temperature
        t = s["tokens"][r:r + step].long()
        on = t >= 0
        z = torch.logsumexp(x, 1, keepdim=True)
        lp = x - z
        p = torch.exp(lp)
        plogp = torch.where(p > 0, p * lp, torch.zeros_like(p))
        hh = -plogp.sum(1)
        pick = torch.nn.functional.one_hot(t.clamp(min=0), case["vocab"]).bool() & on[:, None]
        if op == "logprob":
            got["lp"].append(torch.where(pick, lp, torch.zeros_like(lp)).sum(1))
            got["entropy"].append(torch.where(on, hh, torch.zeros_like(hh)))
            best = x.max(1).values
            st = torch.stack([best * temperature, z[:, 0] - best], 1)
            got["stats"].append(torch.where(on[:, None], st, torch.zeros_like(st)))
            if case["topk"]:
                v = lp.sort(1, descending=True).values[:, :case["topk"]]
                got["top_lp"].append(torch.where(on[:, None], v, torch.zeros_like(v)))
            continue
        g, ge = s["grad_lp"][r:r + step].double()[:, None], s["grad_entropy"][r:r + step].double()[:, None]
        d = g * (pick.double() - p) - ge * (plogp + p * hh[:, None])
        got.append(torch.where(on[:, None], d / temperature, torch.zeros_like(d)))
    if op == "logprob":
        return {**{n: torch.cat(v) if v else None for n, v in got.items()}, "ids": None}
    return torch.cat(got)
