"""The token loop around a rollout's decoder, as cases to measure.

Between its linears and attentions a rollout rotates queries and keys by their
positions (``rotary``, also backwards, and ``rotary_kv_append`` joined with the
append to the E4M3 cache), draws the next token from the logits (``sample``), and
keeps the pages of the cache: room for new tokens (``kv_reserve``), a prompt's
pages shared by several answers (``kv_fork``), used pages moved together
(``kv_compact``).

``run`` computes each in its plain form (elementary torch operations in fp32, in
64 bits where a token is decided by a sum or an angle is far, one rounding at the
end), or, with ``own`` set, through the package.  Head counts, widths and
vocabularies are those the benchmark, the tests and ``perf/operators.py`` use.
"""
import math
import random

import torch

own = False

E4M3 = torch.float8_e4m3fn


# ------------------------------------------------------------------ the cases

def _sample(rows, vocab, dtype, temperature, top_k, top_p, min_p, mixed=False, **more):
    # mixed: every row has parameters of its own, up to these
    return {"op": "sample", "rows": rows, "vocab": vocab, "dtype": dtype, "temperature": temperature, "top_k": top_k,
            "top_p": top_p, "min_p": min_p, "mixed": mixed, **more}


def _rotary(op, tokens, hq, hkv, d, axes, far, interleaved=False, part=1.0, **more):
    # axes: 1 (text) or 3 (time, height, width); far: the largest position; part: of the head that is rotated
    return {"op": op, "tokens": tokens, "hq": hq, "hkv": hkv, "d": d, "axes": axes, "far": far, "interleaved": interleaved,
            "part": part, **more}


def _reserve(rows, least, most, new, width, page, caches, layout, prompts=False, **more):
    # rows of `least` to `most` tokens; each gets `new` more, or (prompts) up to `new`
    return {"op": "reserve", "rows": rows, "least": least, "most": most, "new": new, "width": width, "page": page, "caches": caches,
            "layout": layout, "prompts": prompts, **more}


def _fork(prompts, answers, least, most, width, page, caches, layout, **more):
    return {"op": "fork", "prompts": prompts, "answers": answers, "least": least, "most": most, "width": width, "page": page,
            "caches": caches, "layout": layout, **more}


def _compact(rows, least, most, spare, width, page, caches, layout, **more):
    # `spare`: free pages for one used page
    return {"op": "compact", "rows": rows, "least": least, "most": most, "spare": spare, "width": width, "page": page,
            "caches": caches, "layout": layout, **more}


def listed():
    return [
        # the answers of one decode step, requests of different parameters
        _sample(16, 151936, "bf16", 1.0, 50, 0.95, 0.05, True, name="sample 16 rows mixed"),
        # a rollout batch drawn as the policy says it, nothing cut off
        _sample(1024, 151936, "bf16", 1.0, 0, 1.0, 0.0, name="sample 1024 rows"),
        # evaluation: nucleus sampling of fp32 logits, an odd vocabulary
        _sample(61, 32001, "fp32", 0.6, 0, 0.95, 0.0, name="sample 61 rows top-p"),
        # the packed prompts of a rollout step, one layer
        _rotary("rotary", 8192, 32, 8, 128, 1, 131071, name="rotary 8192 tokens"),
        # backward pass of a batch with images: three axes, odd length
        _rotary("rotary_grad", 1771, 32, 4, 128, 3, 4000, name="rotary grad 1771 tokens three axes"),
        # one decode step's tokens: the call is launch latency
        _rotary("rotary_append", 16, 32, 8, 128, 1, 20000, name="rotary append 16 tokens"),
        # prompts that join a running rollout: the scales are there
        _rotary("rotary_append", 4001, 32, 8, 128, 1, 4000, name="rotary append 4001 tokens"),
        # one decode step's book-keeping of a rollout batch: a page for one row in 16
        _reserve(256, 0, 4095, 1, 1024, 16, 2, 3, name="reserve 256 rows"),
        # one group of answers to one prompt begins: few pages, few layers
        _fork(1, 16, 500, 500, 512, 16, 8, 5, name="fork 1 prompt to 16"),
        # a rollout step begins: 16 answers to each prompt, the shared last page copied in all 36 layers
        _fork(32, 16, 100, 400, 1024, 16, 72, 7, name="fork 32 prompts to 16"),
        # one layer's cache, between two groups of answers
        _compact(8, 100, 300, 0.5, 1024, 16, 2, 9, name="compact 8 rows"),
        # the cache of 36 layers made small before the weights change
        _compact(64, 100, 1000, 0.5, 1024, 16, 72, 11, name="compact 64 rows"),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sample", "sample", "rotary", "rotary_grad", "rotary_append", "reserve", "fork", "compact"])
    if op == "sample":
        vocab = rng.choice([rng.choice([32000, 50257, 128256, 151936]), _log_uniform(rng, 100, 150000)])
        rows = min(_log_uniform(rng, 1, 1.5e8 / vocab), 4096)
        mixed = rng.random() < 0.3
        return _sample(rows, vocab, rng.choice(["bf16", "fp32"]), rng.choice([1.0, 0.6, 1.3]), rng.choice([0, 0, 1, 20, 50, 300]),
                       rng.choice([1.0, 1.0, 0.95, 0.9, 0.5]), rng.choice([0.0, 0.0, 0.05, 0.1]), mixed)
    if op.startswith("rotary"):
        hq, hkv = rng.choice([(32, 8), (32, 4), (16, 16), (12, 2), (24, 8), (40, 4)])
        return _rotary(op, _log_uniform(rng, 1, 300000 / (hq + hkv)), hq, hkv, rng.choice([128, 128, 64]), rng.choice([1, 1, 3]),
                       _log_uniform(rng, 100, 1000000), rng.random() < 0.25, rng.choice([1.0, 1.0, 0.5]))
    width, page = rng.choice([512, 1024, 256, 2048]), rng.choice([16, 16, 32, 64])
    layers, layout = _log_uniform(rng, 1, 36), rng.randrange(1 << 20)
    if op == "reserve":
        prompts = rng.random() < 0.5
        rows = _log_uniform(rng, 1, 512)
        return _reserve(rows, 0, _log_uniform(rng, 16, 4096), _log_uniform(rng, 2, min(2048, 40000 // rows + 2)) if prompts else 1,
                        width, page, 2 * min(layers, 4), layout, prompts)
    if op == "fork":
        most = _log_uniform(rng, 10, 600)
        return _fork(_log_uniform(rng, 1, 24), rng.choice([2, 4, 8, 16]), max(1, most // 3), most, width, page, 2 * layers, layout)
    most = _log_uniform(rng, 20, 1000)
    rows = _log_uniform(rng, 1, max(1, 24e6 / (most * layers * width / 16)))
    return _compact(min(rows, 256), most // 4, most, rng.choice([0.1, 0.5, 2.0]), width, page, 2 * layers, layout)


# ------------------------------------------------------------------ page book-keeping

def _blocks(n, page):
    return -(-n // page)


def _layout(case):
    """A cache in use, by the case alone: (pages of every row, lens, tokens each row asks for, pages in all)."""
    r = random.Random(case["layout"] * 1000003 + case["page"])
    page = case["page"]
    if case["op"] == "fork":
        lens = [r.randint(case["least"], case["most"]) for _ in range(case["prompts"])]
        held = sum(_blocks(n, page) for n in lens)
        pages = 2 * held + case["prompts"] * case["answers"] + 8
        new = [1] * (case["prompts"] * case["answers"])
    else:
        lens = [r.randint(case["least"], case["most"]) for _ in range(case["rows"])]
        held = sum(_blocks(n, page) for n in lens)
        if case["op"] == "reserve":
            new = [r.randint(1, case["new"]) if case["prompts"] else case["new"] for _ in lens]
            if case["prompts"]:  # prompts come to rows that are empty
                lens = [0 if r.random() < 0.7 else n for n in lens]
            elif len(new) > 3:  # answers that have ended ask for nothing
                new[r.randrange(len(new))] = 0
            held = sum(_blocks(n, page) for n in lens)
            pages = 2 * held + sum(_blocks(n, page) + 1 for n in new) + 8
        else:
            new = [0] * len(lens)
            pages = held + int(held * case["spare"]) + 1
    at = list(range(pages))
    r.shuffle(at)
    rows = []
    for n in lens:
        rows.append([at.pop() for _ in range(_blocks(n, page))])
    return rows, lens, new, pages


def _moves(rows):
    """Pages that a compaction moves."""
    used = sorted(p for row in rows for p in row)
    return sum(p >= len(used) for p in used)


def work(case):
    op = case["op"]
    if op == "sample":
        n = case["rows"] * case["vocab"]
        return {"bytes": n * (2 if case["dtype"] == "bf16" else 4) + case["rows"] * (24 + (16 if case["mixed"] else 0)), "flops": 5 * n}
    if op.startswith("rotary"):
        t, hq, hkv, d = case["tokens"], case["hq"], case["hkv"], case["d"]
        size = t * 4 * case["axes"]
        if op == "rotary_append":  # q, k and v in; q, the codes of k and v out
            return {"bytes": size + t * (4 * hq * d + 6 * hkv * d + 4), "flops": 3 * t * (hq + hkv) * d + 2 * t * hkv * d}
        return {"bytes": size + 4 * t * (hq + hkv) * d, "flops": 3 * t * (hq + hkv) * d}
    rows, lens, new, pages = _layout(case)
    page, line = case["page"], case["width"] * case["caches"]
    if op == "reserve":
        added = sum(_blocks(n + k, page) - _blocks(n, page) for n, k in zip(lens, new))
        return {"bytes": 4 * pages + 8 * added + 12 * len(lens) + 4 * sum(new), "flops": pages}
    if op == "fork":
        tails = [n % page for n in lens]
        copied = case["answers"] * sum(tails)
        entries = case["answers"] * sum(len(r) for r in rows)
        return {"bytes": 2 * copied * line + 4 * pages + 8 * entries + 16 * len(new), "flops": pages + entries}
    moved = _moves(rows)
    return {"bytes": 2 * moved * page * line + 8 * pages + 8 * moved, "flops": pages}


# ------------------------------------------------------------------ inputs

def _inverse_frequencies(case):
    n = int(case["d"] * case["part"]) // 2
    return [10000.0 ** (-i / n) for i in range(n)]


def _sections(case):
    """Pairs of each axis: a quarter in time, the rest in height and width."""
    n = len(_inverse_frequencies(case))
    if case["axes"] == 1:
        return [n]
    a = (n - n // 4) // 2
    return [n - 2 * a, a, a]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(dev)
    g.manual_seed(seed)
    op = case["op"]
    s = {"case": case}

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32)

    def uniform(*shape, dtype=torch.float32):
        return torch.rand(*shape, generator=g, device=dev, dtype=dtype)

    def integers(low, high, shape, dtype=torch.int32):
        return torch.randint(low, high, shape, generator=g, device=dev, dtype=dtype)

    if op == "sample":
        rows, vocab = case["rows"], case["vocab"]
        x = normal(rows, vocab).mul_(1.5)
        # most rows are sure of a few tokens, some of none
        few = min(40, vocab)
        at = integers(0, vocab, (rows, few), torch.int64)
        sure = 10 + 10 * torch.sqrt(uniform(rows, 1))
        x.scatter_add_(1, at, sure * (1 - torch.arange(few, device=dev) / 40) ** 0.5 * uniform(rows, few) ** 0.3)
        x[:, vocab - vocab // 100:] = -math.inf  # rows of the embedding that no token has
        s["logits"] = x.to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)
        s["uniform"] = uniform(rows, dtype=torch.float64)
        if rows > 8:  # one row in 32 has no request
            s["uniform"][uniform(rows) < 1 / 32] = -1
        if case["mixed"]:
            pick = integers(0, 4, (4, rows))
            s["temperature"] = torch.where(pick[0] == 0, 1.0, case["temperature"] * (0.5 + uniform(rows)))
            s["top_k"] = torch.where(pick[1] == 0, 0, integers(0, case["top_k"] + 1, (rows,))).to(torch.int32)
            s["top_p"] = torch.where(pick[2] == 0, 1.0, case["top_p"] * (0.7 + 0.3 * uniform(rows)))
            s["min_p"] = torch.where(pick[3] == 0, 0.0, case["min_p"] * uniform(rows))
        else:
            s.update({n: case[n] for n in ("temperature", "top_k", "top_p", "min_p")})
    elif op.startswith("rotary"):
        t, hq, hkv, d = case["tokens"], case["hq"], case["hkv"], case["d"]
        # q, k and v are column ranges of one projection's output
        qkv = normal(t, (hq + 2 * hkv) * d).bfloat16()
        s["q"] = qkv[:, :hq * d].view(t, hq, d)
        s["k"] = qkv[:, hq * d:(hq + hkv) * d].view(t, hkv, d)
        s["v"] = qkv[:, (hq + hkv) * d:].view(t, hkv, d)
        if op == "rotary_grad":  # the attention's gradients stand alone
            s["q"], s["k"] = s["q"].contiguous(), s["k"].contiguous()
        s["positions"] = integers(0, case["far"] + 1, (case["axes"], t))
        if op == "rotary_append":
            slots = 2 * t + 64
            s["slots"] = torch.randperm(slots, generator=g, device=dev)[:t].to(torch.int32)
            if t > 8:  # padding
                s["slots"][uniform(t) < 1 / 32] = -1
            # the scales a calibration gives N(0, 1) rows; the last ones a little small, so that some saturate
            s["scales"] = torch.tensor([5.3 / 448, 4.1 / 448], device=dev)
            s["k_cache"], s["v_cache"] = (integers(0, 120, (slots, hkv * d), torch.uint8) for _ in range(2))
        s["frequencies"] = None  # laid out once, as a model's weights are
    else:
        rows, lens, new, pages = _layout(case)
        page, width = case["page"], case["width"]
        # the book-keeping in one piece, so that every pass starts from the same
        n_rows = len(new) if op != "fork" else len(lens)
        cols = max(_blocks(n + k, page) for n, k in zip(lens, new)) if op != "fork" else _blocks(max(lens) + 1, page)
        cols = max(cols, 1) + 1
        table = torch.tensor([r + [-1] * (cols - len(r)) for r in rows], dtype=torch.int32)
        refs = torch.zeros(pages, dtype=torch.int32)
        for r in rows:
            refs[torch.tensor(r, dtype=torch.long)] = 1
        s["saved"] = torch.cat([table.flatten(), refs, torch.tensor(lens, dtype=torch.int32)]).to(dev)
        s["live"] = torch.empty_like(s["saved"])
        s["table"] = s["live"][:n_rows * cols].view(n_rows, cols)
        s["refs"] = s["live"][n_rows * cols:n_rows * cols + pages]
        s["lens"] = s["live"][n_rows * cols + pages:]
        s["page"] = page
        s["pool"] = integers(0, 120, (case["caches"], pages * page, width), torch.uint8)  # K and V of every layer
        s["caches"] = list(s["pool"])
        s["handle"] = None  # the list of the layers' caches, made once
        s["count"] = torch.tensor(new, dtype=torch.int32, device=dev)
        if op == "reserve" and case["prompts"]:
            ends = [0]
            for k in new:
                ends.append(ends[-1] + k)
            s["cu_seqlens"], s["total"] = torch.tensor(ends, dtype=torch.int32, device=dev), ends[-1]
        if op == "fork":
            s["parent"] = torch.arange(len(lens), device=dev, dtype=torch.int32).repeat_interleave(case["answers"])
    return s


# ------------------------------------------------------------------ the calls

def run(s):
    return {"sample": _run_sample, "rotary": _run_rotary, "rotary_grad": _run_rotary, "rotary_append": _run_rotary_append,
            "reserve": _run_reserve, "fork": _run_fork, "compact": _run_compact}[s["case"]["op"]](s)


def _column(v, like):
    """A parameter of every row as a column in 64 bits."""
    if isinstance(v, torch.Tensor):
        return v.double()[:, None]
    # (the call takes it as an fp32 number)
    return torch.full((like.shape[0], 1), v, dtype=torch.float32, device=like.device).double()


def _run_sample(s):
    logits, u = s["logits"], s["uniform"]
    if own:
        import fp8_w8a8_rollout_gb300 as fp8rl
        token, lp, lp_kept, kept = fp8rl.sample(logits, u, s["temperature"], s["top_k"], s["top_p"], s["min_p"])
        return {"token": token, "lp": lp, "lp_kept": lp_kept, "kept": kept}
    rows, vocab = logits.shape
    temperature, top_p, min_p = (_column(s[n], logits) for n in ("temperature", "top_p", "min_p"))
    x = logits.float() + 0.0  # -0 counts as 0
    best = x.amax(1, keepdim=True)
    y = (x.double() - best.double()) / temperature
    w = torch.where(y > -100 * math.log(2), torch.exp(y), 0)
    total = w.sum(1, keepdim=True)
    finite = (x > -math.inf).sum(1, keepdim=True)
    top_k = s["top_k"]
    if isinstance(top_k, torch.Tensor) or top_k > 0 or isinstance(s["top_p"], torch.Tensor) or s["top_p"] < 1 or \
            isinstance(s["min_p"], torch.Tensor) or s["min_p"] > 0:
        # most likely first, equal ones by the lower index
        order = torch.sort(x, dim=1, descending=True, stable=True).indices
        mass = torch.cumsum(w.gather(1, order), 1)
        k = torch.where(_column(top_k, logits).long() > 0, _column(top_k, logits).long(), vocab)
        n = torch.minimum(k, finite)
        all_k = mass.gather(1, (n - 1).clamp(min=0))
        n_p = (mass < top_p * all_k).sum(1, keepdim=True) + 1
        n = torch.where(top_p < 1, torch.minimum(n, n_p), n)
        border = best.double() + temperature * torch.log(min_p)
        n = torch.minimum(n, (x.double() >= border).sum(1, keepdim=True))
        place = torch.empty_like(order).scatter_(1, order, torch.arange(vocab, device=x.device).expand(rows, vocab))
        w = torch.where(place < n, w, 0)
    else:
        n = finite
    cum = torch.cumsum(w, 1)
    mass = cum[:, -1:]
    token = (cum <= u[:, None] * mass).sum(1, keepdim=True)
    last = vocab - 1 - (w > 0).flip(1).int().argmax(1, keepdim=True)
    token = torch.minimum(token, last)
    on = (u >= 0) & (u < 1)
    yt = y.gather(1, token)
    return {"token": torch.where(on, token[:, 0], -1).to(torch.int32),
            "lp": torch.where(on, (yt - torch.log(total))[:, 0], 0).float(),
            "lp_kept": torch.where(on, (yt - torch.log(mass))[:, 0], 0).float(),
            "kept": torch.where(on, n[:, 0], 0).to(torch.int32)}


def _frequencies(s):
    """What a model's rotary positions need, kept with it."""
    if s["frequencies"] is None:
        case = s["case"]
        if own:
            import fp8_w8a8_rollout_gb300 as fp8rl
            s["frequencies"] = fp8rl.rotary_freqs(int(case["d"] * case["part"]), 10000.0, _sections(case), device="cuda")
        else:
            axis = [a for a, n in enumerate(_sections(case)) for _ in range(n)]
            s["frequencies"] = (torch.tensor(_inverse_frequencies(case), dtype=torch.float64, device="cuda"),
                                torch.tensor(axis, device="cuda"))
    return s["frequencies"]


def _rotated(x, positions, frequencies, interleaved, inverse):
    """[tokens, heads, d] in fp32."""
    inv, axis = frequencies
    angle = positions.double()[axis].t() * inv  # [tokens, pairs]
    c, sn = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    if inverse:
        sn = -sn
    n = inv.numel()
    y = x.float().clone()
    at = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    a, b = x[..., at[0]].float(), x[..., at[1]].float()
    y[..., at[0]] = a * c - b * sn
    y[..., at[1]] = a * sn + b * c
    return y


def _run_rotary(s):
    case, f = s["case"], _frequencies(s)
    back = case["op"] == "rotary_grad"
    if own:
        import fp8_w8a8_rollout_gb300 as fp8rl
        q, k = fp8rl.rotary(s["q"], s["k"], s["positions"], f, interleaved=case["interleaved"], inverse=back)
        return {"q": q, "k": k}
    return {n: _rotated(s[n], s["positions"], f, case["interleaved"], back).bfloat16() for n in ("q", "k")}


def _run_rotary_append(s):
    case, f = s["case"], _frequencies(s)
    kc, vc = s["k_cache"], s["v_cache"]
    if own:
        import fp8_w8a8_rollout_gb300 as fp8rl
        q, _ = fp8rl.rotary_kv_append(s["q"], s["k"], s["v"], s["positions"], f, s["slots"], kc, vc, s["scales"],
                                      interleaved=case["interleaved"])
    else:
        q = _rotated(s["q"], s["positions"], f, case["interleaved"], False).bfloat16()
        k = _rotated(s["k"], s["positions"], f, case["interleaved"], False)
        on = s["slots"] >= 0
        at = s["slots"].long()[on]
        for cache, x, scale in ((kc, k, s["scales"][0]), (vc, s["v"].float(), s["scales"][1])):
            cache[at] = (x[on].flatten(1) / scale).clamp(-448, 448).to(E4M3).view(torch.uint8)
    return {"q": q, "k_cache": kc.view(E4M3), "v_cache": vc.view(E4M3)}


def _handle(s):
    if s["handle"] is None:
        import fp8_w8a8_rollout_gb300 as fp8rl
        s["handle"] = fp8rl.KvCaches(s["caches"])
    return s["handle"]


def _contents(s):
    return s["pool"].view(E4M3)


def _plain_reserve(table, lens, refs, count, page, caches):
    """Room for count[r] more tokens in row r: (slots [rows, most], info); the book-keeping in place."""
    rows, cols = table.shape
    pages = refs.numel()
    r = torch.arange(rows, device=table.device)
    lens64, count64 = lens.long(), count.long()
    held = -(-lens64 // page)
    last = table[r, (held - 1).clamp(min=0)].long().clamp(min=0)
    tail = lens64 % page
    shared = (tail > 0) & (count64 > 0) & (refs[last] > 1)
    after = -(-(lens64 + count64) // page)
    fits = after <= cols
    need = torch.where(fits, after - held + shared, 0)
    first = torch.cumsum(need, 0) - need
    free = torch.argsort((refs != 0).to(torch.uint8), stable=True)  # the free pages, lowest first
    n_free = (refs == 0).sum()
    served = fits & ((need == 0) | (first + need <= n_free))
    refs.scatter_add_(0, last, -(shared & served).to(torch.int32))
    # a shared last page is copied
    fresh = free[first.clamp(max=pages - 1)]
    copied = shared & served
    slot = torch.arange(page, device=table.device)
    moved = copied[:, None] & (slot < tail[:, None])
    src = (last[:, None] * page + slot)[moved]
    dst = (fresh[:, None] * page + slot)[moved]
    for c in caches:
        c[dst] = c[src]
    at_last = (held - 1).clamp(min=0)
    table[r, at_last] = torch.where(copied, fresh.to(torch.int32), table[r, at_last])
    col = torch.arange(cols, device=table.device)
    added = served[:, None] & (col >= held[:, None]) & (col < after[:, None])
    at = (first + shared)[:, None] + col - held[:, None]
    given = free[at.clamp(0, pages - 1)].to(torch.int32)
    table.copy_(torch.where(added, given, table))
    taken = torch.cat([given[added].long(), fresh[copied]])
    refs[taken] = 1
    grown = torch.where(served, count64, 0)
    lens.copy_((lens64 + grown).to(torch.int32))
    info = torch.stack([(refs == 0).sum(), (~served).sum()]).to(torch.int32)
    return grown, lens64, info


def _plain_slots(table, before, grown, page, row, i):
    """The slot of new token i of its row, -1 where the row did not get it."""
    pos = before[row] + i
    slot = table[row, (pos // page).clamp(max=table.shape[1] - 1)].long() * page + pos % page
    return torch.where(i < grown[row], slot, -1).to(torch.int32)


def _run_reserve(s):
    case = s["case"]
    s["live"].copy_(s["saved"])
    table, lens, refs, page = s["table"], s["lens"], s["refs"], s["page"]
    if own:
        import fp8_w8a8_rollout_gb300 as fp8rl
        if case["prompts"]:
            slots, info = fp8rl.kv_reserve(table, lens, refs, page, _handle(s), cu_seqlens=s["cu_seqlens"], total_tokens=s["total"])
        else:
            slots, info = fp8rl.kv_reserve(table, lens, refs, page, _handle(s), count=s["count"])
    else:
        grown, before, info = _plain_reserve(table, lens, refs, s["count"], page, s["caches"])
        if case["prompts"]:
            token = torch.arange(s["total"], device=table.device)
            row = torch.searchsorted(s["cu_seqlens"][1:].long(), token, right=True)
            i = token - s["cu_seqlens"].long()[row]
        else:
            row = torch.arange(table.shape[0], device=table.device)
            i = torch.zeros_like(row)
        slots = _plain_slots(table, before, grown, page, row, i)
    return {"slots": slots, "info": info, "table": table, "lens": lens, "refs": refs, "caches": _contents(s)}


def _run_fork(s):
    s["live"].copy_(s["saved"])
    table, lens, refs, page, parent, count = s["table"], s["lens"], s["refs"], s["page"], s["parent"], s["count"]
    if own:
        import fp8_w8a8_rollout_gb300 as fp8rl
        table, lens = fp8rl.kv_fork(table, lens, refs, parent, page)
        # the answers' first tokens
        slots, info = fp8rl.kv_reserve(table, lens, refs, page, _handle(s), count=count)
    else:
        cols = torch.arange(table.shape[1], device=table.device)

        def holds(t, n):
            return cols < (-(-n.long() // page))[:, None]

        def add(t, n, by):
            on = holds(t, n)
            refs.scatter_add_(0, t.long().clamp(min=0).flatten(), (on * by).to(torch.int32).flatten())

        add(table, lens, -1)
        on = parent >= 0
        p = parent.long().clamp(min=0)
        new_lens = torch.where(on, lens[p], 0)
        new_table = torch.where(holds(table[p], new_lens), table[p], -1)
        add(new_table, new_lens, 1)
        table, lens = new_table, new_lens
        grown, before, info = _plain_reserve(table, lens, refs, count, page, s["caches"])
        row = torch.arange(table.shape[0], device=table.device)
        slots = _plain_slots(table, before, grown, page, row, torch.zeros_like(row))
    return {"slots": slots, "info": info, "table": table, "lens": lens, "refs": refs, "caches": _contents(s)}


def _run_compact(s):
    s["live"].copy_(s["saved"])
    table, lens, refs, page = s["table"], s["lens"], s["refs"], s["page"]
    if own:
        import fp8_w8a8_rollout_gb300 as fp8rl
        used = fp8rl.kv_compact(table, lens, refs, page, _handle(s))
    else:
        number = torch.arange(refs.numel(), device=table.device)
        taken = refs > 0
        n = taken.sum()
        src = (taken & (number >= n)).nonzero()[:, 0]
        dst = (~taken & (number < n)).nonzero()[:, 0]
        for c in s["caches"]:
            pages = c.view(refs.numel(), -1)
            pages[dst] = pages[src]
        to = number.to(torch.int32)
        to[src] = dst.to(torch.int32)
        refs[dst] = refs[src]
        refs[src] = 0
        on = torch.arange(table.shape[1], device=table.device) < (-(-lens.long() // page))[:, None]
        table.copy_(torch.where(on, to[table.long().clamp(min=0)], table))
        used = n.to(torch.int32).view(1)
    return {"used": used, "table": table, "lens": lens, "refs": refs, "caches": _contents(s)}


# ------------------------------------------------------------------ from the definition, in 64 bits

def exact(case, seed):
    op = case["op"]
    if op in ("reserve", "fork", "compact"):
        return None  # whole numbers and copied bytes
    s = prepare(case, seed)
    if op == "sample":
        rows = case["rows"]
        param = {n: s[n].tolist() if isinstance(s[n], torch.Tensor) else [s[n]] * rows for n in ("temperature", "top_k", "top_p", "min_p")}
        us = s["uniform"].tolist()
        f32 = lambda v: torch.tensor(v, dtype=torch.float32).item()
        lp, lp_kept = [], []
        zero = torch.zeros((), dtype=torch.float64, device="cuda")
        for r in range(rows):
            if not 0 <= us[r] < 1:
                lp.append(zero)
                lp_kept.append(zero)
                continue
            x = s["logits"][r].double()
            t, k, p, q = f32(param["temperature"][r]), param["top_k"][r], f32(param["top_p"][r]), f32(param["min_p"][r])
            logp = x / t - torch.logsumexp(x / t, 0)
            prob = torch.exp(logp)
            by = torch.sort(x, descending=True, stable=True)
            ids = by.indices[:int((x > -math.inf).sum())]
            if k > 0:
                ids = ids[:k]
            if p < 1:
                c = torch.cumsum(prob[ids], 0)
                ids = ids[:int((c < p * c[-1]).sum()) + 1]
            if q > 0:
                ids = ids[x[ids] >= by.values[0] + t * math.log(q)]
            ids = torch.sort(ids).values
            c = torch.cumsum(prob[ids], 0)
            at = ids[torch.clamp((c <= us[r] * c[-1]).sum(), max=len(ids) - 1)]
            lp.append(logp[at])
            lp_kept.append(-torch.log(c[-1] / prob[at]))
        return {"token": None, "lp": torch.stack(lp), "lp_kept": torch.stack(lp_kept), "kept": None}
    inv = _inverse_frequencies(case)
    pos = s["positions"].double()
    axis = [a for a, n in enumerate(_sections(case)) for _ in range(n)]
    sign = -1.0 if op == "rotary_grad" else 1.0
    out = {}
    for name in ("q", "k"):
        y = s[name].double()
        for i, f in enumerate(inv):
            at = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + len(inv))
            turn = torch.polar(torch.ones_like(pos[0]), sign * pos[axis[i]] * f)[:, None]
            z = torch.complex(s[name][..., at[0]].double(), s[name][..., at[1]].double()) * turn
            y[..., at[0]], y[..., at[1]] = z.real, z.imag
        out[name] = y
    if op != "rotary_append":
        return out
    caches = {}
    for name, x, scale in (("k_cache", out["k"], s["scales"][0]), ("v_cache", s["v"].double(), s["scales"][1])):
        values = s[name].view(E4M3).double()
        x = (x.flatten(1) / scale.double()).clamp(-448, 448)
        for t, slot in enumerate(s["slots"].tolist()):
            if slot >= 0:
                values[slot] = x[t]
        caches[name] = values
    return {"q": out["q"], **caches}
