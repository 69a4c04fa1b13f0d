"""One step of FP8 rollout RL on a small random decoder, with every stage on the
library's kernels.

    python examples/rollout_step.py [--layers 4] [--prompts 8] [--answers 4] [--new-tokens 32]

1. weight sync: the bf16 weights are quantised to E4M3 (128x128 blocks);
2. prefill of packed prompts: norm with E4M3 output, qkv GEMM, rotary positions,
   causal attention over the packed prompts, KV calibration and append into the
   paged E4M3 cache, output projection, fused gate-up, down projection;
3. several answers to each prompt: the cache's rows are forked, the prompts' pages
   shared (the last one copied by the answers that write to it);
4. decode, a token per answer and step: room in the cache, the same layers with
   the rotation and the append in one call and attention over the E4M3 cache, then
   a token drawn from the logits; answers that end give their pages back;
5. scoring by the training policy: the bf16 weights in torch matmuls, the same
   packed attention, log probabilities of the sampled tokens;
6. truncated importance sampling weights and the mismatch KL, and the gradient
   of the weighted loss with respect to the trainer's logits.

The decoder has the usual parts (RMS norms, grouped query heads, rotary
positions, SwiGLU); the embedding lookup is plain torch.
"""
from __future__ import annotations

import argparse
import dataclasses
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_w8a8_rollout_gb300 as fp8rl  # noqa: E402


@dataclasses.dataclass
class Config:
    layers: int = 4
    hidden: int = 1024
    q_heads: int = 16
    kv_heads: int = 2
    head_dim: int = 128
    inter: int = 2048
    vocab: int = 8192
    page: int = 16
    eps: float = 1e-6

    @property
    def qkv_dim(self):
        return (self.q_heads + 2 * self.kv_heads) * self.head_dim


def make_weights(cfg: Config, seed: int = 0, device="cuda"):
    g = torch.Generator(device).manual_seed(seed)

    def w(n, k):
        return (torch.randn(n, k, generator=g, device=device) * k ** -0.5).bfloat16()

    layers = [{"norm1": torch.ones(cfg.hidden, device=device).bfloat16(), "qkv": w(cfg.qkv_dim, cfg.hidden),
               "o": w(cfg.hidden, cfg.q_heads * cfg.head_dim), "norm2": torch.ones(cfg.hidden, device=device).bfloat16(),
               "gate": w(cfg.inter, cfg.hidden), "up": w(cfg.inter, cfg.hidden), "down": w(cfg.hidden, cfg.inter)}
              for _ in range(cfg.layers)]
    return {"layers": layers, "embed": torch.randn(cfg.vocab, cfg.hidden, generator=g, device=device).bfloat16(),
            "norm": torch.ones(cfg.hidden, device=device).bfloat16(), "head": w(cfg.vocab, cfg.hidden) * 4,
            "rotary": fp8rl.rotary_freqs(cfg.head_dim, device=device)}


def weight_sync(cfg: Config, weights):
    """The E4M3 weights of a step's rollout: (codes, scales) per linear."""
    out = []
    for lw in weights["layers"]:
        out.append({n: fp8rl.quant_weight(lw[n]) for n in ("qkv", "o", "down")} |
                   {"gate_up": fp8rl.quant_gate_up_interleaved(lw["gate"], lw["up"])})
    return {"layers": out, "head": fp8rl.quant_weight(weights["head"])}


class Cache:
    """The paged E4M3 KV cache of a batch: per layer K, V and their scales, and the
    pages' book-keeping (table, lens, refs), which all layers share."""

    def __init__(self, cfg: Config, batch: int, max_len: int, answers: int = 1, device="cuda"):
        blocks = -(-max_len // cfg.page)
        pages = batch * answers * blocks + batch * blocks  # (the prompts' own until the answers have theirs)
        self.page = cfg.page
        self.k = [torch.zeros(pages * cfg.page, cfg.kv_heads * cfg.head_dim, dtype=torch.uint8, device=device) for _ in range(cfg.layers)]
        self.v = [torch.zeros_like(k) for k in self.k]
        self.scales = [None] * cfg.layers
        self.all = fp8rl.KvCaches(self.k + self.v)
        self.table = torch.full((batch, blocks), -1, dtype=torch.int32, device=device)
        self.lens = torch.zeros(batch, dtype=torch.int32, device=device)
        self.refs = torch.zeros(pages, dtype=torch.int32, device=device)
        self.workspace = fp8rl.attn_decode_workspace(cfg.q_heads, cfg.kv_heads, cfg.head_dim)

    def reserve(self, **what) -> torch.Tensor:
        """Cache rows for new tokens (prompts: cu_seqlens and total_tokens; decode: count)."""
        return fp8rl.kv_reserve(self.table, self.lens, self.refs, self.page, self.all, **what)[0]

    def select(self, parent: torch.Tensor, in_place: bool = False) -> None:
        """Row i goes on from what row parent[i] holds; -1 gives its pages back."""
        out = (self.table, self.lens) if in_place else None
        self.table, self.lens = fp8rl.kv_fork(self.table, self.lens, self.refs, parent, self.page, out=out)

    def compact(self) -> int:
        """The pages in use, moved to the front: the rest of the caches is free for other things."""
        return int(fp8rl.kv_compact(self.table, self.lens, self.refs, self.page, self.all))


def rollout_layers(cfg: Config, weights, q8, x, attend):
    """The FP8 decoder stack on x [tokens, hidden]; attend(layer, q, k, v), the
    heads before their rotation, returns [tokens, q_heads * head_dim].  Returns
    the E4M3 final norm."""
    h, delta = x, None  # the residual stream, and what the last branch adds to it
    for i, (lw, qw) in enumerate(zip(weights["layers"], q8["layers"])):
        if delta is None:
            xq, sx, _ = fp8rl.rmsnorm_quant(h, lw["norm1"], eps=cfg.eps)
        else:
            xq, sx, h = fp8rl.rmsnorm_quant(delta, lw["norm1"], h, eps=cfg.eps)
        qkv = fp8rl.gemm(xq, sx, *qw["qkv"]).view(-1, cfg.q_heads + 2 * cfg.kv_heads, cfg.head_dim)
        nq, nk = cfg.q_heads, cfg.q_heads + cfg.kv_heads
        o, _, _ = fp8rl.gemm_act_quant(attend(i, qkv[:, :nq], qkv[:, nq:nk], qkv[:, nk:]), *qw["o"])
        xq, sx, h = fp8rl.rmsnorm_quant(o, lw["norm2"], h, eps=cfg.eps)
        hq, hs = fp8rl.gemm_swiglu_quant(xq, sx, *qw["gate_up"])
        delta = fp8rl.gemm(hq, hs, *qw["down"])
    xq, sx, _ = fp8rl.rmsnorm_quant(delta, weights["norm"], h, eps=cfg.eps)
    return xq, sx


def prefill(cfg: Config, weights, q8, tokens, cu, seq, pos, cache: Cache):
    """Fills the cache with packed prompts; logits bf16 of each prompt's last token."""
    plan = fp8rl.attn_prefill_plan(cu, tokens.numel(), cfg.q_heads, cfg.kv_heads)
    slots, at = cache.reserve(cu_seqlens=cu, total_tokens=tokens.numel()), pos.to(torch.int32)

    def attend(i, q, k, v):
        q, k = fp8rl.rotary(q, k, at, weights["rotary"])
        k2, v2 = k.reshape(len(k), -1), v.reshape(len(v), -1)
        cache.scales[i] = fp8rl.kv_calibrate(k2, v2)
        fp8rl.kv_append(k2, v2, slots, cache.k[i], cache.v[i], cache.scales[i])
        return fp8rl.attn_prefill(q, k, v, plan)[0].view(len(q), -1)

    xq, sx = rollout_layers(cfg, weights, q8, weights["embed"][tokens.long()], attend)
    last = cu[1:].long() - 1
    return fp8rl.gemm(xq[last], sx[:, last].contiguous(), *q8["head"])


def decode(cfg: Config, weights, q8, tokens, lens, cache: Cache, going=None):
    """One token per sequence at position lens (device int32), or for those with
    going = 1 (device int32); the logits."""
    slots = cache.reserve(count=going)

    def attend(i, q, k, v):
        q, _ = fp8rl.rotary_kv_append(q, k, v, lens, weights["rotary"], slots, cache.k[i], cache.v[i], cache.scales[i])
        return fp8rl.attn_decode(q, cache.k[i], cache.v[i], cache.table, cache.lens, cache.scales[i], cache.page,
                                 workspace=cache.workspace)[0].view(len(q), -1)

    xq, sx = rollout_layers(cfg, weights, q8, weights["embed"][tokens.long()], attend)
    return fp8rl.gemm(xq, sx, *q8["head"])


def train_logits(cfg: Config, weights, tokens, cu, pos):
    """The training policy's logits (bf16 linears) of packed sequences, for scoring:
    the attention has no backward pass, so gradients end at these logits."""
    plan = fp8rl.attn_prefill_plan(cu, tokens.numel(), cfg.q_heads, cfg.kv_heads)

    def norm(x, w):
        x = x.float()
        return (x * torch.rsqrt((x * x).mean(-1, keepdim=True) + cfg.eps) * w.float()).bfloat16()

    h = weights["embed"][tokens.long()]
    nq, nk = cfg.q_heads, cfg.q_heads + cfg.kv_heads
    for lw in weights["layers"]:
        qkv = (norm(h, lw["norm1"]) @ lw["qkv"].T).view(-1, cfg.q_heads + 2 * cfg.kv_heads, cfg.head_dim)
        q, k = fp8rl.rotary(qkv[:, :nq], qkv[:, nq:nk], pos.to(torch.int32), weights["rotary"])
        h = h + fp8rl.attn_prefill(q, k, qkv[:, nk:], plan)[0].view(len(h), -1) @ lw["o"].T
        y = norm(h, lw["norm2"])
        h = h + (torch.nn.functional.silu(y @ lw["gate"].T) * (y @ lw["up"].T)) @ lw["down"].T
    return norm(h, weights["norm"]) @ weights["head"].T


def run(cfg: Config, prompts: int = 8, new_tokens: int = 32, seed: int = 0, temperature: float = 1.0, answers: int = 1,
        top_p: float = 1.0, eos: int = -1):
    """One step; an answer ends with the token `eos` (-1: none does)."""
    dev = torch.device("cuda")
    g = torch.Generator(dev).manual_seed(seed)
    weights = make_weights(cfg, seed)
    q8 = weight_sync(cfg, weights)
    lens = torch.randint(5, 200, (prompts,), generator=g, device=dev)
    total = int(lens.sum())
    cu = torch.cat([lens.new_zeros(1), lens.cumsum(0)]).to(torch.int32)
    seq = torch.repeat_interleave(torch.arange(prompts, device=dev), lens)
    pos = torch.arange(total, device=dev) - cu[:-1].long()[seq]
    prompt = torch.randint(0, cfg.vocab, (total,), generator=g, device=dev).to(torch.int32)
    cache = Cache(cfg, prompts, int(lens.max()) + new_tokens, answers)

    # rollout: `answers` to each prompt, a token drawn each step, with its log probability
    logits = prefill(cfg, weights, q8, prompt, cu, seq, pos, cache)
    of = torch.arange(prompts, device=dev).repeat_interleave(answers)  # the prompt of each answer
    if answers > 1:
        cache.select(of.to(torch.int32))
        logits = logits[of]
    rows = torch.arange(len(of), device=dev, dtype=torch.int32)
    at = lens[of].to(torch.int32)
    going = torch.ones_like(at)
    answer, lp_rollout = [], []
    for _ in range(new_tokens):
        # (a number below 0: no draw for an answer that has ended, its token is -1)
        uniform = torch.where(going > 0, torch.rand(len(of), generator=g, device=dev, dtype=torch.float64), -1.0)
        token, lp, _, _ = fp8rl.sample(logits, uniform, temperature, top_p=top_p)
        answer.append(token)
        lp_rollout.append(lp)
        if eos >= 0:
            going = going * (token != eos)
            cache.select(torch.where(going > 0, rows, -1), in_place=True)
        logits = decode(cfg, weights, q8, token.clamp(min=0), at, cache, going)
        at = at + 1
    answer, lp_rollout = torch.stack(answer, 1), torch.stack(lp_rollout, 1)

    # scoring: position i predicts token i + 1; only generated tokens count
    full_lens = lens[of] + new_tokens
    cu2 = torch.cat([lens.new_zeros(1), full_lens.cumsum(0)]).to(torch.int32)
    seq2 = torch.repeat_interleave(torch.arange(len(of), device=dev), full_lens)
    pos2 = torch.arange(int(full_lens.sum()), device=dev) - cu2[:-1].long()[seq2]
    tokens = torch.empty_like(pos2, dtype=torch.int32)
    generated = pos2 >= lens[of][seq2]
    tokens[~generated] = prompt[(cu[:-1].long()[of][seq2] + pos2)[~generated]]
    tokens[generated] = answer.reshape(-1)
    target = torch.full_like(tokens, -1)
    target[:-1] = torch.where(generated[1:], tokens[1:], -1)  # -1: prompt positions (and ended answers) have no token to score
    logits = train_logits(cfg, weights, tokens.clamp(min=0), cu2, pos2)
    lp, entropy, stats, _, _ = fp8rl.logprobs(logits, target, temperature=temperature)
    on = target >= 0
    rollout = torch.zeros_like(lp)
    rollout[on] = lp_rollout.reshape(-1)[answer.reshape(-1) >= 0]
    w, kl = fp8rl.tis_weights(lp, rollout, on.to(torch.uint8))
    # loss = -sum w A lp / n - 0.01 sum entropy / n, with a random advantage per answer
    advantage = torch.randn(len(of), generator=g, device=dev)[seq2]
    n = on.sum()
    grad = fp8rl.logprobs_backward(logits, target, stats, entropy, -w * advantage / n, -0.01 * on / n, temperature=temperature)
    status = fp8rl.fp8rl_sync_status()
    if status != 0:
        raise fp8rl.Fp8rlError(status, "rollout step")
    return {"answer": answer, "lp_rollout": lp_rollout, "lp_train": lp, "entropy": entropy, "weights": w, "kl": kl, "grad": grad,
            "scored": on, "logits": logits, "target": target, "cache": cache, "going": going}


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--prompts", type=int, default=8)
    ap.add_argument("--answers", type=int, default=4)
    ap.add_argument("--new-tokens", type=int, default=32)
    a = ap.parse_args()
    fp8rl.load_library(build_if_missing=True)
    r = run(Config(layers=a.layers), a.prompts, a.new_tokens, answers=a.answers)
    on = r["scored"]
    mean, total, count = r["kl"].tolist()
    print(f"{int(count)} generated tokens; mean log probability rollout {r['lp_rollout'][r['answer'] >= 0].mean():.4f}, training "
          f"{r['lp_train'][on].mean():.4f}; mismatch KL {mean:.5f}; mean weight {r['weights'][on].mean():.4f}; "
          f"mean entropy {r['entropy'][on].mean():.4f}; |d logits| {r['grad'].float().norm():.5f}; "
          f"{r['cache'].compact()} pages in use")


if __name__ == "__main__":
    main()
