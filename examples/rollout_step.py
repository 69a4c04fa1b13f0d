"""One step of FP8 rollout RL on a small random decoder, with every stage on the
library's kernels.

    python examples/rollout_step.py [--layers 4] [--prompts 8] [--new-tokens 32]

1. weight sync: the bf16 weights are quantised to E4M3 (128x128 blocks);
2. prefill of packed prompts: norm with E4M3 output, qkv GEMM, causal attention
   over the packed prompts, KV calibration and append into the paged E4M3
   cache, output projection, fused gate-up, down projection;
3. decode, a token per sequence and step: the same layers with attention over
   the E4M3 cache, then the logits' log probabilities, entropy and best
   alternatives (the most likely token is taken);
4. scoring by the training policy: the bf16 weights in torch matmuls, the same
   packed attention, log probabilities of the sampled tokens;
5. truncated importance sampling weights and the mismatch KL, and the gradient
   of the weighted loss with respect to the trainer's logits.

The decoder has the usual parts (RMS norms, grouped query heads, rotary
positions, SwiGLU); rotary positions and embedding lookup are plain torch.
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
            "norm": torch.ones(cfg.hidden, device=device).bfloat16(), "head": w(cfg.vocab, cfg.hidden) * 4}


def weight_sync(cfg: Config, weights):
    """The E4M3 weights of a step's rollout: (codes, scales) per linear."""
    out = []
    for lw in weights["layers"]:
        out.append({n: fp8rl.quant_weight(lw[n]) for n in ("qkv", "o", "down")} |
                   {"gate_up": fp8rl.quant_gate_up_interleaved(lw["gate"], lw["up"])})
    return {"layers": out, "head": fp8rl.quant_weight(weights["head"])}


def rotary(x: torch.Tensor, pos: torch.Tensor) -> torch.Tensor:
    """Rotary positions of [tokens, heads, d] at int positions [tokens]."""
    half = x.shape[-1] // 2
    angle = pos.float()[:, None] * 10000.0 ** (-torch.arange(half, device=x.device).float() / half)
    c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    a, b = x[..., :half].float(), x[..., half:].float()
    return torch.cat([a * c - b * s, a * s + b * c], -1).to(x.dtype)


class Cache:
    """The paged E4M3 KV cache of a batch: per layer K, V and their scales."""

    def __init__(self, cfg: Config, batch: int, max_len: int, device="cuda"):
        self.blocks = -(-max_len // cfg.page)
        slots = batch * self.blocks * cfg.page
        self.k = [torch.zeros(slots, cfg.kv_heads * cfg.head_dim, dtype=torch.uint8, device=device) for _ in range(cfg.layers)]
        self.v = [torch.zeros_like(k) for k in self.k]
        self.scales = [None] * cfg.layers
        perm = torch.randperm(batch * self.blocks, device=device).to(torch.int32)  # pages are where they are
        self.table = perm.view(batch, self.blocks)
        self.page = cfg.page
        self.workspace = fp8rl.attn_decode_workspace(cfg.q_heads, cfg.kv_heads, cfg.head_dim)

    def slots(self, seq: torch.Tensor, pos: torch.Tensor) -> torch.Tensor:
        return (self.table[seq, pos // self.page] * self.page + pos % self.page).to(torch.int32)


def rollout_layers(cfg: Config, weights, q8, x, pos, attend):
    """The FP8 decoder stack on x [tokens, hidden]; attend(layer, q, k, v)
    returns [tokens, q_heads * head_dim].  Returns the E4M3 final norm."""
    h, delta = x, None  # the residual stream, and what the last branch adds to it
    for i, (lw, qw) in enumerate(zip(weights["layers"], q8["layers"])):
        if delta is None:
            xq, sx, _ = fp8rl.rmsnorm_quant(h, lw["norm1"], eps=cfg.eps)
        else:
            xq, sx, h = fp8rl.rmsnorm_quant(delta, lw["norm1"], h, eps=cfg.eps)
        qkv = fp8rl.gemm(xq, sx, *qw["qkv"]).view(-1, cfg.q_heads + 2 * cfg.kv_heads, cfg.head_dim)
        nq, nk = cfg.q_heads, cfg.q_heads + cfg.kv_heads
        q, k = rotary(qkv[:, :nq], pos), rotary(qkv[:, nq:nk], pos)
        o, _, _ = fp8rl.gemm_act_quant(attend(i, q, k, qkv[:, nk:]), *qw["o"])
        xq, sx, h = fp8rl.rmsnorm_quant(o, lw["norm2"], h, eps=cfg.eps)
        hq, hs = fp8rl.gemm_swiglu_quant(xq, sx, *qw["gate_up"])
        delta = fp8rl.gemm(hq, hs, *qw["down"])
    xq, sx, _ = fp8rl.rmsnorm_quant(delta, weights["norm"], h, eps=cfg.eps)
    return xq, sx


def prefill(cfg: Config, weights, q8, tokens, cu, seq, pos, cache: Cache):
    """Fills the cache with packed prompts; logits bf16 of each prompt's last token."""
    plan = fp8rl.attn_prefill_plan(cu, tokens.numel(), cfg.q_heads, cfg.kv_heads)
    slots = cache.slots(seq, pos)

    def attend(i, q, k, v):
        k2, v2 = k.reshape(len(k), -1), v.reshape(len(v), -1)
        cache.scales[i] = fp8rl.kv_calibrate(k2, v2)
        fp8rl.kv_append(k2, v2, slots, cache.k[i], cache.v[i], cache.scales[i])
        return fp8rl.attn_prefill(q, k, v, plan)[0].view(len(q), -1)

    xq, sx = rollout_layers(cfg, weights, q8, weights["embed"][tokens.long()], pos, attend)
    last = cu[1:].long() - 1
    return fp8rl.gemm(xq[last], sx[:, last].contiguous(), *q8["head"])


def decode(cfg: Config, weights, q8, tokens, lens, cache: Cache):
    """One token per sequence at position lens (device int32); its logits."""
    seq = torch.arange(tokens.numel(), device=tokens.device)
    slots, after = cache.slots(seq, lens), lens + 1

    def attend(i, q, k, v):
        fp8rl.kv_append(k.reshape(len(k), -1), v.reshape(len(v), -1), slots, cache.k[i], cache.v[i], cache.scales[i])
        return fp8rl.attn_decode(q, cache.k[i], cache.v[i], cache.table, after, cache.scales[i], cache.page,
                                 workspace=cache.workspace)[0].view(len(q), -1)

    xq, sx = rollout_layers(cfg, weights, q8, weights["embed"][tokens.long()], lens, attend)
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
        q, k = rotary(qkv[:, :nq], pos), rotary(qkv[:, nq:nk], pos)
        h = h + fp8rl.attn_prefill(q, k, qkv[:, nk:], plan)[0].view(len(h), -1) @ lw["o"].T
        y = norm(h, lw["norm2"])
        h = h + (torch.nn.functional.silu(y @ lw["gate"].T) * (y @ lw["up"].T)) @ lw["down"].T
    return norm(h, weights["norm"]) @ weights["head"].T


def run(cfg: Config, prompts: int = 8, new_tokens: int = 32, seed: int = 0, temperature: float = 1.0, topk: int = 5):
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
    cache = Cache(cfg, prompts, int(lens.max()) + new_tokens)

    # rollout: the most likely token each step, with its log probability
    logits = prefill(cfg, weights, q8, prompt, cu, seq, pos, cache)
    at = lens.to(torch.int32)
    answer, lp_rollout = [], []
    for _ in range(new_tokens):
        # (any valid token scores the row; the first alternative is the one taken)
        _, _, _, ids, top_lp = fp8rl.logprobs(logits, at.clamp(max=0), temperature=temperature, topk=topk)
        answer.append(ids[:, 0].contiguous())
        lp_rollout.append(top_lp[:, 0])
        logits = decode(cfg, weights, q8, answer[-1], at, cache)
        at = at + 1
    answer, lp_rollout = torch.stack(answer, 1), torch.stack(lp_rollout, 1)

    # scoring: position i predicts token i + 1; only generated tokens count
    full_lens = lens + new_tokens
    cu2 = torch.cat([lens.new_zeros(1), full_lens.cumsum(0)]).to(torch.int32)
    seq2 = torch.repeat_interleave(torch.arange(prompts, device=dev), full_lens)
    pos2 = torch.arange(int(full_lens.sum()), device=dev) - cu2[:-1].long()[seq2]
    tokens = torch.empty_like(pos2, dtype=torch.int32)
    generated = pos2 >= lens[seq2]
    tokens[~generated] = prompt
    tokens[generated] = answer.reshape(-1)
    target = torch.full_like(tokens, -1)
    target[:-1] = torch.where(generated[1:], tokens[1:], -1)  # -1: prompt positions have no token to score
    logits = train_logits(cfg, weights, tokens, cu2, pos2)
    lp, entropy, stats, _, _ = fp8rl.logprobs(logits, target, temperature=temperature)
    on = target >= 0
    rollout = torch.zeros_like(lp)
    rollout[on] = lp_rollout.reshape(-1)
    w, kl = fp8rl.tis_weights(lp, rollout, on.to(torch.uint8))
    # loss = -sum w A lp / n - 0.01 sum entropy / n, with a random advantage per sequence
    advantage = torch.randn(prompts, generator=g, device=dev)[seq2]
    n = on.sum()
    grad = fp8rl.logprobs_backward(logits, target, stats, entropy, -w * advantage / n, -0.01 * on / n, temperature=temperature)
    status = fp8rl.fp8rl_sync_status()
    if status != 0:
        raise fp8rl.Fp8rlError(status, "rollout step")
    return {"answer": answer, "lp_rollout": lp_rollout, "lp_train": lp, "entropy": entropy, "weights": w, "kl": kl, "grad": grad,
            "scored": on, "logits": logits, "target": target}


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--prompts", type=int, default=8)
    ap.add_argument("--new-tokens", type=int, default=32)
    a = ap.parse_args()
    fp8rl.load_library(build_if_missing=True)
    r = run(Config(layers=a.layers), a.prompts, a.new_tokens)
    on = r["scored"]
    mean, total, count = r["kl"].tolist()
    print(f"{int(count)} generated tokens; mean log probability rollout {r['lp_rollout'].mean():.4f}, training "
          f"{r['lp_train'][on].mean():.4f}; mismatch KL {mean:.5f}; mean weight {r['weights'][on].mean():.4f}; "
          f"mean entropy {r['entropy'][on].mean():.4f}; |d logits| {r['grad'].float().norm():.5f}")


if __name__ == "__main__":
    main()
