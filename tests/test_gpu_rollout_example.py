"""The example rollout step end to end: prefill, decode over the E4M3 cache,
scoring, importance weights and the gradient, and what ties them together."""
import importlib.util
import os

import pytest
import torch

import fp8_w8a8_rollout_gb300 as fp8rl

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    fp8rl.load_library(build_if_missing=True)
    spec = importlib.util.spec_from_file_location("rollout_step", os.path.join(ROOT, "examples", "rollout_step.py"))
    m = importlib.util.module_from_spec(spec)
    import sys
    sys.modules["rollout_step"] = m
    spec.loader.exec_module(m)
    return m


def test_rollout_step(example):
    r = example.run(example.Config(layers=3), prompts=5, new_tokens=12, seed=3)
    on = r["scored"]
    assert int(on.sum()) == 5 * 12 and r["kl"][2].item() == 60
    assert bool(torch.isfinite(r["lp_train"]).all()) and bool(torch.isfinite(r["lp_rollout"]).all())
    # the weights are those of the two log probabilities
    ratio = torch.exp(r["lp_train"][on].double() - r["lp_rollout"].reshape(-1).double()).clamp(max=2.0)
    assert bool(((r["weights"][on].double() - ratio).abs() <= 1e-5).all()) and bool((r["weights"][~on] == 0).all())
    # log probabilities against fp64 on the trainer's own logits
    ref = torch.log_softmax(r["logits"].double(), 1).gather(1, r["target"].clamp(min=0).long()[:, None])[:, 0]
    assert bool(((r["lp_train"] - ref).abs()[on] <= 1e-5).all())
    # a softmax gradient's row sums to zero (bf16 rounding of its terms aside), and unscored rows have none
    g = r["grad"].double()
    assert bool((g.sum(1).abs() <= 2.0 ** -8 * g.abs().sum(1)).all()) and bool((g[~on] == 0).all())
    # the FP8 rollout and the bf16 trainer agree on a random model to well within one nat
    assert abs(r["kl"][0].item()) < 0.5


def test_decode_continues_what_prefill_would_give(example):
    """A prompt's next-token logits from prefill, and from prefill of all but
    its last token and one decode step: the same model, but that the decode step
    reads its keys and values as E4M3."""
    cfg = example.Config(layers=2)
    weights = example.make_weights(cfg, 1)
    q8 = example.weight_sync(cfg, weights)
    g = torch.Generator("cuda").manual_seed(2)
    n = 150
    tokens = torch.randint(0, cfg.vocab, (n,), generator=g, device="cuda").to(torch.int32)

    def fill(m):
        cache = example.Cache(cfg, 1, n + 1)
        cu = torch.tensor([0, m], dtype=torch.int32, device="cuda")
        pos = torch.arange(m, device="cuda")
        return cache, example.prefill(cfg, weights, q8, tokens[:m], cu, torch.zeros_like(pos), pos, cache)

    _, want = fill(n)
    cache, _ = fill(n - 1)
    got = example.decode(cfg, weights, q8, tokens[n - 1:], torch.tensor([n - 1], dtype=torch.int32, device="cuda"), cache)
    assert fp8rl.fp8rl_sync_status() == 0
    a, b = want.double().flatten(), got.double().flatten()
    # E4M3 keeps 4 significant bits: a relative error of at most 2^-4 on every key and value, averaged over 150 of them
    assert float((a - b).norm() / a.norm()) < 2.0 ** -4
